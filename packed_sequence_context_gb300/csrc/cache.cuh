// The paged key-value cache (thd_kv_cache in the header) as the kernels of
// cache.cu and decode.cu see it, and what they share: where a slot lies, the
// power-of-two scales of an 8-bit cache, the sticky status word.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"

namespace thd {

// A slot-wise array [pages][slots][heads]: element strides, in whichever order.
struct SlotStrides {
  int64_t page, slot, head;
};

// Division by a number the host knows, without a division: for 0 <= x <= 2^30 and
// 1 <= d <= 2^30, x / d = x mul >> shift with mul = ceil(2^shift / d), shift =
// 30 + ceil(log2 d) (mul d exceeds 2^shift by less than d, x times which stays
// below 2^shift).
struct Divisor {
  uint32_t d, mul, shift;
};
inline Divisor divisor(uint32_t d) {
  uint32_t log = 0;
  while ((1u << log) < d) ++log;
  return Divisor{d, (uint32_t)((((uint64_t)1 << (30 + log)) + d - 1) / d), 30 + log};
}

struct CacheView {
  uint8_t* k;
  uint8_t* v;
  uint8_t* k_exp;  // null: bf16
  uint8_t* v_exp;
  SlotStrides row;  // of k and v, in bytes
  SlotStrides exp;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* kv_len;
  int64_t num_pages;
  int64_t capacity;  // slots a sequence's row of the table names: max_pages * page_size
  Divisor page;      // slots of one
  int B, Hkv, D;
};

struct AppendParams {
  CacheView c;
  const uint16_t* in[2];  // k, v: rows of [Hkv, D]
  int64_t in_stride[2];
  int64_t T;
  const int32_t* cu;  // null: row t is sequence t's
  float* weight;      // may be null, as pos
  SlotStrides weight_at;
  int32_t* pos;
  SlotStrides pos_at;
  const int32_t* seen;  // null: kv_len
  int32_t* status;
  int tokens;     // a block
  Divisor heads;  // Hkv
};

// An item that several blocks shared, as its last block leaves it for the join:
// query heads h .. h + heads - 1 of sequence b, parts of `count` blocks from
// `first` on.  count 0: none.
struct DecodeJoin {
  int b, h, heads, first, count;
};

struct DecodeParams {
  CacheView c;
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* o;
  float* lse;  // [Hq][B]
  int Hq, G, blocks;  // query heads of a kv head; how many runs of kHeads (a work item's) they are cut into
  float scale, cap;   // cap 0: none
  const float* slopes;
  const int32_t* start;
  const int32_t* pos;
  SlotStrides pos_at;
  const int32_t* seen;
  const float* weight_in;
  float* weight_out;  // null: no weights
  SlotStrides weight_at;
  int32_t* status;
  // workspace
  float* part;      // [2 grid][heads of an item][D]
  float* part_ml;   // [2 grid][heads of an item][3]
  DecodeJoin* joins;  // [items], or of the items that end in a block's share [grid]
  float* lse2;      // [B][Hq] in base 2, with weights
  float* scores;    // [B][Hkv][capacity][G], with weights
  int grid;
  bool by_item;
};

struct EvictParams {
  CacheView c;
  const float* weight_in;
  float* weight_out;
  SlotStrides weight_at;
  const int32_t* pos_in;
  int32_t* pos_out;
  SlotStrides pos_at;
  const int32_t* seen;
  int32_t* new_len;
  int32_t* status;
  int32_t* moves;  // [B Hkv][2][room]: evicted slots in front of the budget, kept ones behind it
  int64_t room;
  int budget, sinks, recent;
  int share;  // blocks of an item (one cluster)
  int held;   // slots whose keys a block holds in shared memory
};

cudaError_t launch_append(const AppendParams& p, cudaStream_t st);
cudaError_t launch_decode(DecodeParams p, cudaStream_t st);
cudaError_t launch_evict(EvictParams p, cudaStream_t st);

constexpr int kDecodeMaxGrid = 512;    // blocks of a decode launch (the workspace holds two parts for each)
constexpr int kDecodeMaxGroup = 512;   // query heads of a kv head
int decode_heads(int G);               // query heads of a work item
// The most blocks that a decode of these sizes has work for, whatever the lengths.
int decode_blocks(int B, int Hkv, int G, int64_t capacity);

// A kernel's limit of dynamic shared memory, raised once on each device (`done`:
// the kernel's own).
template <typename K>
cudaError_t allow_smem(K* kernel, size_t bytes, bool (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev >= 0 && dev < 64 && done[dev])) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  return e;
}

// Launches a kernel that may start while the one in front of it in the stream
// ends: its blocks begin with depend(), which waits for that kernel's end and
// the writes of it, and with follow(), which lets the next such kernel start.
// What this hides is the launch, a microsecond or two of each.
template <typename... A>
cudaError_t launch_following(void (*kernel)(A...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  count_launch();
  return e;
}

#ifdef __CUDACC__
__device__ inline void follow() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ inline void depend() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The status word of the cache's operators is sticky: the largest code since
// its owner zeroed it (whatever the order of the blocks).
__device__ inline void raise(int32_t* status, int code) { atomicMax(status, code); }

// A sequence's slots, or 0 where its length lies outside what the table can hold.
__device__ inline int slots_of(const CacheView& c, int b, bool& bad) {
  const int n = c.kv_len[b];
  bad = n < 0 || n > c.capacity;
  return bad ? 0 : n;
}

struct Place {
  uint32_t page, slot;
};
__device__ inline Place place_of(const CacheView& c, int j) {
  const uint32_t q = (uint32_t)(((uint64_t)(uint32_t)j * c.page.mul) >> c.page.shift);
  return Place{q, (uint32_t)j - q * c.page.d};
}

// The page of a sequence's slot, or -1 where the table names none of the cache.
__device__ inline int page_of(const CacheView& c, int b, uint32_t page_index) {
  const int p = c.table[b * c.table_stride + page_index];
  return (uint32_t)p < (uint64_t)c.num_pages && p >= 0 ? p : -1;
}

__device__ inline int64_t at(const SlotStrides& s, int page, uint32_t slot, int head) {
  return page * s.page + slot * s.slot + head * s.head;
}
#endif

}  // namespace thd
