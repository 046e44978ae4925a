// What fills a paged key-value cache and what keeps it small: thd_cache_append
// and thd_cache_evict (see the header).
#include <cooperative_groups.h>
#include <cuda_fp8.h>

#include "cache.cuh"
#include "ptx.cuh"
#include "vec8.cuh"

namespace thd {

// ------------------------------------------------------------------ append
// A block takes `tokens` rows; its first threads find each row's sequence (a
// binary search of the offsets) and where its slot lies, then its warps walk
// (token, head) pairs, the key's row on some lanes and the value's on others, two
// runs of eight elements a lane, three pairs in flight.  Bound by HBM: the rows are
// read and written once, 16 bytes a lane (8 written for e4m3).  The search and the page
// are three to six loads one after the other, so a block takes many rows where
// there are many (up to 64; 32: 136 us, 64: 130 for 131,072 tokens of 8 heads of
// 128 to e4m3, 93% of the rate of a plain copy; a packed batch of 14,900 tokens of 16
// heads as bf16 44 us, 86%).
//
// e4m3 with a power of two for each row and head: e is the smallest exponent
// with max |row| <= 448 * 2^e, so dividing is exact and the only rounding is the
// one to e4m3's grid; a row of bf16 products keeps all of the format's precision
// (a scale of max / 448 would round twice and gain nothing but the last half
// binade).
constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 64;  // at most, a block

// The stored exponent of a row whose largest magnitude (bf16, sign off) is
// `big`: 448 = 1.75 * 2^8, so 2^(x - 8) serves up to a mantissa of 1.75.  No
// lower than 2^-60: what a row of smaller numbers would gain no score or output
// shows.  A row of zeros takes 1; one with an infinity or NaN is marked NaN.
__device__ inline int row_exponent(uint32_t big) {
  if (big >= 0x7f80u) return 255;
  if (big == 0) return 127;
  const int e = (int)(big >> 7) - 8 + ((big & 0x7fu) > 0x60u ? 1 : 0);
  return e < 67 ? 67 : e;
}

// Where a block's row goes: byte offset of its slot's rows, element offsets of
// its numbers; row -1: nowhere.
struct AppendRow {
  int64_t row, exp, weight, pos;
  int number;
};

template <bool kFp8, int D>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
  __shared__ AppendRow s_row[kAppendTokens];
  const CacheView& c = p.c;
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
  const int count = (int)(p.T - t0 < p.tokens ? p.T - t0 : p.tokens);
  if (p.cu && blockIdx.x == 0) {  // what no row shows: the offsets themselves
    for (int b = threadIdx.x; b < c.B; b += kAppendThreads) {
      if (b == 0 && p.cu[0] != 0) raise(p.status, THD_DEV_ERR_NONZERO_START);
      if (p.cu[b + 1] < p.cu[b]) raise(p.status, THD_DEV_ERR_NOT_MONOTONE);
      if (p.cu[b + 1] > p.T) raise(p.status, THD_DEV_ERR_EXCEEDS_BUF);
    }
  }
  if (threadIdx.x < count) {
    const int64_t t = t0 + threadIdx.x;
    AppendRow out = {-1, 0, 0, 0, 0};
    int b = (int)t;
    int64_t back = 1;  // rows from this one to its sequence's end
    bool mine = t < c.B;
    if (p.cu) {  // the last sequence that starts at or before t
      int lo = 0, hi = c.B;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (p.cu[mid + 1] <= t) lo = mid + 1; else hi = mid;
      }
      b = lo;
      mine = b < c.B && p.cu[b] <= t;
      back = mine ? p.cu[b + 1] - t : 0;
    }
    if (mine) {
      const int64_t n = c.kv_len[b], j = n - back;
      if (n > c.capacity || j < 0) {
        raise(p.status, THD_DEV_ERR_KV_LEN);
      } else {
        const Place x = place_of(c, (int)j);
        const int page = page_of(c, b, x.page);
        if (page < 0) {
          raise(p.status, THD_DEV_ERR_PAGE);
        } else {
          out.row = at(c.row, page, x.slot, 0);
          out.exp = at(c.exp, page, x.slot, 0);
          out.weight = at(p.weight_at, page, x.slot, 0);
          out.pos = at(p.pos_at, page, x.slot, 0);
        }
        out.number = (int)((p.seen ? (int64_t)p.seen[b] : n) - back);
      }
    }
    s_row[threadIdx.x] = out;
  }
  __syncthreads();
  constexpr int kLanes = D / 16, kPairs = 32 / (2 * kLanes);  // of a row; a warp's (token, head) pairs at a time
  constexpr int kAtOnce = 3, kStride = kPairs * kAppendThreads / 32;
  const int lane = threadIdx.x & 31, piece = lane % kLanes, kv = lane / kLanes & 1;
  const uint16_t* const in = p.in[kv] + t0 * p.in_stride[kv] + 8 * piece;  // and D / 2 elements further
  uint8_t* const cache = (kv ? c.v : c.k) + (kFp8 ? 8 : 16) * piece;
  const int pairs = count * c.Hkv;
  // every lane walks alike: the exponent is a shuffle
  for (int r0 = (threadIdx.x >> 5) * kPairs; r0 < pairs; r0 += kAtOnce * kStride) {
    Vec8<uint16_t> x[kAtOnce][2];
    int tok[kAtOnce], g[kAtOnce];
    bool ok[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int r = r0 + u * kStride + lane / (2 * kLanes);
      tok[u] = r < pairs ? (int)(((uint64_t)(uint32_t)r * p.heads.mul) >> p.heads.shift) : 0;
      g[u] = r - tok[u] * c.Hkv;
      ok[u] = r < pairs && s_row[tok[u]].row >= 0;
      x[u][0].v = x[u][1].v = make_uint4(0, 0, 0, 0);
      if (ok[u]) {
        const uint16_t* const from = in + tok[u] * p.in_stride[kv] + g[u] * D;
        x[u][0].load(from);
        x[u][1].load(from + D / 2);
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const AppendRow& to = s_row[tok[u]];
      uint8_t* const out = cache + to.row + g[u] * c.row.head;
      if (!kFp8) {
        if (ok[u]) {
          x[u][0].store(reinterpret_cast<uint16_t*>(out));
          x[u][1].store(reinterpret_cast<uint16_t*>(out) + D / 2);
        }
      } else {
        const uint32_t w[8] = {x[u][0].v.x, x[u][0].v.y, x[u][0].v.z, x[u][0].v.w, x[u][1].v.x, x[u][1].v.y, x[u][1].v.z, x[u][1].v.w};
        uint32_t big = 0;  // of both halves: a bf16's order is its bits'
#pragma unroll
        for (int q = 0; q < 8; ++q) big = __vmaxu2(big, w[q] & 0x7fff7fffu);
#pragma unroll
        for (int d = kLanes / 2; d > 0; d >>= 1) big = __vmaxu2(big, __shfl_xor_sync(0xffffffffu, big, d));
        big = max(big >> 16, big & 0xffffu);
        const int e = row_exponent(big);
        const float inv = __uint_as_float((uint32_t)(254 - e) << 23);  // 2^(127 - e)
        uint32_t y[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float f[4];
          fmul2(f[0], f[1], __uint_as_float(w[2 * q] << 16), __uint_as_float(w[2 * q] & 0xffff0000u), inv, inv);
          fmul2(f[2], f[3], __uint_as_float(w[2 * q + 1] << 16), __uint_as_float(w[2 * q + 1] & 0xffff0000u), inv, inv);
          const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[0], f[1]), __NV_SATFINITE, __NV_E4M3);
          const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[2], f[3]), __NV_SATFINITE, __NV_E4M3);
          y[q] = lo | hi << 16;
        }
        if (e == 255) y[0] = y[1] = y[2] = y[3] = 0x7f7f7f7fu;
        if (ok[u]) {
          *reinterpret_cast<uint2*>(out) = make_uint2(y[0], y[1]);
          *reinterpret_cast<uint2*>(out + D / 2) = make_uint2(y[2], y[3]);
          if (piece == 0) (kv ? c.v_exp : c.k_exp)[to.exp + g[u] * c.exp.head] = (uint8_t)e;
        }
      }
      if (ok[u] && piece == 0) {
        if (kv == 0 && p.weight) p.weight[to.weight + g[u] * p.weight_at.head] = 0.f;
        if (kv == 1 && p.pos) p.pos[to.pos + g[u] * p.pos_at.head] = to.number;
      }
    }
  }
}

cudaError_t launch_append(const AppendParams& a, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  AppendParams p = a;
  const int64_t n = (a.T + 16 * num_sms() - 1) / (16 * num_sms());  // 16 blocks an SM first
  p.tokens = (int)(n > kAppendTokens ? kAppendTokens : n);
  p.heads = divisor((uint32_t)a.c.Hkv);
  const unsigned grid = (unsigned)((a.T + p.tokens - 1) / p.tokens);
  prof_before(THD_KERNEL_CACHE_APPEND, st);
  if (a.c.k_exp && a.c.D == 64) append_kernel<true, 64><<<grid, kAppendThreads, 0, st>>>(p);
  if (a.c.k_exp && a.c.D == 128) append_kernel<true, 128><<<grid, kAppendThreads, 0, st>>>(p);
  if (!a.c.k_exp && a.c.D == 64) append_kernel<false, 64><<<grid, kAppendThreads, 0, st>>>(p);
  if (!a.c.k_exp && a.c.D == 128) append_kernel<false, 128><<<grid, kAppendThreads, 0, st>>>(p);
  count_launch();
  const cudaError_t e = cudaGetLastError();
  prof_after(THD_KERNEL_CACHE_APPEND, st);
  return e;
}

// ------------------------------------------------------------------ evict
// One cluster of `share` blocks an item (sequence, kv head).  Every block holds
// its part of the slots' weights in shared memory as integers of the same
// order (protected slots on top), so they are read once; the budget-th largest
// is found by its 8-bit digits (a histogram each, added up over the cluster
// through distributed shared memory; after two of them the candidates are mostly
// few enough to be compared), ties and the slots to move are numbered by
// counts and ballots, and the cluster's blocks then move rows.  Kept
// slots in front of the budget stay where they are and evicted ones there take
// the kept ones behind it, in order: the fewest bytes that can move, sources
// (behind) and targets (in front) that never meet, and nothing to wait for
// between them.
//
// Bound by latency, but for the moves.  By the blocks' clocks (at 1.9 GHz), 4
// sequences of 32,768 slots and 8 kv heads cut to 4096 in clusters of 8: keys 6.7 us,
// the two digits 5.3 and 4.9 (a walk over the keys and two barriers of the cluster
// each), candidates 4.0, counts 2.6, lists of moves 2.9, the barrier behind
// them 1.6, moves at the rate of a plain copy 17.4, the numbers that stay 2.3: 48
// of 49 us.  32 of 2000 to 2112 slots cut to 2048, a block an item: 2.7, 2.7 and 2.1,
// 1.8, 1.6, 1.7, 0.7, 1.8, 1.5: 16.5 of 19 us, walks over four keys a thread each.
namespace cg = cooperative_groups;

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kBins = 256;
// Candidates that are compared with one another instead of counted by two more
// digits.  Comparing is quadratic: of 4 sequences of 32,768 slots and 8 kv heads
// with 16, 128, 256, 512, 1024 candidates an item 50.0, 51.4, 54.6, 66.8, 120 us,
// with the digits 51.4 to 52.3; one sequence of 8192 slots 18.5, 19.4, 21.3, 28.4,
// 57.5 against 19.0 to 19.5; 32 of 2112 with 16 and 64 candidates 19.4, 20.3
// against 21.5, 21.9.
constexpr int kFew = 128;
constexpr int kEvictMaxHeld = 40960;  // keys in a block's shared memory (160 KB)

// An integer of the order in which slots stay.  Protected tokens (`age`: how many
// came after) above every weight, +infinity too, the newest on top: where the
// budget holds fewer than are protected, the oldest leave first.  Weights end at
// 0xff800000, which leaves 2^23 - 1 ages apart; those beyond count as one.
__device__ inline uint32_t order_of(float w, bool kept, int64_t age) {
  if (kept) return 0xffffffffu - (age < 0 ? 0u : age < 0x7ffffe ? (uint32_t)age : 0x7ffffeu);
  if (!(w == w)) return 0u;                 // NaN: below everything
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 counts as 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kEvictThreads, 2) evict_kernel(const EvictParams p) {
  extern __shared__ uint32_t s_key[];  // [held]
  __shared__ uint32_t s_hist[kBins], s_scan[kBins / 32];
  __shared__ uint32_t s_digit, s_left, s_many, s_mine;
  __shared__ __align__(16) uint16_t s_few[kFew], s_their[kFew];
  // larger and equal keys in front of the budget and behind it: a warp's, a block's
  __shared__ uint4 s_cnt[kEvictWarps], s_sum;
  const CacheView& c = p.c;
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)(blockIdx.x % p.share), item = (int)(blockIdx.x / p.share);
  const int b = item / c.Hkv, g = item % c.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  bool bad;
  const int n = slots_of(c, b, bad);
  if (g == 0 && rank == 0 && tid == 0) {
    if (bad) raise(p.status, THD_DEV_ERR_KV_LEN);
    p.new_len[b] = n < p.budget ? n : p.budget;
  }
  const int chunk = (n + p.share - 1) / p.share;
  const int lo = rank * chunk < n ? rank * chunk : n, hi = lo + chunk < n ? lo + chunk : n;
  const bool copy_w = p.weight_out != p.weight_in, copy_p = p.pos_out != p.pos_in;

  // weight and position of a slot to the outputs' slot of the same number
  auto carry = [&](int i) {
    const Place x = place_of(c, i);
    const int page = page_of(c, b, x.page);
    if (page < 0) {
      raise(p.status, THD_DEV_ERR_PAGE);
      return;
    }
    const int64_t w = at(p.weight_at, page, x.slot, g), q = at(p.pos_at, page, x.slot, g);
    if (copy_w) p.weight_out[w] = p.weight_in[w];
    if (copy_p) p.pos_out[q] = p.pos_in[q];
  };
  if (n <= p.budget) {  // the whole cluster
    if (copy_w || copy_p)
      for (int i = lo + tid; i < hi; i += kEvictThreads) carry(i);
    return;
  }

  const int seen = p.seen[b];
  auto read_key = [&](int i) -> uint32_t {
    const Place x = place_of(c, i);
    const int page = page_of(c, b, x.page);
    if (page < 0) {
      raise(p.status, THD_DEV_ERR_PAGE);
      return 0u;
    }
    const int pos = p.pos_in[at(p.pos_at, page, x.slot, g)];
    const int64_t age = (int64_t)seen - 1 - pos;
    return order_of(p.weight_in[at(p.weight_at, page, x.slot, g)], pos < p.sinks || age < p.recent, age);
  };
  {
    const int m = hi - lo < p.held ? hi - lo : p.held;
#pragma unroll 8
    for (int i = tid; i < m; i += kEvictThreads) s_key[i] = read_key(lo + i);
  }
  auto key = [&](int i) { return i - lo < p.held ? s_key[i - lo] : read_key(i); };

  // the budget-th largest, digit by digit
  uint32_t prefix = 0, mask = 0, left = (uint32_t)p.budget;
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < kBins) s_hist[tid] = 0;
    __syncthreads();
    for (int i0 = lo; i0 < hi; i0 += kEvictThreads) {
      const int i = i0 + tid;
      const uint32_t k = i < hi ? key(i) : 0u;
      const bool in = i < hi && (k & mask) == prefix;
      const uint32_t d = (k >> shift) & (kBins - 1);
      if (!__any_sync(0xffffffffu, in)) continue;
      // equals in a warp add once
      const uint32_t same = __match_any_sync(0xffffffffu, in ? d : 0xffffffffu);
      if (in && lane == __ffs(same) - 1) atomicAdd(&s_hist[d], (uint32_t)__popc(same));
    }
    cluster.sync();
    uint32_t mine = 0, inc = 0;
    const int bin = kBins - 1 - tid;  // thread 0 has the top one
    if (tid < kBins) {
#pragma unroll 8
      for (int r = 0; r < p.share; ++r) mine += cluster.map_shared_rank(s_hist, r)[bin];
      inc = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += y;
      }
      if (lane == 31) s_scan[warp] = inc;
    }
    __syncthreads();
    if (tid < kBins) {
      for (int w = 0; w < warp; ++w) inc += s_scan[w];
      if (inc - mine < left && left <= inc) {
        s_digit = (uint32_t)bin;
        s_left = left - (inc - mine);
        s_many = mine;
      }
    }
    cluster.sync();  // also: every block has read the histograms
    prefix |= s_digit << shift;
    mask |= (uint32_t)(kBins - 1) << shift;
    left = s_left;
    // Half of the key is known.  If few slots share it, every block takes all
    // their other halves and compares each with each: two rounds of sums over
    // the cluster less.
    const uint32_t many = s_many;
    if (shift != 16 || many > kFew) continue;
    if (tid == 0) s_mine = 0;
    __syncthreads();
    for (int i = lo + tid; i < hi; i += kEvictThreads) {
      const uint32_t k = key(i);
      if ((k & mask) == prefix) s_few[atomicAdd(&s_mine, 1u)] = (uint16_t)k;
    }
    cluster.sync();
    uint32_t count = lane < p.share ? *cluster.map_shared_rank(&s_mine, lane) : 0u, first = count;
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, first, d);
      if (lane >= d) first += y;
    }
    first -= count;
    for (int r = 0; r < p.share; ++r) {
      const uint32_t n_r = __shfl_sync(0xffffffffu, count, r), at_r = __shfl_sync(0xffffffffu, first, r);
      const uint16_t* const from = cluster.map_shared_rank(s_few, r);
      for (uint32_t i = tid; i < n_r; i += kEvictThreads) s_their[at_r + i] = from[i];
    }
    const uint32_t whole = (many + 7) & ~7u;  // padded with the smallest; none of those is counted
    if (many + tid < whole) s_their[many + tid] = 0;
    __syncthreads();
    for (uint32_t i = tid; i < many; i += kEvictThreads) {
      const uint32_t me = s_their[i];
      uint32_t larger = 0, equal = 0;
      for (uint32_t j = 0; j < whole; j += 8) {
        const uint4 v = *reinterpret_cast<const uint4*>(s_their + j);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          larger += ((w[q] & 0xffffu) > me ? 1u : 0u) + ((w[q] >> 16) > me ? 1u : 0u);
          equal += ((w[q] & 0xffffu) == me ? 1u : 0u) + ((w[q] >> 16) == me ? 1u : 0u);
        }
      }
      if (me == 0) equal -= whole - many;
      if (larger < left && left <= larger + equal) {  // so says every thread that has this number
        s_digit = me;
        s_left = left - larger;
      }
    }
    __syncthreads();
    prefix |= s_digit;
    left = s_left;
    break;
  }
  // Kept: keys above `prefix`, and the first `left` slots equal to it.  Every warp
  // counts both kinds in its slots, in front of the budget and behind it; which
  // of the equal ones stay follows from how many there are in front, and with
  // that how many slots each warp has to give and to take.
  const int part = ((hi - lo + kEvictWarps - 1) / kEvictWarps + 31) / 32 * 32;  // a warp's slots
  const int wlo = lo + warp * part < hi ? lo + warp * part : hi, whi = wlo + part < hi ? wlo + part : hi;
  {
    uint4 n4 = make_uint4(0, 0, 0, 0);
    for (int i = wlo + lane; i < whi; i += 32) {
      const uint32_t k = key(i);
      const uint32_t larger = k > prefix ? 1u : 0u, equal = k == prefix ? 1u : 0u, front = i < p.budget ? 1u : 0u;
      n4.x += larger & front;
      n4.y += larger & ~front;
      n4.z += equal & front;
      n4.w += equal & ~front;
    }
    n4.x = __reduce_add_sync(0xffffffffu, n4.x);
    n4.y = __reduce_add_sync(0xffffffffu, n4.y);
    n4.z = __reduce_add_sync(0xffffffffu, n4.z);
    n4.w = __reduce_add_sync(0xffffffffu, n4.w);
    if (lane == 0) s_cnt[warp] = n4;
  }
  __syncthreads();
  const uint4 of_warp = lane < kEvictWarps ? s_cnt[lane] : make_uint4(0, 0, 0, 0);
  if (warp == 0) {
    uint4 n4;
    n4.x = __reduce_add_sync(0xffffffffu, of_warp.x);
    n4.y = __reduce_add_sync(0xffffffffu, of_warp.y);
    n4.z = __reduce_add_sync(0xffffffffu, of_warp.z);
    n4.w = __reduce_add_sync(0xffffffffu, of_warp.w);
    if (lane == 0) s_sum = n4;
  }
  cluster.sync();
  // A row of lanes (blocks, or warps), the counts and the first slot of each:
  // what lies in front of lane `me` (equal ones, evicted slots in front of the
  // budget, kept ones behind it), given what lies in front of lane 0.
  uint32_t equal_before = 0, hole_at = 0, mover_at = 0, total = 0;
  auto number = [&](const uint4& n4, int first, int end, int me) {
    uint32_t eq = n4.z + n4.w, inc = eq;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += y;
    }
    const uint32_t before = equal_before + inc - eq;
    const uint32_t stay = before >= left ? 0u : left - before < eq ? left - before : eq;
    const uint32_t stay_front = stay < n4.z ? stay : n4.z;
    const int front = (end < p.budget ? end : p.budget) - first;
    const uint32_t holes = (front > 0 ? (uint32_t)front : 0u) - n4.x - stay_front, movers = n4.y + stay - stay_front;
    total = __reduce_add_sync(0xffffffffu, movers);
    equal_before = __shfl_sync(0xffffffffu, before, me);
    hole_at += __reduce_add_sync(0xffffffffu, lane < me ? holes : 0u);
    mover_at += __reduce_add_sync(0xffffffffu, lane < me ? movers : 0u);
  };
  auto clip = [](int x, int most) { return x < most ? x : most; };
  {
    const int first = clip((lane < p.share ? lane : 0) * chunk, n);
    const uint4 of_block = lane < p.share ? *cluster.map_shared_rank(&s_sum, lane) : make_uint4(0, 0, 0, 0);
    number(of_block, lane < p.share ? first : 0, lane < p.share ? clip(first + chunk, n) : 0, rank);
  }
  const uint32_t moves = total;
  {
    const int first = clip(lo + (lane < kEvictWarps ? lane : 0) * part, hi);
    number(of_warp, lane < kEvictWarps ? first : 0, lane < kEvictWarps ? clip(first + part, hi) : 0, warp);
  }
  int32_t* const to = p.moves + (int64_t)item * 2 * p.room;
  int32_t* const of = to + p.room;
  for (int i0 = wlo; i0 < whi; i0 += 32) {
    const int i = i0 + lane;
    const bool in = i < whi;
    const uint32_t k = in ? key(i) : 0u, under = (1u << lane) - 1u;
    const uint32_t eq = __ballot_sync(0xffffffffu, in && k == prefix);
    const bool keep = in && (k > prefix || (k == prefix && equal_before + __popc(eq & under) < left));
    equal_before += __popc(eq);
    const bool hole = in && !keep && i < p.budget, mover = keep && i >= p.budget;
    const uint32_t bh = __ballot_sync(0xffffffffu, hole), bm = __ballot_sync(0xffffffffu, mover);
    if (hole) to[hole_at + __popc(bh & under)] = i;
    if (mover) of[mover_at + __popc(bm & under)] = i;
    hole_at += __popc(bh);
    mover_at += __popc(bm);
    if (in && i < p.budget && (copy_w || copy_p)) {
      if (i - lo < p.held) s_key[i - lo] = keep ? 1u : 0u;  // the key is needed no more
      else if (keep) carry(i);
    }
  }
  __threadfence();
  cluster.sync();  // the lists; and no block leaves while another reads its counts

  // A warp takes up to 32 moves: a lane finds a move's places and carries its
  // numbers, then the lanes copy the rows side by side, keys next to values,
  // kAtOnce of them in flight.
  const int row16 = c.D * (c.k_exp ? 1 : 2) / 16;  // 16-byte pieces of a row
  const int lanes = 2 * row16, per = 32 / lanes;   // of a move; moves of a warp-wide copy
  const int sub = lane / lanes, piece = lane % lanes;
  const bool val = piece >= row16;
  uint8_t* const rows = (val ? c.v : c.k) + (piece - (val ? row16 : 0)) * 16;
  const uint32_t warps = (uint32_t)(p.share * kEvictWarps);
  const uint32_t each = moves > 32 * warps ? 32u : (moves + warps - 1) / warps;
  for (uint32_t m0 = (uint32_t)(rank * kEvictWarps + warp) * each; m0 < moves; m0 += warps * each) {
    const uint32_t here = moves - m0 < each ? moves - m0 : each;
    int64_t rf = -1, rt = 0;
    if ((uint32_t)lane < here) {
      const Place f = place_of(c, of[m0 + lane]), t = place_of(c, to[m0 + lane]);
      const int pf = page_of(c, b, f.page), pt = page_of(c, b, t.page);
      if (pf >= 0 && pt >= 0) {
        rf = at(c.row, pf, f.slot, g);
        rt = at(c.row, pt, t.slot, g);
        const float w = p.weight_in[at(p.weight_at, pf, f.slot, g)];
        const int number = p.pos_in[at(p.pos_at, pf, f.slot, g)];
        if (c.k_exp) {
          const int64_t ef = at(c.exp, pf, f.slot, g), et = at(c.exp, pt, t.slot, g);
          const uint8_t ke = c.k_exp[ef], ve = c.v_exp[ef];
          c.k_exp[et] = ke;
          c.v_exp[et] = ve;
        }
        p.weight_out[at(p.weight_at, pt, t.slot, g)] = w;
        p.pos_out[at(p.pos_at, pt, t.slot, g)] = number;
      }
    }
    constexpr int kAtOnce = 4;
    for (uint32_t m = 0; m < here; m += kAtOnce * per) {
      uint4 x[kAtOnce];
      int64_t into[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const uint32_t k = m + u * per + sub;
        const int64_t from = __shfl_sync(0xffffffffu, rf, k & 31);
        into[u] = __shfl_sync(0xffffffffu, rt, k & 31);
        if (k >= here || from < 0) into[u] = -1;
        if (into[u] >= 0) x[u] = *reinterpret_cast<const uint4*>(rows + from);
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        if (into[u] >= 0) *reinterpret_cast<uint4*>(rows + into[u]) = x[u];
    }
  }
  if (copy_w || copy_p) {  // what stays, to the other arrays
    const int m = hi - lo < p.held ? hi - lo : p.held, end = p.budget - lo < m ? p.budget - lo : m;
    constexpr int kAtOnce = 4;
    for (int i0 = tid; i0 < end; i0 += kAtOnce * kEvictThreads) {
      int64_t a[kAtOnce], q[kAtOnce];
      float w[kAtOnce];
      int number[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int i = i0 + u * kEvictThreads;
        a[u] = -1;
        if (i < end && s_key[i]) {
          const Place x = place_of(c, lo + i);
          const int page = page_of(c, b, x.page);
          if (page >= 0) a[u] = at(p.weight_at, page, x.slot, g), q[u] = at(p.pos_at, page, x.slot, g);
        }
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        if (a[u] >= 0) w[u] = p.weight_in[a[u]], number[u] = p.pos_in[q[u]];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        if (a[u] >= 0) {
          if (copy_w) p.weight_out[a[u]] = w[u];
          if (copy_p) p.pos_out[q[u]] = number[u];
        }
    }
  }
}

cudaError_t launch_evict(EvictParams p, cudaStream_t st) {
  const int64_t items = (int64_t)p.c.B * p.c.Hkv;
  // blocks of an item: as many as leave two an SM, while each still has 1024 slots
  // (64 items of 25,331 slots: 4 blocks each 49 us, 8 in two waves 63), and as many
  // as it takes to hold the keys.  Both go by the table's width, the lengths being on
  // the device: from about 28,000 slots a block on the keys' shared memory leaves
  // one block an SM, and wide tables of short sequences take several waves (32 of
  // 2112 slots, 8 kv heads: a table for 2112 slots 19 us, for 131,072 58, for
  // 1,048,576 111)
  int share = 1;
  while (share < 8 && ((items * share <= num_sms() && p.c.capacity / share > 1024) || p.c.capacity / share > kEvictMaxHeld))
    share *= 2;
  int64_t held = (p.c.capacity + share - 1) / share;
  if (held > kEvictMaxHeld) held = kEvictMaxHeld;
  p.share = share;
  p.held = (int)held;
  if (items * share >= ((int64_t)1 << 31)) return cudaErrorInvalidConfiguration;
  const size_t smem = sizeof(uint32_t) * (size_t)held;
  static bool allowed[64] = {};
  cudaError_t e = allow_smem(evict_kernel, sizeof(uint32_t) * kEvictMaxHeld, allowed);
  if (e != cudaSuccess) return e;
  prof_before(THD_KERNEL_CACHE_EVICT, st);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)share;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * share));
  cfg.blockDim = dim3(kEvictThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, evict_kernel, p);
  count_launch();
  prof_after(THD_KERNEL_CACHE_EVICT, st);
  return e;
}

}  // namespace thd
