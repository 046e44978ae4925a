// What fills a paged key-value cache and what keeps it small: thd_cache_append
// and thd_cache_evict (see the header).
#include <cooperative_groups.h>
#include <cuda_fp8.h>

#include "cache.cuh"
#ifndef MPDL
#define MPDL 0
#endif
#ifndef APDL
#define APDL 1
#endif
#include "vec8.cuh"

namespace thd {

// ------------------------------------------------------------------ append
// A block takes `tokens` rows; its first threads find each row's sequence (a
// binary search of the offsets) and slot, then all threads walk the rows of
// (token, head, k or v), eight elements a lane.  Bound by HBM: the rows are read
// and written once, 16 bytes a lane (8 written for e4m3).
//
// e4m3 with a power of two for each row and head: e is the smallest exponent
// with max |row| <= 448 * 2^e, so dividing is exact and the only rounding is the
// one to e4m3's grid; a row of bf16 products keeps all of the format's precision
// (a scale of max / 448 would round twice and gain nothing but the last half
// binade).
constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 8;  // at most, a block

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

template <bool kFp8>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
  __shared__ int s_page[kAppendTokens], s_slot[kAppendTokens], s_pos[kAppendTokens];
  follow();
  depend();
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
    int page = -1, slot = 0, pos = 0;
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
        const Place at_j = place_of(c, (int)j);
        page = page_of(c, b, at_j.page);
        if (page < 0) raise(p.status, THD_DEV_ERR_PAGE);
        slot = (int)at_j.slot;
        pos = (int)((p.seen ? (int64_t)p.seen[b] : n) - back);
      }
    }
    s_page[threadIdx.x] = page;
    s_slot[threadIdx.x] = slot;
    s_pos[threadIdx.x] = pos;
  }
  __syncthreads();
  const int lanes = c.D / 8;                       // of a row
  const int rows = count * c.Hkv * 2;              // (token, head, k or v)
  const int per = kAppendThreads / lanes, lane = threadIdx.x % lanes;
  const int steps = (rows + per - 1) / per;        // every lane walks alike: the exponent is a shuffle
  for (int i0 = 0; i0 < steps; i0 += 4) {
    Vec8<uint16_t> x[4];
    bool ok[4];
    int tok[4], g[4], kv[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = (i0 + u) * per + threadIdx.x / lanes;
      ok[u] = r < rows;
      kv[u] = r & 1;
      g[u] = (r >> 1) % c.Hkv;
      tok[u] = ok[u] ? (r >> 1) / c.Hkv : 0;
      ok[u] = ok[u] && s_page[tok[u]] >= 0;
      x[u].v = make_uint4(0, 0, 0, 0);
      if (ok[u]) x[u].load(p.in[kv[u]] + (t0 + tok[u]) * p.in_stride[kv[u]] + (int64_t)g[u] * c.D + 8 * lane);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      uint8_t* out = (kv[u] ? c.v : c.k);
      if (!kFp8) {
        if (ok[u]) x[u].store(reinterpret_cast<uint16_t*>(out + at(c.row, s_page[tok[u]], s_slot[tok[u]], g[u])) + 8 * lane);
      } else {
        const uint32_t w[4] = {x[u].v.x, x[u].v.y, x[u].v.z, x[u].v.w};
        uint32_t big = 0;  // of both halves: a bf16's order is its bits'
#pragma unroll
        for (int q = 0; q < 4; ++q) big = __vmaxu2(big, w[q] & 0x7fff7fffu);
        big = max(big >> 16, big & 0xffffu);
        for (int d = lanes / 2; d > 0; d >>= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, d));
        const int e = row_exponent(big);
        const float inv = __uint_as_float((uint32_t)(254 - e) << 23);  // 2^(127 - e)
        float f[8];
        x[u].get(f);
        uint32_t y[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * q] * inv, f[4 * q + 1] * inv), __NV_SATFINITE, __NV_E4M3);
          uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * q + 2] * inv, f[4 * q + 3] * inv), __NV_SATFINITE, __NV_E4M3);
          y[q] = e == 255 ? 0x7f7f7f7fu : lo | hi << 16;
        }
        if (ok[u]) {
          *reinterpret_cast<uint2*>(out + at(c.row, s_page[tok[u]], s_slot[tok[u]], g[u]) + 8 * lane) = make_uint2(y[0], y[1]);
          if (lane == 0) (kv[u] ? c.v_exp : c.k_exp)[at(c.exp, s_page[tok[u]], s_slot[tok[u]], g[u])] = (uint8_t)e;
        }
      }
      if (ok[u] && lane == 0 && kv[u] == 0) {
        if (p.weight) p.weight[at(p.weight_at, s_page[tok[u]], s_slot[tok[u]], g[u])] = 0.f;
        if (p.pos) p.pos[at(p.pos_at, s_page[tok[u]], s_slot[tok[u]], g[u])] = s_pos[tok[u]];
      }
    }
  }
}

cudaError_t launch_append(const AppendParams& a, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  AppendParams p = a;
  int64_t n = (a.T + 2 * num_sms() - 1) / (2 * num_sms());  // two blocks an SM first
  p.tokens = (int)(n > kAppendTokens ? kAppendTokens : n);
  const int64_t grid = (a.T + p.tokens - 1) / p.tokens;
  prof_before(THD_KERNEL_CACHE_APPEND, st);
  const cudaError_t e = launch_following(a.c.k_exp ? append_kernel<true> : append_kernel<false>, dim3((unsigned)grid),
                                         kAppendThreads, 0, st, APDL, (const AppendParams)p);
  prof_after(THD_KERNEL_CACHE_APPEND, st);
  return e;
}

// ------------------------------------------------------------------ evict
// One cluster of `share` blocks an item (sequence, kv head).  Every block holds
// its part of the slots' weights in shared memory as integers of the same
// order (protected slots on top), so they are read once; the budget-th largest
// is found by its digits (11, 11 and 10 bits, a histogram each, added up over
// the cluster through distributed shared memory), ties and the slots to move are
// numbered by ballots and counts, and the cluster's blocks then move rows.  Kept
// slots in front of the budget stay where they are and evicted ones there take
// the kept ones behind it, in order: the fewest bytes that can move, sources
// (behind) and targets (in front) that never meet, and nothing to wait for
// between them.
namespace cg = cooperative_groups;

constexpr int kEvictThreads = 256;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kBins = 2048;
constexpr int kEvictMaxHeld = 40960;  // keys in a block's shared memory (160 KB)

__device__ inline uint32_t order_of(float w, bool kept) {
  if (kept) return 0xff800000u;             // as +infinity
  if (!(w == w)) return 0u;                 // NaN: below everything
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 counts as 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const EvictParams p) {
  extern __shared__ uint32_t s_key[];  // [held]
  __shared__ uint32_t s_hist[kBins];
  __shared__ uint32_t s_scan[kEvictWarps], s_cnt[kEvictWarps][2];
  __shared__ uint32_t s_digit, s_left, s_sum[3];  // this block's equal slots, holes, movers
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
    if (page < 0) return;
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
    return order_of(p.weight_in[at(p.weight_at, page, x.slot, g)],
                    pos < p.sinks || (int64_t)pos >= (int64_t)seen - p.recent);
  };
  {
    const int m = hi - lo < p.held ? hi - lo : p.held;
#pragma unroll 4
    for (int i = tid; i < m; i += kEvictThreads) s_key[i] = read_key(lo + i);
  }
  auto key = [&](int i) { return i - lo < p.held ? s_key[i - lo] : read_key(i); };

  // the budget-th largest, digit by digit
  uint32_t prefix = 0, mask = 0, left = (uint32_t)p.budget;
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digits = pass == 2 ? 0x3ffu : 0x7ffu;
    for (int i = tid; i < kBins; i += kEvictThreads) s_hist[i] = 0;
    __syncthreads();
    for (int i0 = lo; i0 < hi; i0 += kEvictThreads) {
      const int i = i0 + tid;
      const uint32_t k = i < hi ? key(i) : 0u;
      const bool in = i < hi && (k & mask) == prefix;
      const uint32_t d = (k >> shift) & digits;
      // a warp of equals (protected slots, tokens nobody looked at) adds once
      const uint32_t act = __ballot_sync(0xffffffffu, in);
      if (act) {
        const uint32_t d0 = __shfl_sync(0xffffffffu, d, __ffs(act) - 1);
        if (__all_sync(0xffffffffu, !in || d == d0)) {
          if (lane == 0) atomicAdd(&s_hist[d0], (uint32_t)__popc(act));
        } else if (in) {
          atomicAdd(&s_hist[d], 1u);
        }
      }
    }
    cluster.sync();
    uint32_t mine[kBins / kEvictThreads], sum = 0;
    const int first = kBins - (tid + 1) * (kBins / kEvictThreads);  // thread 0 has the top bins
#pragma unroll
    for (int k = 0; k < kBins / kEvictThreads; ++k) mine[k] = 0;
    for (int r = 0; r < p.share; ++r) {
      const uint32_t* h = cluster.map_shared_rank(s_hist, r) + first;
#pragma unroll
      for (int k = 0; k < kBins / kEvictThreads; ++k) mine[k] += h[k];
    }
#pragma unroll
    for (int k = 0; k < kBins / kEvictThreads; ++k) sum += mine[k];
    uint32_t inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += y;
    }
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
    uint32_t above = inc - sum;
    for (int w = 0; w < warp; ++w) above += s_scan[w];
    if (above < left && left <= above + sum) {
      uint32_t rest = left - above;
      int k = kBins / kEvictThreads - 1;
      for (; k > 0 && rest > mine[k]; --k) rest -= mine[k];
      s_digit = (uint32_t)(first + k);
      s_left = rest;
    }
    cluster.sync();  // also: every block has read the histograms
    prefix |= s_digit << shift;
    mask |= digits << shift;
    left = s_left;
  }
  // kept: keys above `prefix`, and the first `left` slots equal to it
  const int part = ((hi - lo + kEvictWarps - 1) / kEvictWarps + 31) / 32 * 32;  // a warp's slots
  const int wlo = lo + warp * part < hi ? lo + warp * part : hi, whi = wlo + part < hi ? wlo + part : hi;
  // numbers the warp's slots: f(slot, kept) with the warp converged
  auto walk = [&](uint32_t equal_before, auto&& f) {
    for (int i0 = wlo; i0 < whi; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t k = i < whi ? key(i) : 0u;
      const bool eq = i < whi && k == prefix;
      const uint32_t bal = __ballot_sync(0xffffffffu, eq);
      const uint32_t before = equal_before + __popc(bal & ((1u << lane) - 1u));
      f(i, i < whi, i < whi && (k > prefix || (eq && before < left)));
      equal_before += __popc(bal);
    }
  };
  uint32_t equal = 0;
  for (int i = wlo + lane; i < whi; i += 32) equal += key(i) == prefix ? 1u : 0u;
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) s_scan[warp] = equal;
  __syncthreads();
  if (tid == 0) {
    uint32_t s = 0;
    for (int w = 0; w < kEvictWarps; ++w) s += s_scan[w];
    s_sum[0] = s;
  }
  cluster.sync();
  uint32_t equal_before = 0;
  for (int r = 0; r < rank; ++r) equal_before += *cluster.map_shared_rank(&s_sum[0], r);
  for (int w = 0; w < warp; ++w) equal_before += s_scan[w];
  uint32_t holes = 0, movers = 0;
  walk(equal_before, [&](int i, bool in, bool keep) {
    holes += __popc(__ballot_sync(0xffffffffu, in && !keep && i < p.budget));
    movers += __popc(__ballot_sync(0xffffffffu, keep && i >= p.budget));
  });
  if (lane == 0) s_cnt[warp][0] = holes, s_cnt[warp][1] = movers;
  __syncthreads();
  if (tid < 2) {
    uint32_t s = 0;
    for (int w = 0; w < kEvictWarps; ++w) s += s_cnt[w][tid];
    s_sum[1 + tid] = s;
  }
  cluster.sync();
  uint32_t hole_at = 0, mover_at = 0, total = 0;
  for (int r = 0; r < p.share; ++r) {
    const uint32_t* s = cluster.map_shared_rank(s_sum, r);
    if (r < rank) hole_at += s[1], mover_at += s[2];
    total += s[2];
  }
  for (int w = 0; w < warp; ++w) hole_at += s_cnt[w][0], mover_at += s_cnt[w][1];
  int32_t* const to = p.moves + (int64_t)item * 2 * p.room;
  int32_t* const of = to + p.room;
  walk(equal_before, [&](int i, bool in, bool keep) {
    const bool hole = in && !keep && i < p.budget, mover = keep && i >= p.budget;
    const uint32_t bh = __ballot_sync(0xffffffffu, hole), bm = __ballot_sync(0xffffffffu, mover);
    const uint32_t under = (1u << lane) - 1u;
    if (hole) to[hole_at + __popc(bh & under)] = i;
    if (mover) of[mover_at + __popc(bm & under)] = i;
    hole_at += __popc(bh);
    mover_at += __popc(bm);
    if (keep && i < p.budget && (copy_w || copy_p)) carry(i);
  });
  __threadfence();
  cluster.sync();  // the lists; and no block leaves while another reads its counts

  const int row16 = c.D * (c.k_exp ? 1 : 2) / 16;       // 16-byte pieces of a row
  const int lanes = 2 * row16, per = 32 / lanes;        // keys and values side by side in a warp
  const int sub = lane / lanes, piece = lane % lanes;
  const bool val = piece >= row16;
  uint8_t* const rows = (val ? c.v : c.k) + (piece - (val ? row16 : 0)) * 16;
  const uint32_t stride = (uint32_t)(p.share * kEvictWarps * per);
  for (uint32_t i0 = (uint32_t)((rank * kEvictWarps + warp) * per + sub); i0 < total; i0 += 4 * stride) {
    uint4 x[4];
    int pf[4], pt[4];
    uint32_t sf[4], st[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t i = i0 + u * stride;
      pf[u] = pt[u] = -1;
      if (i < total) {
        const Place f = place_of(c, of[i]), t = place_of(c, to[i]);
        pf[u] = page_of(c, b, f.page), sf[u] = f.slot;
        pt[u] = page_of(c, b, t.page), st[u] = t.slot;
        if (pt[u] < 0) pf[u] = -1;
      }
      if (pf[u] >= 0) x[u] = *reinterpret_cast<const uint4*>(rows + at(c.row, pf[u], sf[u], g));
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (pf[u] < 0) continue;
      *reinterpret_cast<uint4*>(rows + at(c.row, pt[u], st[u], g)) = x[u];
      if (piece == 0) {
        p.weight_out[at(p.weight_at, pt[u], st[u], g)] = p.weight_in[at(p.weight_at, pf[u], sf[u], g)];
        p.pos_out[at(p.pos_at, pt[u], st[u], g)] = p.pos_in[at(p.pos_at, pf[u], sf[u], g)];
        if (c.k_exp) {
          const int64_t f = at(c.exp, pf[u], sf[u], g), t = at(c.exp, pt[u], st[u], g);
          c.k_exp[t] = c.k_exp[f];
          c.v_exp[t] = c.v_exp[f];
        }
      }
    }
  }
}

cudaError_t launch_evict(EvictParams p, cudaStream_t st) {
  const int64_t items = (int64_t)p.c.B * p.c.Hkv;
  // blocks of an item: until the SMs have two each, while one still has 1024
  // slots, and as many as it takes to hold the keys
  int share = 1;
  while (share < 8 && ((items * share < 2LL * num_sms() && p.c.capacity / share > 1024) ||
                       p.c.capacity / share > kEvictMaxHeld))
    share *= 2;
  int64_t held = (p.c.capacity + share - 1) / share;
  if (held > kEvictMaxHeld) held = kEvictMaxHeld;
  p.share = share;
  p.held = (int)held;
  if (items * share >= ((int64_t)1 << 31)) return cudaErrorInvalidConfiguration;
  const size_t smem = sizeof(uint32_t) * (size_t)held;
  cudaError_t e = cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)(sizeof(uint32_t) * kEvictMaxHeld));
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
