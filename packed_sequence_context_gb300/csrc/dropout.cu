// Dropout from a counter-based generator, plus the residual, on packed rows
// (see thd_dropout_add in the header): out = residual + keep(row, column) *
// x / (1 - p).  The mask is a function of (seed, offset, row number, column):
// it is computed where it is used, forward and backward, and never stored, and
// a rank's shard draws what the unsplit tensor draws for the same rows.
//
// Generator: Philox 4x32 with ten rounds (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC 2011).  One call gives
// eight columns of a row 16 bits each: counter (column / 8, row, offset),
// key = seed; column 8 g + 2 w + h takes half h of word w.  Sixteen bits set
// the drop probability in steps of 2^-16 (the scale goes by the rounded
// probability, so the mean is exact) at half the generator's work of 32.
//
// What bounds it: HBM, where the rows take 16-byte accesses.  Measured on one
// GB300, inputs larger than L2, of the rate of a plain copy: 41,888 x 4,096 bf16
// with a residual 153 us (99%), without one (2/3 of the bytes to as much of the
// generator) 119 us (85%), fp32 with one 292 us (104%); rows of 1,111 columns,
// off every alignment, fp32 91% and bf16 with a residual 67% (its elements move one
// to a lane, 64 bytes a warp's access).
#include "common.cuh"
#include "dropout.cuh"
#include "vec8.cuh"

namespace thd {

constexpr int kDropThreads = 256;
constexpr int kDropBatch = 4;  // groups of eight columns a thread has in flight

// The four words of columns 8 g .. 8 g + 7 of a row.
__device__ inline uint4 draw(uint32_t g, uint32_t row, uint64_t offset, uint64_t seed) {
  uint32_t c0 = g, c1 = row, c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// Bit e of the result: column 8 g + e is kept (16 bits at least `drop`; the
// comparisons are of the words against drop << 16, the low halves shifted up).
__device__ inline uint32_t keep_mask(const uint4& v, uint32_t drop16) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    m |= (w[k] << 16 >= drop16 ? 1u : 0u) << (2 * k);
    m |= (w[k] >= drop16 ? 1u : 0u) << (2 * k + 1);
  }
  return m;
}

// C a multiple of 8 and 16-byte aligned tensors: a thread moves groups of
// eight columns with 16-byte accesses, kDropBatch of them in flight while it
// draws their bits.
template <typename E, bool kResidual>
__global__ void __launch_bounds__(kDropThreads) dropout_vec_kernel(const DropoutParams p) {
  const int64_t total = p.T * (int64_t)p.G;
  const int64_t base = (int64_t)blockIdx.x * (kDropThreads * kDropBatch) + threadIdx.x;
  Vec8<E> x[kDropBatch], r[kDropBatch];
#pragma unroll
  for (int k = 0; k < kDropBatch; ++k) {
    const int64_t i = base + k * kDropThreads;
    if (i < total) {
      x[k].load(static_cast<const E*>(p.x) + 8 * i);
      if (kResidual) r[k].load(static_cast<const E*>(p.residual) + 8 * i);
    }
  }
  const uint64_t seed = p.rng[0], offset = p.rng[1];
  const uint32_t drop16 = p.drop << 16;
  int64_t row = base / p.G;
  uint32_t g = (uint32_t)(base - row * p.G);
#pragma unroll
  for (int k = 0; k < kDropBatch; ++k) {
    const int64_t i = base + k * kDropThreads;
    if (i < total) {
      const uint4 w4 = draw(g, p.row_ids ? (uint32_t)p.row_ids[row] : (uint32_t)row, offset, seed);
      const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
      float f[8], h[8];
      x[k].get(f);
      if (kResidual) r[k].get(h);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool keep = (e & 1 ? w[e / 2] : w[e / 2] << 16) >= drop16;  // the half against drop
        f[e] = keep ? f[e] * p.scale : 0.f;
        if (kResidual) f[e] += h[e];
      }
      x[k].set(f);
      x[k].store(static_cast<E*>(p.out) + 8 * i);
    }
    row += p.step_rows;  // kDropThreads groups on
    g += p.step_groups;
    if (g >= p.G) {
      g -= p.G;
      ++row;
    }
  }
}

// Any C and alignment: a warp takes a row, 256 columns at a time (short rows
// few enough to leave the GPU idle are shared by several); each lane draws the
// mask of one group of eight, and the elements move one to a lane (coalesced
// whatever the row's alignment), their mask byte fetched from the lane that
// drew it.
template <typename E, bool kResidual>
__global__ void __launch_bounds__(kDropThreads) dropout_any_kernel(const DropoutParams p) {
  const uint64_t seed = p.rng[0], offset = p.rng[1];
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * (kDropThreads / 32) + (threadIdx.x >> 5);
  if (row >= p.T) return;  // the whole warp
  const uint32_t id = p.row_ids ? (uint32_t)p.row_ids[row] : (uint32_t)row;
  for (int64_t c0 = (int64_t)blockIdx.y * 256; c0 < p.C; c0 += (int64_t)gridDim.y * 256) {
    const int64_t at = row * p.C + c0;
    const int n = (int)(p.C - c0 < 256 ? p.C - c0 : 256);
    E x[8], r[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (32 * k + lane < n) {
        x[k] = static_cast<const E*>(p.x)[at + 32 * k + lane];
        if (kResidual) r[k] = static_cast<const E*>(p.residual)[at + 32 * k + lane];
      }
    }
    const uint32_t mine = keep_mask(draw((uint32_t)(c0 / 8) + lane, id, offset, seed), p.drop << 16);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t m = __shfl_sync(0xffffffffu, mine, 4 * k + (lane >> 3));
      if (32 * k + lane < n) {
        float f = (m >> (lane & 7)) & 1u ? to_f32(x[k]) * p.scale : 0.f;
        if (kResidual) f += to_f32(r[k]);
        put(static_cast<E*>(p.out) + at + 32 * k + lane, f);
      }
    }
  }
}

template <typename E, bool kResidual>
static cudaError_t launch_dropout_t(DropoutParams p, cudaStream_t st) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.out) |
                      reinterpret_cast<uintptr_t>(p.residual);
  const bool vec = p.C % 8 == 0 && (a & 15u) == 0;
  if (vec) {
    p.G = (uint32_t)(p.C / 8);
    p.step_rows = kDropThreads / p.G;
    p.step_groups = kDropThreads % p.G;
  }
  const int64_t per_block = kDropThreads * kDropBatch, vec_grid = vec ? (p.T * (int64_t)p.G + per_block - 1) / per_block : 0;
  if (vec_grid >= ((int64_t)1 << 31)) return cudaErrorInvalidConfiguration;  // 2^42 elements and more
  prof_before(THD_KERNEL_DROPOUT, st);
  if (vec) {
    dropout_vec_kernel<E, kResidual><<<(unsigned)vec_grid, kDropThreads, 0, st>>>(p);
  } else {
    // enough warps for 64 on every SM, if the columns give them
    const int64_t runs = (p.C + 255) / 256;
    int64_t y = (64LL * num_sms() + p.T - 1) / p.T;
    y = y > runs ? runs : y;
    y = y > 65535 ? 65535 : y;
    const dim3 grid((unsigned)((p.T + kDropThreads / 32 - 1) / (kDropThreads / 32)), (unsigned)y);
    dropout_any_kernel<E, kResidual><<<grid, kDropThreads, 0, st>>>(p);
  }
  count_launch();
  cudaError_t e = cudaGetLastError();
  prof_after(THD_KERNEL_DROPOUT, st);
  return e;
}

cudaError_t launch_dropout(const DropoutParams& p, int dtype, cudaStream_t st) {
  if (p.T == 0 || p.C == 0) return cudaSuccess;
  if (dtype == THD_DTYPE_BF16)
    return p.residual ? launch_dropout_t<uint16_t, true>(p, st) : launch_dropout_t<uint16_t, false>(p, st);
  return p.residual ? launch_dropout_t<float, true>(p, st) : launch_dropout_t<float, false>(p, st);
}

}  // namespace thd
