// Rotary positions with several axes (time, height, width) on packed THD
// queries and keys, forward and backward, in one launch.
//
// Pair i of a head (elements i and i + rot/2, or 2i and 2i + 1) is turned by
//   angle_i = position[axis_i] * f_i
//   (a, b) -> (a cos - b sin, b cos + a sin)          backward: -angle
// and the elements past rot_dim are copied.
//
// The angle is reduced exactly, without floating point: the host gives f_i as
// F_i = f_i / (2 pi) in turns, a 64-bit binary fraction (rope_turn), and
// position * F_i modulo 2^64 is the fraction of a turn whatever the position (a
// 32-bit product would be off by position * 2^-33 turns; this one by
// position * 2^-64).  Its quarter turns are taken off as integers too, and what
// is left, at most 1/8 turn either way, goes to sincospif: 24 bits of it round
// the angle by 2^-27 turns, of the whole fraction they would by 2^-25.
//
// What bounds it: HBM.  Every element is read and written once; a token's
// cosines and sines are computed once and shared by all of its heads (40 heads
// of 128 elements cost 64 sincos).  A block takes a few tokens with all their
// heads: a thread keeps one (token, 8 pairs) and walks the heads, the loads of
// its first ones in flight while one thread per (token, pair) leaves cos and
// sin in shared memory.  Measured on one GB300, inputs larger than L2: 131,072
// tokens of 32 + 8 heads of 128, bf16, 394 us (6816 GB/s, the rate of a plain
// copy); with the loads after the angles, and both as floats (122 registers, two
// blocks per SM instead of three), 675 us.
#include "common.cuh"
#include "rope.cuh"
#include "vec8.cuh"

namespace thd {

constexpr int kRopeThreads = 256;
constexpr int kRopeMinTokens = 4;  // tokens per block, at least
constexpr int kRopeHeads = 4;      // heads a thread walks, at least, where a token has as many

// cos and sin of the angle of pair i at token t
__device__ inline float2 rope_cos_sin(const RopeParams& p, int64_t t, int i) {
  const int64_t pos = p.pos[(int64_t)p.axis[i] * p.T + t];
  const uint64_t frac = (uint64_t)pos * p.turn[i];
  const uint32_t quarters = (uint32_t)((frac + (1ull << 61)) >> 62);  // the nearest, mod 4
  const float half_turns = (float)(int64_t)(frac - ((uint64_t)quarters << 62)) * 0x1p-63f;  // within +-1/4 of it
  float s, c;
  sincospif(half_turns, &s, &c);
  const float x = quarters & 1 ? -s : c, y = quarters & 1 ? c : s;
  const float cs = quarters & 2 ? -x : x, sn = quarters & 2 ? -y : y;
  return make_float2(cs, p.inverse ? -sn : sn);
}

// 16-byte vectors: D a multiple of 8, rot of 16 (halves) or 8 (adjacent
// pairs), every row 16-byte aligned.  A unit is what one thread moves of a
// head: 8 pairs from two vectors (halves), 4 pairs from one (adjacent), or one
// vector past rot that is copied.  Query and key heads are one list.
template <typename E, bool kAdjacent>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_vec_kernel(const __grid_constant__ RopeParams p, int units,
                                                                   int slots, int tokens) {
  extern __shared__ float2 s_cs[];  // [tokens][rot / 2]
  const int half = p.rot / 2, tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  const int nt = (int)(p.T - t0 < tokens ? p.T - t0 : tokens);
  const int group = tid / units, u = tid - group * units;
  const int tl = group / slots, slot = group - tl * slots;  // `slots` heads of a token side by side
  const bool works = tl < nt;
  const int64_t t = t0 + (works ? tl : 0);
  const int rot_units = kAdjacent ? p.rot / 8 : p.rot / 16;
  const bool rotates = u < rot_units;
  const int c0 = rotates ? 8 * u : p.rot + 8 * (u - rot_units);
  const int heads = works ? p.x[0].H + p.x[1].H : 0;
  const E* in[2];
  E* out[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {  // key heads follow the queries'
    const int64_t first = w == 0 ? 0 : -(int64_t)p.x[0].H * p.D;
    in[w] = static_cast<const E*>(p.x[w].in) + t * p.x[w].in_stride + first + c0;
    out[w] = static_cast<E*>(p.x[w].out) + t * p.x[w].out_stride + first + c0;
  }
  constexpr int kBatch = sizeof(E) == 2 ? 4 : 2;  // heads in flight: 32 registers of loads
  Vec8<E> a[kBatch], b[kBatch];
  auto load = [&](int h0) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = h0 + k * slots;
      if (h < heads) {
        const E* src = (h < p.x[0].H ? in[0] : in[1]) + (int64_t)h * p.D;
        a[k].load(src);
        if (!kAdjacent && rotates) b[k].load(src + half);
      }
    }
  };
  load(slot);  // in flight while the angles are made
  for (int i = tid; i < nt * half; i += kRopeThreads) {
    const int il = i / half;
    s_cs[i] = rope_cos_sin(p, t0 + il, i - il * half);
  }
  __syncthreads();
  constexpr int kPairs = kAdjacent ? 4 : 8;
  float2 cs[kPairs];
#pragma unroll
  for (int k = 0; k < kPairs; ++k) cs[k] = rotates && works ? s_cs[tl * half + kPairs * u + k] : make_float2(1.f, 0.f);
  for (int h0 = slot; h0 < heads; h0 += slots * kBatch) {
    if (h0 != slot) load(h0);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = h0 + k * slots;
      if (h >= heads) break;
      E* dst = (h < p.x[0].H ? out[0] : out[1]) + (int64_t)h * p.D;
      if (rotates) {
        float x[8], y[8];
        a[k].get(x);
        if constexpr (kAdjacent) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float r = x[2 * e], i = x[2 * e + 1];
            x[2 * e] = r * cs[e].x - i * cs[e].y;
            x[2 * e + 1] = i * cs[e].x + r * cs[e].y;
          }
        } else {
          b[k].get(y);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float r = x[e], i = y[e];
            x[e] = r * cs[e].x - i * cs[e].y;
            y[e] = i * cs[e].x + r * cs[e].y;
          }
          b[k].set(y);
          b[k].store(dst + half);
        }
        a[k].set(x);
      }
      a[k].store(dst);
    }
  }
}

// Any head size, rotated size and alignment: one thread per pair (or copied
// element) of a token's heads, with the same cos and sin table.  One element an
// access and a division for each pair bound it: 65,536 tokens of 32 + 8 heads, of
// the rate of a plain copy: heads of 128 one element off the grid bf16 43%
// (465 us), fp32 72%; of 80 elements, 40 of them rotated, 27% and 46%.
template <typename E, bool kAdjacent>
__global__ void __launch_bounds__(kRopeThreads) rope_scalar_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float2 s_cs[kRopeMinTokens * kRopeMaxPairs];
  const int half = p.rot / 2, rest = p.D - p.rot, per_head = half + rest;
  const int64_t t0 = (int64_t)blockIdx.x * kRopeMinTokens;
  const int nt = (int)(p.T - t0 < kRopeMinTokens ? p.T - t0 : kRopeMinTokens);
  for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
    const int tl = i / half;
    s_cs[i] = rope_cos_sin(p, t0 + tl, i - tl * half);
  }
  __syncthreads();
  for (int w = 0; w < 2; ++w) {
    const RopeTensor& x = p.x[w];
    for (int tl = 0; tl < nt; ++tl) {
      const E* in = static_cast<const E*>(x.in) + (t0 + tl) * x.in_stride;
      E* out = static_cast<E*>(x.out) + (t0 + tl) * x.out_stride;
      const int n = x.H * per_head;
      for (int i = threadIdx.x; i < n; i += kRopeThreads) {
        const int h = i / per_head, j = i - h * per_head;
        const int64_t base = (int64_t)h * p.D;
        if (j >= half) {  // past rot_dim: copied
          out[base + p.rot + j - half] = in[base + p.rot + j - half];
          continue;
        }
        const int64_t ia = base + (kAdjacent ? 2 * j : j), ib = base + (kAdjacent ? 2 * j + 1 : j + half);
        const float2 cs = s_cs[tl * half + j];
        const float a = to_f32(in[ia]), b = to_f32(in[ib]);
        put(out + ia, a * cs.x - b * cs.y);
        put(out + ib, b * cs.x + a * cs.y);
      }
    }
  }
}

static bool vec_ok(const RopeTensor& x, int esize) {
  if (x.H == 0) return true;
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.in) | reinterpret_cast<uintptr_t>(x.out);
  return (a & 15u) == 0 && (x.in_stride * esize) % 16 == 0 && (x.out_stride * esize) % 16 == 0;
}

template <typename E, bool kAdjacent>
static cudaError_t launch_rope_t(const RopeParams& p, cudaStream_t st) {
  const int heads = p.x[0].H + p.x[1].H;
  const bool vec = p.D % 8 == 0 && p.rot % (kAdjacent ? 8 : 16) == 0 && vec_ok(p.x[0], sizeof(E)) &&
                   vec_ok(p.x[1], sizeof(E));
  prof_before(THD_KERNEL_ROPE, st);
  if (vec) {
    const int units = (kAdjacent ? p.rot / 8 : p.rot / 16) + (p.D - p.rot) / 8;
    const int groups = kRopeThreads / units;
    int slots = groups / kRopeMinTokens;
    if (slots > (heads + kRopeHeads - 1) / kRopeHeads) slots = (heads + kRopeHeads - 1) / kRopeHeads;
    if (slots < 1) slots = 1;
    const int tokens = groups / slots;
    const size_t smem = sizeof(float2) * (size_t)tokens * (p.rot / 2);
    rope_vec_kernel<E, kAdjacent><<<(unsigned)((p.T + tokens - 1) / tokens), kRopeThreads, smem, st>>>(
        p, units, slots, tokens);
  } else {
    rope_scalar_kernel<E, kAdjacent>
        <<<(unsigned)((p.T + kRopeMinTokens - 1) / kRopeMinTokens), kRopeThreads, 0, st>>>(p);
  }
  count_launch();
  cudaError_t e = cudaGetLastError();
  prof_after(THD_KERNEL_ROPE, st);
  return e;
}

cudaError_t launch_rope(const RopeParams& p, int dtype, bool adjacent, cudaStream_t st) {
  if (p.T == 0 || p.x[0].H + p.x[1].H == 0) return cudaSuccess;
  if (dtype == THD_DTYPE_BF16)
    return adjacent ? launch_rope_t<uint16_t, true>(p, st) : launch_rope_t<uint16_t, false>(p, st);
  return adjacent ? launch_rope_t<float, true>(p, st) : launch_rope_t<float, false>(p, st);
}

}  // namespace thd
