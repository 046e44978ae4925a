// Rotary positions with several axes (time, height, width) on packed THD
// queries and keys, forward and backward, in one launch.
//
// Pair i of a head (elements i and i + rot/2, or 2i and 2i + 1) is turned by
//   angle_i = position[axis_i] * f_i
//   (a, b) -> (a cos - b sin, b cos + a sin)          backward: -angle
// and the elements past rot_dim are copied.
//
// The angle is reduced exactly, without floating point: the host gives f_i as
// F_i = f_i / (2 pi) in turns, a 64-bit binary fraction, and position * F_i
// modulo 2^64 is the fraction of a turn whatever the position (a 32-bit
// product would be off by position * 2^-33 turns; this one by position * 2^-55,
// the rounding of f_i itself).  Its top 32 bits, as a signed number of half
// turns, go to sincospif.
//
// What bounds it: HBM.  Every element is read and written once; a token's
// cosines and sines are computed once and shared by all of its heads (40 heads
// of 128 elements cost 64 sincos).  A block takes a few tokens with all their
// heads: first one thread per (token, pair) leaves cos and sin in shared
// memory, then a thread keeps one (token, 8 pairs) in registers and walks the
// heads, kRopeBatch heads' 16-byte loads in flight at once.
#include <cuda_bf16.h>

#include "common.cuh"
#include "rope.cuh"

namespace thd {

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 4;     // heads a thread has in flight
constexpr int kRopeMinTokens = 4;  // tokens per block, at least

// cos and sin of the angle of pair i at token t
__device__ inline float2 rope_cos_sin(const RopeParams& p, int64_t t, int i) {
  const int64_t pos = p.pos[(int64_t)p.axis[i] * p.T + t];
  const uint64_t frac = (uint64_t)pos * p.turn[i] + 0x80000000ull;  // rounded to 32 bits
  const float half_turns = (float)(int32_t)(frac >> 32) * 0x1p-31f;
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c, p.inverse ? -s : s);
}

// Eight consecutive elements.
__device__ inline void load8(const uint16_t* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = __uint_as_float(w[k] << 16);
    v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}
__device__ inline void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ inline void store8(uint16_t* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
    w[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ inline void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// 16-byte vectors: D a multiple of 8, rot of 16 (halves) or 8 (adjacent
// pairs), every row 16-byte aligned.  A unit is what one thread moves of a
// head: 8 pairs from two vectors (halves), 4 pairs from one (adjacent), or one
// vector past rot that is copied.
template <typename E, bool kAdjacent>
__global__ void __launch_bounds__(kRopeThreads) rope_vec_kernel(const __grid_constant__ RopeParams p, int units,
                                                                int slots, int tokens) {
  extern __shared__ float2 s_cs[];  // [tokens][rot / 2]
  const int half = p.rot / 2, tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  const int nt = (int)(p.T - t0 < tokens ? p.T - t0 : tokens);
  for (int i = tid; i < nt * half; i += kRopeThreads) {
    const int tl = i / half;
    s_cs[i] = rope_cos_sin(p, t0 + tl, i - tl * half);
  }
  __syncthreads();
  const int group = tid / units, u = tid - group * units;
  const int tl = group / slots, slot = group - tl * slots;  // `slots` heads of a token side by side
  if (tl >= nt) return;
  const int64_t t = t0 + tl;
  const int rot_units = kAdjacent ? p.rot / 8 : p.rot / 16;
  const bool rotates = u < rot_units;
  const int c0 = rotates ? 8 * u : p.rot + 8 * (u - rot_units);
  constexpr int kPairs = kAdjacent ? 4 : 8;
  float2 cs[kPairs];
  if (rotates) {
#pragma unroll
    for (int k = 0; k < kPairs; ++k) cs[k] = s_cs[tl * half + kPairs * u + k];
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const RopeTensor& x = p.x[w];
    const E* in = static_cast<const E*>(x.in) + t * x.in_stride + c0;
    E* out = static_cast<E*>(x.out) + t * x.out_stride + c0;
    for (int h0 = slot; h0 < x.H; h0 += slots * kRopeBatch) {
      float a[kRopeBatch][8], b[kRopeBatch][8];
#pragma unroll
      for (int k = 0; k < kRopeBatch; ++k) {
        const int h = h0 + k * slots;
        if (h < x.H) {
          load8(in + h * p.D, a[k]);
          if (!kAdjacent && rotates) load8(in + h * p.D + half, b[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < kRopeBatch; ++k) {
        const int h = h0 + k * slots;
        if (h >= x.H) break;
        if (rotates) {
          if constexpr (kAdjacent) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float r = a[k][2 * e], i = a[k][2 * e + 1];
              a[k][2 * e] = r * cs[e].x - i * cs[e].y;
              a[k][2 * e + 1] = i * cs[e].x + r * cs[e].y;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float r = a[k][e], i = b[k][e];
              a[k][e] = r * cs[e].x - i * cs[e].y;
              b[k][e] = i * cs[e].x + r * cs[e].y;
            }
            store8(out + h * p.D + half, b[k]);
          }
        }
        store8(out + h * p.D, a[k]);
      }
    }
  }
}

// Any head size, rotated size and alignment: one thread per pair (or copied
// element) of a token's heads, with the same cos and sin table.
__device__ inline float load1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ inline float load1(const float* p) { return *p; }
__device__ inline void store1(uint16_t* p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
__device__ inline void store1(float* p, float v) { *p = v; }

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
        const float a = load1(in + ia), b = load1(in + ib);
        store1(out + ia, a * cs.x - b * cs.y);
        store1(out + ib, b * cs.x + a * cs.y);
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
  const int heads = p.x[0].H > p.x[1].H ? p.x[0].H : p.x[1].H;
  const bool vec = p.D % 8 == 0 && p.rot % (kAdjacent ? 8 : 16) == 0 && vec_ok(p.x[0], sizeof(E)) &&
                   vec_ok(p.x[1], sizeof(E));
  prof_before(THD_KERNEL_ROPE, st);
  if (vec) {
    const int units = (kAdjacent ? p.rot / 8 : p.rot / 16) + (p.D - p.rot) / 8;
    const int groups = kRopeThreads / units;
    int slots = groups / kRopeMinTokens;
    slots = slots < 1 ? 1 : (slots > heads ? heads : slots);
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
