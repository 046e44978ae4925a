// Eight consecutive elements of a row as they are loaded and stored (16-byte
// pieces), and single elements; bf16 (uint16_t) and fp32.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

namespace thd {

template <typename E>
struct Vec8;
template <>
struct Vec8<uint16_t> {
  uint4 v;
  __device__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ void store(uint16_t* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(w[k] << 16);
      f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
  __device__ void set(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  __device__ void set(const float (&f)[8]) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
};

__device__ inline float to_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ inline float to_f32(float v) { return v; }
__device__ inline void put(uint16_t* p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
__device__ inline void put(float* p, float v) { *p = v; }

}  // namespace thd
