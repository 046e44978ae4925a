// Rotary positions with several axes on packed THD rows (see thd_rope in the
// header): the parameters the host hands to the kernels of rope.cu.
#pragma once

#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

namespace thd {

constexpr int kRopeMaxPairs = 128;  // rot_dim / 2
constexpr int kRopeMaxAxes = 16;

struct RopeTensor {
  const void* in;
  void* out;
  int64_t in_stride, out_stride;  // elements between tokens
  int H;
};

struct RopeParams {
  RopeTensor x[2];  // queries, keys (H = 0: none)
  const int32_t* pos;  // [n_axes][T]
  int64_t T;
  int D, rot, n_axes;
  int inverse;
  // turns per position of each pair, as a 64-bit binary fraction
  uint64_t turn[kRopeMaxPairs];
  uint8_t axis[kRopeMaxPairs];
};

// f / (2 pi) modulo 1 as a 64-bit binary fraction, rounded: right to 2^-64 for |f|
// up to 2^40, so that position * fraction is right to 2^-33 turns at any 32-bit
// position.  One product with 1 / (2 pi) in a double would be off by |f| 2^-55, 2
// thousandths of a turn at f = 1000 and a far position; here 1 / (2 pi) has two
// parts and the product its low part.
inline uint64_t rope_turn(double f) {
  const double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  const double a = std::fabs(f);
  volatile double product = a * hi;  // rounded here, not fused into what follows
  const double p = product;
  double e = std::fma(a, hi, -p) + a * lo;
  e -= std::rint(e);  // whole turns drop out at whole positions
  const double s = (p - std::floor(p)) * 0x1p64, whole = std::floor(s);  // both exact, s < 2^64
  const double rest = (s - whole) + e * 0x1p64;                        // |rest| <= 2^63 + 1
  const uint64_t r = (uint64_t)std::rint(std::fabs(rest));
  const uint64_t turn = (uint64_t)whole + (rest < 0 ? 0 - r : r);
  return f < 0 ? 0 - turn : turn;
}

cudaError_t launch_rope(const RopeParams& p, int dtype, bool adjacent, cudaStream_t st);

}  // namespace thd
