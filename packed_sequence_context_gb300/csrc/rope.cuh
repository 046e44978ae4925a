// Rotary positions with several axes on packed THD rows (see thd_rope in the
// header): the parameters the host hands to the kernels of rope.cu.
#pragma once

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

cudaError_t launch_rope(const RopeParams& p, int dtype, bool adjacent, cudaStream_t st);

}  // namespace thd
