// Dropout plus residual (see thd_dropout_add in the header): the parameters
// the host hands to the kernels of dropout.cu.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace thd {

struct DropoutParams {
  const void* x;
  const void* residual;  // may be null
  void* out;
  const int32_t* row_ids;  // may be null: the row's index
  const uint64_t* rng;     // device: seed, offset
  int64_t T, C;
  uint32_t drop;  // drop where the 16 random bits are below this
  float scale;    // 65536 / (65536 - drop)
  uint32_t G, step_rows, step_groups;  // vector path: C / 8; kDropThreads groups on, in rows and groups
};

cudaError_t launch_dropout(const DropoutParams& p, int dtype, cudaStream_t st);

}  // namespace thd
