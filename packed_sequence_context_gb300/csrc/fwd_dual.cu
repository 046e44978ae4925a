// The plain instantiations of the forward kernel with two items in flight.
#include "fwd_dual.cuh"

namespace thd {

cudaError_t launch_fwd_dual(const FwdParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int D, bool step_mode,
                            int grid, cudaStream_t st) {
  if (D == 128) return step_mode ? launch_fwd_dual_t<128, true, 0>(p, tk, tv, grid, st)
                                 : launch_fwd_dual_t<128, false, 0>(p, tk, tv, grid, st);
  return step_mode ? launch_fwd_dual_t<64, true, 0>(p, tk, tv, grid, st) : launch_fwd_dual_t<64, false, 0>(p, tk, tv, grid, st);
}

}  // namespace thd
