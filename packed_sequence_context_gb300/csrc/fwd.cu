// The plain instantiations of the forward kernel for long sequences.
#include "fwd.cuh"

namespace thd {

template <int D>
static cudaError_t launch_fwd_d(const FwdParams& p, const CUtensorMap& tk, const CUtensorMap& tv, bool step_mode,
                                bool dyn, int grid, cudaStream_t st) {
  if (step_mode)
    return dyn ? launch_fwd_t<D, true, true, 0>(p, tk, tv, grid, st) : launch_fwd_t<D, true, false, 0>(p, tk, tv, grid, st);
  return dyn ? launch_fwd_t<D, false, true, 0>(p, tk, tv, grid, st) : launch_fwd_t<D, false, false, 0>(p, tk, tv, grid, st);
}

cudaError_t launch_fwd(const FwdParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int D, bool step_mode,
                       bool dyn, int grid, cudaStream_t st) {
  return D == 128 ? launch_fwd_d<128>(p, tk, tv, step_mode, dyn, grid, st)
                  : launch_fwd_d<64>(p, tk, tv, step_mode, dyn, grid, st);
}

}  // namespace thd
