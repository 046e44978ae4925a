// The plain instantiations of the dK/dV kernel.
#include "bwd.cuh"

namespace thd {

cudaError_t launch_bwd(const BwdParams& p, const CUtensorMap& tq, const CUtensorMap& tdo, const CUtensorMap& tk,
                       const CUtensorMap& tv, int D, bool grouped, int grid, cudaStream_t st) {
  if (D == 128)
    return grouped ? launch_bwd_t<128, true, 0>(p, tq, tdo, tk, tv, grid, st)
                   : launch_bwd_t<128, false, 0>(p, tq, tdo, tk, tv, grid, st);
  return grouped ? launch_bwd_t<64, true, 0>(p, tq, tdo, tk, tv, grid, st)
                 : launch_bwd_t<64, false, 0>(p, tq, tdo, tk, tv, grid, st);
}

}  // namespace thd
