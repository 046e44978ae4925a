// The plain instantiations of the dQ kernel.
#include "dq.cuh"

namespace thd {

cudaError_t launch_dq(const DqParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int D, bool grouped, int grid,
                      cudaStream_t st) {
  if (D == 128) return grouped ? launch_dq_t<128, true, 0>(p, tk, tv, grid, st) : launch_dq_t<128, false, 0>(p, tk, tv, grid, st);
  return grouped ? launch_dq_t<64, true, 0>(p, tk, tv, grid, st) : launch_dq_t<64, false, 0>(p, tk, tv, grid, st);
}

}  // namespace thd
