// The scored instantiations of the dQ kernel: interval masks alone, and
// with the tanh cap, the distance bias, or both.
#include "dq.cuh"

namespace thd {

template <int D, bool kGrouped>
static cudaError_t launch_d(const DqParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int mod, int grid,
                            cudaStream_t st) {
  switch (mod) {
    case kScored: return launch_dq_t<D, kGrouped, kScored>(p, tk, tv, grid, st);
    case kScored | kModCap: return launch_dq_t<D, kGrouped, kScored | kModCap>(p, tk, tv, grid, st);
    case kScored | kModDist: return launch_dq_t<D, kGrouped, kScored | kModDist>(p, tk, tv, grid, st);
    default: return launch_dq_t<D, kGrouped, kScored | kModCap | kModDist>(p, tk, tv, grid, st);
  }
}

cudaError_t launch_score_dq(const DqParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int D,
                             bool grouped, int mod, int grid, cudaStream_t st) {
  if (D == 128)
    return grouped ? launch_d<128, true>(p, tk, tv, mod, grid, st) : launch_d<128, false>(p, tk, tv, mod, grid, st);
  return grouped ? launch_d<64, true>(p, tk, tv, mod, grid, st) : launch_d<64, false>(p, tk, tv, mod, grid, st);
}

}  // namespace thd
