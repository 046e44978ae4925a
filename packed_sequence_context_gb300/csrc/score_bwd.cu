// The scored instantiations of the dK/dV kernel: interval masks alone, and
// with the tanh cap, the distance bias, or both.
#include "bwd.cuh"

namespace thd {

template <int D, bool kGrouped>
static cudaError_t launch_d(const BwdParams& p, const CUtensorMap& tq, const CUtensorMap& tdo, const CUtensorMap& tk,
                             const CUtensorMap& tv, int mod, int grid,
                            cudaStream_t st) {
  switch (mod) {
    case kScored: return launch_bwd_t<D, kGrouped, kScored>(p, tq, tdo, tk, tv, grid, st);
    case kScored | kModCap: return launch_bwd_t<D, kGrouped, kScored | kModCap>(p, tq, tdo, tk, tv, grid, st);
    case kScored | kModDist: return launch_bwd_t<D, kGrouped, kScored | kModDist>(p, tq, tdo, tk, tv, grid, st);
    default: return launch_bwd_t<D, kGrouped, kScored | kModCap | kModDist>(p, tq, tdo, tk, tv, grid, st);
  }
}

cudaError_t launch_score_bwd(const BwdParams& p, const CUtensorMap& tq, const CUtensorMap& tdo, const CUtensorMap& tk,
                             const CUtensorMap& tv, int D,
                             bool grouped, int mod, int grid, cudaStream_t st) {
  if (D == 128)
    return grouped ? launch_d<128, true>(p, tq, tdo, tk, tv, mod, grid, st) : launch_d<128, false>(p, tq, tdo, tk, tv, mod, grid, st);
  return grouped ? launch_d<64, true>(p, tq, tdo, tk, tv, mod, grid, st) : launch_d<64, false>(p, tq, tdo, tk, tv, mod, grid, st);
}

}  // namespace thd
