// The scored instantiations of the forward kernel with two items in flight: interval masks alone, and
// with the tanh cap, the distance bias, or both.
#include "fwd_dual.cuh"

namespace thd {

template <int D>
static cudaError_t launch_d(const FwdParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int mod, int grid,
                            cudaStream_t st) {
  switch (mod) {
    case kScored: return launch_fwd_dual_t<D, false, kScored>(p, tk, tv, grid, st);
    case kScored | kModCap: return launch_fwd_dual_t<D, false, kScored | kModCap>(p, tk, tv, grid, st);
    case kScored | kModCap | kModBounded:
      return launch_fwd_dual_t<D, false, kScored | kModCap | kModBounded>(p, tk, tv, grid, st);
    case kScored | kModDist: return launch_fwd_dual_t<D, false, kScored | kModDist>(p, tk, tv, grid, st);
    case kScored | kModCap | kModDist | kModBounded:
      return launch_fwd_dual_t<D, false, kScored | kModCap | kModDist | kModBounded>(p, tk, tv, grid, st);
    default: return launch_fwd_dual_t<D, false, kScored | kModCap | kModDist>(p, tk, tv, grid, st);
  }
}

cudaError_t launch_score_fwd_dual(const FwdParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int D, int mod,
                                  int grid, cudaStream_t st) {
  return D == 128 ? launch_d<128>(p, tk, tv, mod, grid, st) : launch_d<64>(p, tk, tv, mod, grid, st);
}

}  // namespace thd
