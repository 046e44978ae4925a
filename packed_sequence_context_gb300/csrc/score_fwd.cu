// The scored instantiations of the forward kernel for long sequences: interval masks alone, and
// with the tanh cap, the distance bias, or both.
#include "fwd.cuh"

namespace thd {

template <int D>
static cudaError_t launch_d(const FwdParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int mod, int grid,
                            cudaStream_t st) {
  switch (mod) {
    case kScored: return launch_fwd_t<D, false, true, kScored>(p, tk, tv, grid, st);
    case kScored | kModCap: return launch_fwd_t<D, false, true, kScored | kModCap>(p, tk, tv, grid, st);
    case kScored | kModCap | kModBounded:
      return launch_fwd_t<D, false, true, kScored | kModCap | kModBounded>(p, tk, tv, grid, st);
    case kScored | kModDist: return launch_fwd_t<D, false, true, kScored | kModDist>(p, tk, tv, grid, st);
    case kScored | kModCap | kModDist | kModBounded:
      return launch_fwd_t<D, false, true, kScored | kModCap | kModDist | kModBounded>(p, tk, tv, grid, st);
    default: return launch_fwd_t<D, false, true, kScored | kModCap | kModDist>(p, tk, tv, grid, st);
  }
}

cudaError_t launch_score_fwd(const FwdParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int D, int mod,
                             int grid, cudaStream_t st) {
  return D == 128 ? launch_d<128>(p, tk, tv, mod, grid, st) : launch_d<64>(p, tk, tv, mod, grid, st);
}

}  // namespace thd
