// The scored instantiations of the dK/dV kernel whose work items share key
// tiles (see bwd_parts).  Entry-major: with so few items the kv heads' order
// makes no difference to L2.
#include "bwd.cuh"

namespace thd {

template <int D>
static cudaError_t launch_d(const BwdParams& p, const CUtensorMap& tq, const CUtensorMap& tdo, const CUtensorMap& tk,
                            const CUtensorMap& tv, int mod, int grid, cudaStream_t st) {
  constexpr int kBase = kScored | kModParts;
  switch (mod) {
    case kScored: return launch_bwd_t<D, false, kBase>(p, tq, tdo, tk, tv, grid, st);
    case kScored | kModCap: return launch_bwd_t<D, false, kBase | kModCap>(p, tq, tdo, tk, tv, grid, st);
    case kScored | kModDist: return launch_bwd_t<D, false, kBase | kModDist>(p, tq, tdo, tk, tv, grid, st);
    default: return launch_bwd_t<D, false, kBase | kModCap | kModDist>(p, tq, tdo, tk, tv, grid, st);
  }
}

cudaError_t launch_score_bwd_parts(const BwdParams& p, const CUtensorMap& tq, const CUtensorMap& tdo,
                                   const CUtensorMap& tk, const CUtensorMap& tv, int D, int mod, int grid,
                                   cudaStream_t st) {
  return D == 128 ? launch_d<128>(p, tq, tdo, tk, tv, mod, grid, st) : launch_d<64>(p, tq, tdo, tk, tv, mod, grid, st);
}

}  // namespace thd
