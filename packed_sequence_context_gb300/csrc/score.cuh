// The score function of scored attention, for one thread's run of scores.
//
//   x = softmax_scale * s                       (s = q . k, fp32 in TMEM)
//   y = softcap tanh(x / softcap)   or  x
//   y -= slope |i' - j|                         (i' = i + koff: the key position a query sits at)
// in log2 units (y log2(e)), as the softmax takes them.
//
// tanh u = 1 - 2 r, r = 1 / (1 + e^(2u)): one 2^x and one reciprocal, exact to
// fp32 rounding in absolute terms (softcap 2^-22; the hardware's one-step tanh
// is off by 2^-11, 0.02 at a cap of 50).  Two scores share a reciprocal:
// 1/a = b / (ab), 1/b = a / (ab), with the exponents held to 2^60 so that ab
// stays finite (tanh is 1 to the last bit long before).  The derivative is
// 1 - tanh^2 = 4 r (1 - r).
//
// The bias is linear in j on either side of i', so a row that sees only keys
// up to its own position (every causal row without a prefix) takes one fused
// multiply-add for it; other rows take the absolute value.
#pragma once

#include "common.cuh"
#include "ptx.cuh"

namespace thd {

THD_DEV float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// r = 1 / (1 + 2^(c s)) of two scores
THD_DEV void cap_pair(float& r0, float& r1, float s0, float s1, float c) {
  float x0, x1, a0, a1;
  fmul2(x0, x1, s0, s1, c, c);
  fadd2(a0, a1, ex2(fminf(x0, 60.f)), ex2(fminf(x1, 60.f)), 1.f, 1.f);
  const float q = rcp(a0 * a1);
  fmul2(r0, r1, q, q, a1, a0);
}

struct ScoreConsts {
  float sl2;    // softmax_scale log2(e)
  float cap_a;  // softcap log2(e)
  float cap_c;
  float slope;  // the head's slope log2(e)
};
template <int kMod, class P>
THD_DEV ScoreConsts score_consts(const P& p, int h) {
  ScoreConsts k;
  k.sl2 = p.scale_log2;
  k.cap_a = p.mods.cap_a;
  k.cap_c = p.mods.cap_c;
  k.slope = 0.f;
  if constexpr ((kMod & kModDist) != 0) k.slope = p.mods.slopes[h] * 1.4426950408889634f;
  return k;
}

// One thread's N scores (N even), in place: s[n] becomes y log2(e).  d0 = i' - j
// of the first one and dir = -1 (the scores run along j) or +1 (along i'), so
// score n sits at distance |d0 + dir n|; `abs_needed` (uniform over the warp):
// some visible score has i' < j.  With kGrad, w[n] = 1 - tanh^2.
template <int kMod, bool kGrad, int N, int kDir>
THD_DEV void score_run(float (&s)[N], float* w, const ScoreConsts& k, float d0, bool abs_needed) {
  constexpr bool kCap = (kMod & kModCap) != 0, kDist = (kMod & kModDist) != 0;
  const float base = kDist ? -k.slope * d0 : 0.f;   // bias of score 0, linear side
  const float step = kDist ? -k.slope * kDir : 0.f;  // and what each score adds
  if (kDist && abs_needed) {
#pragma unroll
    for (int n = 0; n < N; n += 2) {
      float b0 = -k.slope * fabsf(d0 + kDir * n), b1 = -k.slope * fabsf(d0 + kDir * (n + 1));
      if constexpr (kCap) {
        float r0, r1;
        cap_pair(r0, r1, s[n], s[n + 1], k.cap_c);
        if constexpr (kGrad) {
          w[n] = 4.f * r0 * (1.f - r0);
          w[n + 1] = 4.f * r1 * (1.f - r1);
        }
        ffma2(s[n], s[n + 1], r0, r1, -2.f * k.cap_a, -2.f * k.cap_a, b0 + k.cap_a, b1 + k.cap_a);
      } else {
        ffma2(s[n], s[n + 1], s[n], s[n + 1], k.sl2, k.sl2, b0, b1);
      }
    }
    return;
  }
  const float top = kCap ? base + k.cap_a : base;
#pragma unroll
  for (int n = 0; n < N; n += 2) {
    float b0 = top, b1 = top;
    if constexpr (kDist) ffma2(b0, b1, step, step, (float)n, (float)(n + 1), top, top);
    if constexpr (kCap) {
      float r0, r1;
      cap_pair(r0, r1, s[n], s[n + 1], k.cap_c);
      if constexpr (kGrad) {
        float t0, t1;
        fmul2(t0, t1, r0, r1, 4.f, 4.f);
        ffma2(w[n], w[n + 1], -t0, -t1, r0, r1, t0, t1);
      }
      ffma2(s[n], s[n + 1], r0, r1, -2.f * k.cap_a, -2.f * k.cap_a, b0, b1);
    } else if constexpr (kDist) {
      ffma2(s[n], s[n + 1], s[n], s[n + 1], k.sl2, k.sl2, b0, b1);
    } else {
      fmul2(s[n], s[n + 1], s[n], s[n + 1], k.sl2, k.sl2);
    }
  }
}

}  // namespace thd
