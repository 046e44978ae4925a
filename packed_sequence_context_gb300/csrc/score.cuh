// The score function of scored attention, for one thread's run of scores.
//
//   x = softmax_scale * s                       (s = q . k, fp32 in TMEM)
//   y = softcap tanh(x / softcap)   or  x
//   y -= slope |i' - j|                         (i' = i + koff: the key position a query sits at)
// in log2 units (y log2(e)), as the softmax takes them.
//
// tanh, chosen per warp and run of scores by the largest |x| of the run (see
// cap_form):
//   s times a polynomial in s^2, a relative minimax fit of tanh(u) / u derived
//     by exchange on the interval: three terms for |x| <= 0.28 softcap (relative
//     error 7.8e-7), five for |x| <= 0.75 softcap (5.7e-7);
//   else 1 - 2 r, r = 1 / (1 + e^(2u)): one 2^x and one reciprocal, shared by
//     two scores (1/a = b / (ab), 1/b = a / (ab), with exponents held to 2^60
//     so that ab stays finite; tanh is 1 to the last bit long before).
// All are exact to fp32 rounding in absolute terms (about softcap 2^-21; the
// hardware's one-step tanh is off by 2^-11, 0.02 at a cap of 50).  What a run
// costs, from a loop of the softmax's steps with two warps per scheduler, in
// cycles per 32 scores: no cap 4.8, three terms 7.0, five 9.6, the reciprocal
// 13.1 -- the softmax's 2^x alone is 4 of them, so the polynomials, which take
// only multiply-adds, run beside it.
//
// The bias is linear in j on either side of i', so a row that sees only keys
// up to its own position (every causal row without a prefix) takes one fused
// multiply-add for it; other rows take the absolute value.  base + step n leaves
// near keys the rounding of the base, 2^-19 of the slope in a run of 32, so heads
// with a steep slope take the absolute value too, and dQ, where that choice took
// 5% of the kernel (cap and bias, 5.94 -> 6.24 ms), forms the distance first
// (kExact: one more addition for two scores, 6.03 ms).
#pragma once

#include <climits>

#include "common.cuh"
#include "ptx.cuh"

namespace thd {

THD_DEV float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct ScoreConsts {
  float sl2;       // softmax_scale log2(e)
  float cap_a;     // softcap log2(e)
  float cap_c;     // 2 log2(e) softmax_scale / softcap
  float cap_n[3], cap_near;  // tanh = s (n0 + n1 s^2 + ..) while |s| <= cap_near; kForward: times cap_a
  float cap_f[5], cap_far;
  float cap_sat;
  float slope;  // the head's slope log2(e)
};
template <int kMod, bool kForward, class P>
THD_DEV ScoreConsts score_consts(const P& p, int h) {
  ScoreConsts k;
  k.sl2 = p.scale_log2;
  k.cap_a = p.mods.cap_a;
  k.cap_c = p.mods.cap_c;
#pragma unroll
  for (int i = 0; i < 3; ++i) k.cap_n[i] = p.mods.cap_n[i] * (kForward ? k.cap_a : 1.f);
#pragma unroll
  for (int i = 0; i < 5; ++i) k.cap_f[i] = p.mods.cap_f[i] * (kForward ? k.cap_a : 1.f);
  k.cap_near = p.mods.cap_near;
  k.cap_far = p.mods.cap_far;
  k.cap_sat = p.mods.cap_sat;
  k.slope = 0.f;
  if constexpr ((kMod & kModDist) != 0) k.slope = p.mods.slopes[h] * 1.4426950408889634f;
  return k;
}

// The largest |s| of a thread's scores.
template <int N>
THD_DEV float score_abs_max(const float (&s)[N]) {
  float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int n = 0; n < N; n += 8)
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = fmax3(m[i], fabsf(s[n + 2 * i]), fabsf(s[n + 2 * i + 1]));
  return fmax3(fmaxf(m[0], m[1]), m[2], m[3]);
}

// The scores outside [from, to) become v.  Runs with masked columns set those
// to 0 before the largest |s| is taken: a masked score, or a column that no
// product wrote, must not choose the form (results stay reproducible).
template <int N>
THD_DEV void score_fill(float (&s)[N], int from, int to, float v) {
  const int lo = from < 0 ? 0 : (from > N ? N : from), hi = to > N ? N : to;
  const uint32_t n_seen = hi > lo ? (uint32_t)(hi - lo) : 0u;
#pragma unroll
  for (int n = 0; n < N; ++n)
    if ((uint32_t)(n - lo) >= n_seen) s[n] = v;
}

// The same for 32 bf16 numbers in pairs, which become 0.
THD_DEV void score_mask(uint32_t (&s)[16], int from, int to) {
  const int lo = from < 0 ? 0 : from, hi = to > 32 ? 32 : to;
  const uint32_t n_seen = hi > lo ? (uint32_t)(hi - lo) : 0u;
#pragma unroll
  for (int n = 0; n < 32; n += 2)
    s[n / 2] &= ((uint32_t)(n - lo) < n_seen ? 0xffffu : 0u) | ((uint32_t)(n + 1 - lo) < n_seen ? 0xffff0000u : 0u);
}

// Which form of tanh the warp's run takes: the first whose range holds the
// largest |s| of every thread (a NaN among the scores may pass for small: it
// stays a NaN in every form), and none below that of the warp's earlier runs in
// the same work item.  A run is computed in the item's form while the maximum
// is taken, instead of after a decision, and again from TMEM if the scores call
// for a wider one; the result depends on the item's scores alone.  (The three
// forms in a loop over "the form to try next" made the compiler move every
// score between registers: 5850 instead of 3560 instructions in a forward tile.)
constexpr int kCapNear = 0, kCapFar = 1, kCapWide = 2;
template <int kForm>
struct CapForm {
  static constexpr int value = kForm;
};
THD_DEV int cap_form(float abs_max, const ScoreConsts& k) {
  if (__all_sync(0xffffffffu, abs_max <= k.cap_near)) return kCapNear;
  return __all_sync(0xffffffffu, abs_max <= k.cap_far) ? kCapFar : kCapWide;
}
// run(CapForm<f>) loads the scores, computes in form f and returns the form the
// scores call for.
template <typename F>
THD_DEV void cap_in_form(int& form, F&& run) {
  bool done = false;
  if (form == kCapNear) {
    form = run(CapForm<kCapNear>{});
    done = form == kCapNear;
  }
  if (!done && form == kCapFar) {
    done = run(CapForm<kCapFar>{}) != kCapWide;
    if (!done) form = kCapWide;
  }
  if (!done) run(CapForm<kCapWide>{});
}

// dK/dV has a form more, for scores past cap_sat (see cap_sat_run).
constexpr int kCapSat = 3;
THD_DEV int cap_form_sat(float abs_max, const ScoreConsts& k) {
  if (__all_sync(0xffffffffu, abs_max <= k.cap_near)) return kCapNear;
  if (__all_sync(0xffffffffu, abs_max <= k.cap_far)) return kCapFar;
  return __any_sync(0xffffffffu, abs_max > k.cap_sat) ? kCapSat : kCapWide;
}
template <typename F>
THD_DEV void cap_in_form_sat(int& form, F&& run) {
  bool done = false;
  if (form == kCapNear) {
    form = run(CapForm<kCapNear>{});
    done = form == kCapNear;
  }
  if (!done && form == kCapFar) {
    const int f = run(CapForm<kCapFar>{});
    done = f <= kCapFar;
    if (!done) form = f;
  }
  if (!done && form == kCapWide) {
    done = run(CapForm<kCapWide>{}) != kCapSat;
    if (!done) form = kCapSat;
  }
  if (!done) run(CapForm<kCapSat>{});
}

// The polynomial's value at two scores: tanh = s times it.
template <int kForm>
THD_DEV void cap_poly(float& q0, float& q1, float s0, float s1, const ScoreConsts& k) {
  float w0, w1;
  fmul2(w0, w1, s0, s1, s0, s1);
  if constexpr (kForm == kCapNear) {
    ffma2(q0, q1, w0, w1, k.cap_n[2], k.cap_n[2], k.cap_n[1], k.cap_n[1]);
    ffma2(q0, q1, w0, w1, q0, q1, k.cap_n[0], k.cap_n[0]);
  } else {
    ffma2(q0, q1, w0, w1, k.cap_f[4], k.cap_f[4], k.cap_f[3], k.cap_f[3]);
    ffma2(q0, q1, w0, w1, q0, q1, k.cap_f[2], k.cap_f[2]);
    ffma2(q0, q1, w0, w1, q0, q1, k.cap_f[1], k.cap_f[1]);
    ffma2(q0, q1, w0, w1, q0, q1, k.cap_f[0], k.cap_f[0]);
  }
}

// r = 1 / (1 + 2^(c s)) of two scores: tanh = 1 - 2 r.
THD_DEV void cap_wide(float& r0, float& r1, float s0, float s1, float c) {
  float x0, x1, a0, a1;
  fmul2(x0, x1, s0, s1, c, c);
  fadd2(a0, a1, ex2(fmin_nan(x0, 60.f)), ex2(fmin_nan(x1, 60.f)), 1.f, 1.f);
  const float q = rcp(a0 * a1);
  fmul2(r0, r1, q, q, a1, a0);
}

// dQ's wide form, of two scores: R = 2 / (1 + e), e = 2^(c s), gives tanh = 1 - R
// and w = 1 - tanh^2 = e R^2, as many instructions as 1 - tanh^2 from tanh, and w
// keeps its relative precision however near to 1 |tanh| is.  From a rounded tanh
// it is off by up to 2^-22 / w: 2e-4 at x / cap = 4, 3% at 7, 20% at 8, and twice
// that at -7 and -8.
THD_DEV void cap_wide_grad(float& r0, float& r1, float& w0, float& w1, float s0, float s1, float c) {
  float x0, x1, a0, a1;
  fmul2(x0, x1, s0, s1, c, c);
  const float e0 = ex2(fmin_nan(x0, 60.f)), e1 = ex2(fmin_nan(x1, 60.f));
  ffma2(a0, a1, e0, e1, 0.5f, 0.5f, 0.5f, 0.5f);
  const float q = rcp(a0 * a1);
  fmul2(r0, r1, q, q, a1, a0);
  fmul2(w0, w1, e0, e1, r0, r1);
  fmul2(w0, w1, w0, w1, r0, r1);
}

// dK/dV's form for saturated scores.  It makes P and 1 - tanh^2 in a pass of their
// own, from one value a score, and has no register left for R and e there: that
// took 9.1 instead of 8.5 ms (32,768 tokens, 16 + 4 heads of 128, cap 50) whatever
// the form.  Here the value is u = sign(s) (1 - |tanh|) = sign(s) 2 z / (1 + z),
// z = 2^(-c |s|); with S = sign(u), tanh = S - u and 1 - tanh^2 = u (S + tanh).  It
// takes more instructions than the wide form (every score past 4: 8.5 -> 10.2 ms),
// hence only from x / cap = 4 on (cap_sat), where that is off by 2e-4.  A fifth copy
// of that pass (with a cap and a bias both sides of it, cut or not) took 10.4
// instead of 8.7 ms, so under a cap the bias of both sides always has the cut.
template <int N>
THD_DEV void cap_sat_run(float (&s)[N], float c) {
#pragma unroll
  for (int n = 0; n < N; n += 2) {
    const float z0 = ex2(-c * fabsf(s[n])), z1 = ex2(-c * fabsf(s[n + 1]));
    float a0, a1, r0, r1;
    ffma2(a0, a1, z0, z1, 0.5f, 0.5f, 0.5f, 0.5f);
    const float q = rcp(a0 * a1);  // z <= 1: no limit on the exponents
    fmul2(r0, r1, q, q, a1, a0);
    fmul2(r0, r1, r0, r1, z0, z1);
    s[n] = copysignf(r0, s[n]);
    s[n + 1] = copysignf(r1, s[n + 1]);
  }
}
// tanh and 1 - tanh^2 of two scores, from tanh or (kSat) from u.
template <bool kSat>
THD_DEV void cap_tanh(float& t0, float& t1, float s0, float s1) {
  t0 = s0, t1 = s1;
  if constexpr (kSat) fadd2(t0, t1, copysignf(1.f, s0), copysignf(1.f, s1), -s0, -s1);
}
template <bool kSat>
THD_DEV void cap_slope(float& w0, float& w1, float s0, float s1, float t0, float t1) {
  if constexpr (kSat) {
    fadd2(w0, w1, copysignf(1.f, s0), copysignf(1.f, s1), t0, t1);
    fmul2(w0, w1, w0, w1, s0, s1);
  } else {
    ffma2(w0, w1, -t0, -t1, t0, t1, 1.f, 1.f);
  }
}

// A run's bias: score n has b(n) = -slope |d0 + dir n|, dir = -1 where the
// scores run along j and +1 along i'.  kAbs: some score sits past its own
// position; else b(n) = base + step n, or with kExact top - slope (d0 + dir n).
template <int kDir, bool kAbs, bool kExact = false>
struct BiasRun {
  float d0, slope, base, step;
  THD_DEV BiasRun(float d0_, float slope_, float top) : d0(d0_), slope(slope_) {
    base = kAbs || kExact ? top : top - slope_ * d0_;
    step = -slope_ * kDir;
  }
  THD_DEV void at(int n, float& b0, float& b1) const {
    if constexpr (kAbs) {
      b0 = fmaf(-slope, fabsf(d0 + kDir * n), base);
      b1 = fmaf(-slope, fabsf(d0 + kDir * (n + 1)), base);
    } else if constexpr (kExact) {
      float t0, t1;
      fadd2(t0, t1, (float)(kDir * n), (float)(kDir * (n + 1)), d0, d0);
      ffma2(b0, b1, t0, t1, -slope, -slope, base, base);
    } else {
      ffma2(b0, b1, step, step, (float)n, (float)(n + 1), base, base);
    }
  }
};

// A row at key position `at` takes the linear side for tiles whose keys it sees up
// to this position: its own, or with a steep slope (log2 units) none.
constexpr float kSteepBias = 4.f;
THD_DEV int linear_to(const ScoreConsts& k, int at) { return fabsf(k.slope) > kSteepBias ? INT_MIN / 2 : at; }

// One thread's N scores, in place: s[n] becomes a s[n] + b(n) + top.
template <int kDir, bool kAbs, int N>
THD_DEV void bias_run(float (&s)[N], float a, float d0, float slope, float top) {
  const BiasRun<kDir, kAbs> b(d0, slope, top);
#pragma unroll
  for (int n = 0; n < N; n += 2) {
    float b0, b1;
    b.at(n, b0, b1);
    ffma2(s[n], s[n + 1], s[n], s[n + 1], a, a, b0, b1);
  }
}

// One thread's N scores become scale tanh + bias + top, in place (polynomials:
// scale is in the coefficients; without a bias top is 0).  Linear side of the
// bias.
template <int kForm, int kDir, bool kDist, int N>
THD_DEV void cap_run(float (&s)[N], const ScoreConsts& k, float scale, float d0, float top) {
  if (kForm == kCapWide) top += scale;
  const BiasRun<kDir, false> b(d0, k.slope, top);
#pragma unroll
  for (int n = 0; n < N; n += 2) {
    float q0, q1, b0 = top, b1 = top;
    if constexpr (kDist) b.at(n, b0, b1);
    if constexpr (kForm == kCapWide) {
      cap_wide(q0, q1, s[n], s[n + 1], k.cap_c);
      ffma2(s[n], s[n + 1], q0, q1, -2.f * scale, -2.f * scale, b0, b1);
    } else {
      cap_poly<kForm>(q0, q1, s[n], s[n + 1], k);
      if constexpr (kDist)
        ffma2(s[n], s[n + 1], s[n], s[n + 1], q0, q1, b0, b1);
      else
        fmul2(s[n], s[n + 1], s[n], s[n + 1], q0, q1);
    }
  }
}

// Forward: one thread's N scores become y log2(e) + top, in place (coefficients
// scaled by cap_a; without a bias top is 0).  d0 and abs_needed as in BiasRun
// (abs_needed uniform over the warp).
template <int kMod, int kForm, int kDir, int N>
THD_DEV void score_run(float (&s)[N], const ScoreConsts& k, float d0, bool abs_needed, float top) {
  constexpr bool kCap = (kMod & kModCap) != 0, kDist = (kMod & kModDist) != 0;
  if constexpr (kCap) {
    if (kDist && !abs_needed) {  // cap and bias in one go
      cap_run<kForm, kDir, true>(s, k, k.cap_a, d0, top);
      return;
    }
    cap_run<kForm, kDir, false>(s, k, k.cap_a, 0.f, 0.f);
  }
  if constexpr (kDist) {
    const float a = kCap ? 1.f : k.sl2;
    if (abs_needed)
      bias_run<kDir, true>(s, a, d0, k.slope, top);
    else
      bias_run<kDir, false>(s, a, d0, k.slope, top);
  }
}

// The largest bias (log2 units) a query at key position `at` gets from the keys
// [lo, hi) it sees: of the nearest, or with a negative slope of the farthest.
THD_DEV float largest_bias(float slope, int at, int lo, int hi) {
  if (hi <= lo) return 0.f;
  const int below = at - lo, above = hi - 1 - at;  // distances to the two ends, where those lie
  const int d = slope >= 0.f ? imax(imax(-below, -above), 0) : imax(below, above);
  return -slope * (float)d;
}

}  // namespace thd
