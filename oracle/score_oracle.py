"""Plain fp64 CPU oracle of scored attention (tanh cap, distance bias,
document and prefix masks) over packed sequences, forward and backward, with
elementwise bounds on what an evaluation in bf16 tensor-core products may be
off by.  numpy only; shares no code with the GPU path.

Bounds.  u = 2^-8 is the largest relative error of a rounding to bf16.  `dl`
bounds the error of a score (natural units) evaluated in fp32: the D products
and sums of s (D 2^-24 sum |q||k|), the cap (softcap 2^-20: one 2^x, one
reciprocal and a fused multiply-add), the bias (2^-22 of it) and the
conversion to log2 units and back (2^-22 |y|).
  lse: dl of the row's largest, plus 2^-20 for the sum and its logarithm,
       plus 2^-22 |lse|
  P = e^(y - lse): relative (u + dl + dlse), u for its own rounding to bf16
  O:  sum of that over P |v|, and its rounding u |O|
  Delta = rowsum(dO O): sum |dO| tol(O), O being stored in bf16
  dS: relative (u + dl + dlse) and P w (tol(Delta) + D 2^-24 sum |dO||v|); w =
      1 - tanh^2 is off relatively by 2^-12 (a rounded tanh's 2^-22 against the
      1.3e-3 it is at x / softcap = 4) and 2 / softcap times the error of x
  dQ, dK, dV: those errors through the product, and the result's rounding."""

from __future__ import annotations

import numpy as np

U = 2.0 ** -8


def visible(lq, lk, causal, prefix, doc_q, doc_k):
    """[lq, lk] bool, and the key position every query sits at."""
    at = np.arange(lq) + (lk - lq if causal == 2 else 0)
    j = np.arange(lk)
    see = np.ones((lq, lk), bool)
    if causal:
        see = (j[None, :] <= at[:, None]) | (j < (prefix or 0))[None, :]
    if doc_q is not None:
        see &= np.asarray(doc_q)[:, None] == np.asarray(doc_k)[None, :]
    return see, at


def _softmax_rows(y):
    m = y.max(-1, keepdims=True) if y.shape[1] else np.full((y.shape[0], 1), -np.inf)
    m = np.where(np.isfinite(m), m, 0.0)
    e = np.exp(y - m)
    l = e.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(l))[:, 0]
    return np.where(l > 0, e / np.where(l > 0, l, 1.0), 0.0), lse


def score(q, k, v, cu_q, cu_k, pad_q, pad_k, *, causal, scale, softcap=0.0, slopes=None, doc_q=None, doc_k=None,
          prefix=None, do=None):
    """q [Tq, Hq, D], k, v [Tk, Hkv, D].  Returns {"o", "lse"} and with do
    {"dq", "dk", "dv"}, each with "tol_..." of its shape."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    tq, hq, D = q.shape
    tk, hkv, _ = k.shape
    G = hq // hkv
    out = {"o": np.zeros((tq, hq, D)), "lse": np.full((hq, tq), -np.inf)}
    out["tol_o"], out["tol_lse"] = np.zeros((tq, hq, D)), np.zeros((hq, tq))
    if do is not None:
        do = np.asarray(do, np.float64)
        for n, shape in (("dq", q.shape), ("dk", k.shape), ("dv", k.shape)):
            out[n], out["tol_" + n] = np.zeros(shape), np.zeros(shape)
    for b in range(len(cu_q) - 1):
        lq, lk = int(cu_q[b + 1] - cu_q[b]), int(cu_k[b + 1] - cu_k[b])
        rq = slice(int(pad_q[b]), int(pad_q[b]) + lq)
        rk = slice(int(pad_k[b]), int(pad_k[b]) + lk)
        if lq == 0 or lk == 0:
            continue
        see, at = visible(lq, lk, causal, None if prefix is None else int(prefix[b]),
                          None if doc_q is None else doc_q[rq], None if doc_k is None else doc_k[rk])
        for h in range(hq):
            Q, K, V = q[rq, h], k[rk, h // G], v[rk, h // G]
            x = scale * (Q @ K.T)
            t = np.tanh(x / softcap) if softcap else np.zeros_like(x)
            y = softcap * t if softcap else x
            far = np.abs(at[:, None] - np.arange(lk)[None, :])
            bias = float(slopes[h]) * far if slopes is not None else np.zeros_like(x)
            y = y - bias
            dl = scale * D * 2.0 ** -24 * (np.abs(Q) @ np.abs(K).T) + softcap * 2.0 ** -20
            dl = dl + 2.0 ** -22 * (np.abs(bias) + np.abs(y))
            P, lse = _softmax_rows(np.where(see, y, -np.inf))
            O = P @ V
            live = np.isfinite(lse)
            tl = np.where(live, (dl * see).max(-1) + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(live, lse, 0)), 0.0)
            rel = (U + dl + tl[:, None]) * P * 1.01
            to = rel @ np.abs(V) + U * 1.01 * np.abs(O) + 1e-30
            out["o"][rq, h], out["lse"][h, rq] = O, lse
            out["tol_o"][rq, h], out["tol_lse"][h, rq] = to, tl
            if do is None:
                continue
            dO = do[rq, h]
            dP = dO @ V.T
            w = 1 - t * t
            delta = (dO * O).sum(-1)
            dS = P * (dP - delta[:, None]) * w
            td = (np.abs(dO) * to).sum(-1)
            es = (U + dl + tl[:, None] + 2.0 ** -20) * np.abs(dS) * 1.01
            es = es + P * (td[:, None] + D * 2.0 ** -23 * (np.abs(dO) @ np.abs(V).T)) * (w + 2.0 ** -20) * 1.02
            if softcap:
                dx = scale * D * 2.0 ** -24 * (np.abs(Q) @ np.abs(K).T)
                es = es + (2.0 ** -12 + 2 / softcap * dx) * np.abs(dS)
            out["dq"][rq, h] = scale * dS @ K
            out["tol_dq"][rq, h] = scale * es @ np.abs(K)
            out["dk"][rk, h // G] += scale * dS.T @ Q
            out["tol_dk"][rk, h // G] += scale * es.T @ np.abs(Q)
            out["dv"][rk, h // G] += P.T @ dO
            out["tol_dv"][rk, h // G] += rel.T @ np.abs(dO)
    if do is not None:
        for n in ("dq", "dk", "dv"):
            out["tol_" + n] = out["tol_" + n] * 1.01 + U * 1.01 * np.abs(out[n]) + 1e-30
    return out
