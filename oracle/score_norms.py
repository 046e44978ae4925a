"""How large the errors of scored attention and its gradients are to be, row by
row and head by head: the root mean square that the roundings to bf16 add up
to, against which an output's distance from fp64 is held.  The elementwise
bounds of score_oracle take every rounding at its worst and in the worst
direction; a mistake of a few percent in a gradient passes under them.  numpy
only; shares no code with the GPU path.

Model.  Rounding x to bf16 (8 significant bits) is off by at most half a unit in
the last place, 2^-9 2^e for |x| in [2^e, 2^(e+1)); over the mantissas its mean
square is at most (2^-8 |x|)^2 / 3, so R = 2^-8 / sqrt(3) bounds the relative
root mean square of one rounding.  Roundings are independent:
  O_i   = sum_j P_ij V_j        mean square  sum_j R^2 P^2 V^2 + R^2 O^2
  dQ_i  = c sum_j dS_ij K_j                  c^2 sum_j R^2 dS^2 K^2 + R^2 dQ^2
  dK_j, dV_j likewise over i, with dS and P.
dS = P (dP - Delta) w with w = 1 - tanh^2.  Where Delta = rowsum(dO O) is taken
from O in bf16 instead of being corrected, Delta's mean square is
sum_d dO^2 (mean square of O) and all of a row's dS share it:
  dQ_i gains c^2 that (sum_j P w K_j)^2.
With heads of 64 dQ is made with Delta from O and corrected in every row, by
how far Delta was off times sum_j P w K_j: both carry that into a rounding,
  dQ_i gains c^2 2 R^2 that sum_j P^2 w^2 K^2.
Errors of fp32: P is off relatively by that of the scores, taken as in
score_oracle at a quarter (they are sums of many roundings, there at their
worst), and dP - Delta by D 2^-24 sum |dO||V| / 4.

A row's error norm is held to 3 times the model's root mean square: a rounding
is at most sqrt(3) R, the keys a row weighs are far from parallel, and the
mean square is met on the average only.  A head's, over all of its rows, is
held to 1.25 times: it averages hundreds of them."""

from __future__ import annotations

import numpy as np

from oracle.score_oracle import _softmax_rows, visible

R = 2.0 ** -8 / np.sqrt(3.0)
ROW, HEAD = 3.0, 1.25


def delta_corrected(see, slope, doc_q, doc_k, tile=128, few=256, steep=0.375):
    """[lq] bool: which rows' dQ is to have the corrected Delta where the head's
    size is not 64.  All of them with a steep slope; else those whose keys lie inside the few keys of their
    tile of rows: from the first row's first key, or the end of its document if
    that row sees many, to the last row's last key, or the start of its
    document."""
    lq, lk = see.shape
    out = np.full(lq, abs(slope) >= steep)
    count = see.sum(1)
    lo, hi = see.argmax(1), lk - see[:, ::-1].argmax(1)
    for t in range(0, lq, tile):
        a, z = t, min(t + tile, lq) - 1
        if not count[a] or not count[z]:   # rows that see nothing: not said here
            continue
        end = lk if doc_q is None else int(np.searchsorted(doc_k, doc_q[a], "right"))
        x = lo[a] if count[a] <= few else end
        y = hi[z] if count[z] <= few else lo[z]
        rows = slice(a, z + 1)
        out[rows] |= (lo[rows] >= x) & (hi[rows] <= y) & (x < y)
    return out


def model(q, k, v, cu_q, cu_k, pad_q, pad_k, *, causal, scale, softcap=0.0, slopes=None, doc_q=None, doc_k=None,
          prefix=None, do=None):
    """As score_oracle.score; the values, and the mean square error of each
    element as "ms_..."."""
    q, k, v, do = (np.asarray(x, np.float64) for x in (q, k, v, do))
    (tq, hq, D), hkv = q.shape, k.shape[1]
    G = hq // hkv
    out = {"o": np.zeros_like(q), "dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v)}
    out |= {"ms_" + n: np.zeros_like(x) for n, x in out.items()}
    for b in range(len(cu_q) - 1):
        lq, lk = int(cu_q[b + 1] - cu_q[b]), int(cu_k[b + 1] - cu_k[b])
        rq = slice(int(pad_q[b]), int(pad_q[b]) + lq)
        rk = slice(int(pad_k[b]), int(pad_k[b]) + lk)
        if lq == 0 or lk == 0:
            continue
        docs = (None, None) if doc_q is None else (np.asarray(doc_q)[rq], np.asarray(doc_k)[rk])
        see, at = visible(lq, lk, causal, None if prefix is None else int(prefix[b]), *docs)
        for h in range(hq):
            Q, K, V, dO = q[rq, h], k[rk, h // G], v[rk, h // G], do[rq, h]
            x = scale * (Q @ K.T)
            t = np.tanh(x / softcap) if softcap else np.zeros_like(x)
            slope = float(slopes[h]) if slopes is not None else 0.0
            bias = slope * np.abs(at[:, None] - np.arange(lk)[None, :])
            y = (softcap * t if softcap else x) - bias
            P, lse = _softmax_rows(np.where(see, y, -np.inf))
            fin = np.where(np.isfinite(lse), lse, 0.0)
            rel = scale * D * 2.0 ** -24 * (np.abs(Q) @ np.abs(K).T) + softcap * 2.0 ** -20
            rel = (rel + 2.0 ** -22 * (np.abs(bias) + np.abs(y) + np.abs(fin)[:, None])) / 4
            w = 1 - t * t
            O, dP = P @ V, dO @ V.T
            dp = dP - (dO * O).sum(-1)[:, None]
            dS = P * dp * w
            P2 = (R * P) ** 2
            ms_o = P2 @ V ** 2 + (R * O) ** 2
            s2 = (R ** 2 + rel ** 2) * dS ** 2
            s2 = s2 + (P * w * D * 2.0 ** -24 / 4 * (np.abs(dO) @ np.abs(V).T)) ** 2
            out["o"][rq, h], out["ms_o"][rq, h] = O, ms_o
            out["dq"][rq, h] = scale * dS @ K
            ms = scale ** 2 * s2 @ K ** 2 + (R * out["dq"][rq, h]) ** 2
            that = (dO ** 2 * ms_o).sum(-1)[:, None]
            if D == 64:
                ms = ms + scale ** 2 * 2 * R ** 2 * that * ((P * w) ** 2 @ K ** 2)
            else:
                that = that * ~delta_corrected(see, slope, *docs)[:, None]
                ms = ms + scale ** 2 * that * ((P * w) @ K) ** 2
            out["ms_dq"][rq, h] = ms
            out["dk"][rk, h // G] += scale * dS.T @ Q
            out["ms_dk"][rk, h // G] += scale ** 2 * s2.T @ Q ** 2
            out["dv"][rk, h // G] += P.T @ dO
            out["ms_dv"][rk, h // G] += (P2 + (rel * P) ** 2).T @ dO ** 2
    for n in ("dk", "dv"):
        out["ms_" + n] += (R * out[n]) ** 2
    return out


def ratios(name, got, m):
    """The largest of a row's and of a head's error norm over its limit."""
    e2 = ((np.asarray(got, np.float64) - m[name]) ** 2).sum(-1)
    ms = m["ms_" + name].sum(-1)
    floor = 1e-12 * (m[name] ** 2).sum(-1).max() + 1e-60
    row = np.sqrt(e2 / (ms + floor)).max() / ROW
    head = np.sqrt(e2.sum(0) / (ms + floor).sum(0)).max() / HEAD
    return float(row), float(head)
