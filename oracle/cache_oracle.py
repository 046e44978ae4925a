"""Plain fp64 CPU oracles of the paged key-value cache: append, attention of one
new token, eviction.  numpy only; shares no code with the GPU path.  A cache
here is a dict of arrays [pages, page_size, heads(, D)]: k, v (values, or for
an 8-bit cache the e4m3 numbers) and k_exp, v_exp (ints, or None)."""

from __future__ import annotations

import numpy as np

# the magnitudes of e4m3 by code: 0 .. 126 (127 is NaN)
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def to_e4m3(x):
    """Nearest e4m3 number, ties to the even code; |x| <= 448."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(E4M3, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return np.copysign(E4M3[code], x)


def row_exponent(row):
    """The stored exponent of a row: 255 for one with an infinity or NaN, 127
    for zeros, else the smallest e >= 67 with max |row| <= 448 * 2^(e - 127)."""
    big = np.max(np.abs(row))
    if not np.isfinite(big):
        return 255
    if big == 0:
        return 127
    e = 67
    while big > 448.0 * 2.0 ** (e - 127):
        e += 1
    return e


def slots(table_row, n, page):
    """(page, slot) of a sequence's first n slots."""
    j = np.arange(n)
    return np.asarray(table_row)[j // page], j % page


def append(cache, k, v, cu, table, kv_len, seen=None, weight=None, pos=None):
    """Copies of the arrays after the call."""
    out = {n: None if a is None else a.copy() for n, a in cache.items()}
    weight, pos = (None if a is None else a.copy() for a in (weight, pos))
    page = cache["k"].shape[1]
    for b in range(len(kv_len)):
        m = int(cu[b + 1] - cu[b])
        p, at = slots(table[b], int(kv_len[b]), page)
        for i in range(m):
            t, s = int(cu[b]) + i, int(kv_len[b]) - m + i
            for name, x in (("k", k), ("v", v)):
                for g in range(x.shape[1]):
                    if cache["k_exp"] is None:
                        out[name][p[s], at[s], g] = x[t, g]
                        continue
                    e = row_exponent(x[t, g])
                    out[name + "_exp"][p[s], at[s], g] = e
                    out[name][p[s], at[s], g] = np.nan if e == 255 else to_e4m3(x[t, g] * 2.0 ** (127 - e))
            if weight is not None:
                weight[p[s], at[s]] = 0
            if pos is not None:
                pos[p[s], at[s]] = (int(seen[b]) if seen is not None else int(kv_len[b])) - m + i
    return out, weight, pos


def decode(q, cache, table, kv_len, *, scale, softcap=0.0, slopes=None, start=None, pos=None, seen=None, weight=None):
    """q [B, Hq, D] -> dict(o, lse [Hq, B], weight) and a bound of each one's
    error in the kernel's arithmetic (tol_o, tol_lse, tol_weight):

    * a score is D products and sums in fp32 (D + 4 roundings of at most
      2^-24 of the sum of magnitudes, the scales included), then factors,
      tanh (4 units of its last place), the bias's product and sum, and the
      subtraction of the maximum: 8 roundings more of the score's, the cap's and
      the bias's magnitude;
    * exp2 to 2^-22, sums in fp32 (n 2^-24, by halves and by tiles: 2^-18 here
      for up to 64 x 1024 slots);
    * next to e4m3 keys, queries as fp16, off by at most 2^-39 of a head's
      largest element (elements far below it; 0 for the others);
    * probabilities rounded to bf16 (2^-8; 2^-16, as two numbers, up to 16 query
      heads a kv head), or next to e4m3 values to fp16 (2^-11, and 2^-32 of the
      largest product of probability and scale, rows of zeros left out: those
      count with the least scale, 2^-112), the output to bf16 (2^-8).
    """
    q = np.asarray(q, np.float64)
    B, Hq, D = q.shape
    page, Hkv = cache["k"].shape[1], cache["k"].shape[2]
    G, e4m3 = Hq // Hkv, cache["k_exp"] is not None
    o, lse = np.zeros((B, Hq, D)), np.full((Hq, B), -np.inf)
    tol_o, tol_lse = np.full((B, Hq, D), 1e-30), np.zeros((Hq, B))
    w = None if weight is None else np.asarray(weight, np.float64).copy()
    tol_w = None if weight is None else np.zeros(w.shape)
    half = 2.0 ** -11 if e4m3 else 2.0 ** -16 if G <= 16 else 2.0 ** -8
    for b in range(B):
        s0 = 0 if start is None else min(max(int(start[b]), 0), int(kv_len[b]))
        p, at = (x[s0:] for x in slots(table[b], int(kv_len[b]), page))
        if not len(p):
            continue
        for h in range(Hq):
            g = h // G
            k, v = (np.asarray(cache[n][p, at, g], np.float64) for n in ("k", "v"))
            if e4m3:
                k = k * 2.0 ** (np.asarray(cache["k_exp"][p, at, g], np.float64) - 127)[:, None]
                v = v * 2.0 ** (np.asarray(cache["v_exp"][p, at, g], np.float64) - 127)[:, None]
            x = scale * (k @ q[b, h])
            size = scale * (np.abs(k) @ np.abs(q[b, h]))
            y = softcap * np.tanh(x / softcap) if softcap else x
            err = 2.0 ** -24 * (D + 12) * size + 2.0 ** -21 * (softcap + np.abs(y))
            if e4m3:
                err = err + 2.0 ** -39 * scale * np.abs(q[b, h]).max() * np.abs(k).sum(1)
            if slopes is not None:
                num = np.asarray(pos[p, at, g], np.float64) if pos is not None else np.arange(s0, int(kv_len[b]))
                far = float(slopes[h]) * ((int(seen[b]) if seen is not None else int(kv_len[b])) - 1 - num)
                y = y - far
                err = err + 2.0 ** -22 * np.abs(far)
            m = y.max()
            e = np.exp(y - m)
            err = err + 2.0 ** -23 * (np.abs(m) + np.minimum(np.abs(y - m), 150))
            z = e.sum()
            pr = e / z
            rel = err + 2.0 ** -21
            dz = float((pr * rel).sum()) + 2.0 ** -18    # of the sum, relative
            o[b, h], lse[h, b] = pr @ v, m + np.log(z)
            tol_lse[h, b] = dz + 2.0 ** -22 * abs(lse[h, b]) + 2.0 ** -22 * abs(m)
            size = np.abs(v)
            # each weight: rounded, off by its score, by the sum; fp16 below its normal numbers (2^-32 of the largest
            # product of weight and value scale)
            tol_o[b, h] += ((pr * (half + rel + dz))[:, None] * size).sum(0) + 2.0 ** -8 * np.abs(o[b, h])
            if e4m3:
                size = 2.0 ** (np.asarray(cache["v_exp"][p, at, g], np.float64) - 127)
                top = float((pr * np.where(np.any(v != 0, 1), size, 2.0 ** -112)).max())
                tol_o[b, h] += 2.0 ** -32 * top * np.abs(np.asarray(cache["v"][p, at, g], np.float64)).sum(0)
            if w is not None:
                w[p, at, g] += pr
                tol_w[p, at, g] += pr * (rel + dz + 2.0 ** -20) + 1e-30
    if w is not None:
        tol_w += 2.0 ** -23 * np.abs(w) * (tol_w > 0)
    return {"o": o, "lse": lse, "weight": w, "tol_o": tol_o, "tol_lse": tol_lse, "tol_weight": tol_w}


def evict(cache, table, kv_len, weight, pos, seen, budget, sinks=0, recent=0):
    """(cache, weight, pos, new_len) after the call, weight and pos in place."""
    out = {n: None if a is None else a.copy() for n, a in cache.items()}
    wo, po = weight.copy(), pos.copy()
    page, Hkv = cache["k"].shape[1], cache["k"].shape[2]
    for b in range(len(kv_len)):
        n = int(kv_len[b])
        p, at = slots(table[b], n, page)
        for g in range(Hkv):
            if n <= budget:
                continue
            w = np.asarray(weight[p, at, g], np.float64).copy()
            # NaN counts as less than all: below -infinity too
            nan = np.isnan(w)
            w[nan] = -np.inf
            # the protected ones before any weight, the newest first
            age = int(seen[b]) - 1 - np.asarray(pos[p, at, g], np.int64)
            safe = (np.asarray(pos[p, at, g], np.int64) < sinks) | (age < recent)
            age = np.clip(age, 0, (1 << 23) - 2)
            order = sorted(range(n), key=lambda j: (0, age[j], j) if safe[j] else (1 + nan[j], -w[j], j))
            keep = np.zeros(n, bool)
            keep[order[:budget]] = True
            to = [j for j in range(budget) if not keep[j]]
            of = [j for j in range(budget, n) if keep[j]]
            for t, f in zip(to, of):
                for name in ("k", "v", "k_exp", "v_exp"):
                    if out[name] is not None:
                        out[name][p[t], at[t], g] = cache[name][p[f], at[f], g]
                wo[p[t], at[t], g] = weight[p[f], at[f], g]
                po[p[t], at[t], g] = pos[p[f], at[f], g]
    return out, wo, po, np.minimum(np.asarray(kv_len), budget)
