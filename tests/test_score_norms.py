"""Scored attention's gradients, row by row and head by head, against the error
that the roundings to bf16 add up to (oracle/score_norms.py).

On the CPU: an evaluation with exactly those roundings keeps the limits, and
each of the mistakes planted in it breaks them, the small ones that pass under
the elementwise bounds among them.  On the GPU: the library's gradients, on
masks and biases that leave rows a few keys each."""

import numpy as np
import pytest
import torch

from oracle import score_norms as sn
from oracle import score_oracle as so
from packed_sequence_context_gb300 import inputs
from packed_sequence_context_gb300 import thd_attn as T


def _docs(lengths, n):
    out = np.repeat(np.arange(1000), np.resize(lengths, 1000))
    return out[:n].astype(np.int32)


CASES = {
    # name: lengths, Hq, Hkv, D, causal, mods
    "plain masks": ([700, 130], 2, 1, 64, 1, {"prefix": [40, 9]}),
    "cap": ([900], 2, 2, 128, 1, {"cap": 20.0, "std": 2.0}),
    "steep": ([1024], 4, 1, 128, 1, {"slopes": [2.0, 0.7071, 0.25, 0.0625]}),
    "gentle": ([1024], 3, 1, 64, 1, {"slopes": [0.06, 0.03, 0.004]}),
    "steep cap": ([1024], 4, 2, 64, 1, {"slopes": [2.0, 0.7071, 0.125, 0.01], "cap": 30.0}),
    "far keys": ([640], 2, 2, 64, 0, {"slopes": [-0.5, -0.01]}),
    "documents of few": ([1000], 2, 2, 64, 1, {"docs": [2, 4, 3]}),
    "documents in wide tiles": ([1200], 2, 1, 128, 1, {"docs": [700, 3, 290, 5]}),
    "documents both ways": ([900], 2, 2, 64, 0, {"docs": [300, 6, 280], "cap": 15.0}),
    "near the cap": ([500], 2, 1, 64, 1, {"cap": 6.0, "std": 5.0}),
    # every score at 5.5 to 8.5 times the cap, of either sign
    "saturated": ([300], 2, 2, 64, 1, {"cap": 5.0, "saturated": 0.5}),
    "saturated below": ([300], 2, 1, 128, 1, {"cap": 5.0, "saturated": 1.0, "slopes": [0.01, -0.02]}),
    # the row's own key or its neighbour has all of the weight, at a bias of 0 beside biases of 1e2 to 1e7
    "very steep": ([500, 37], 4, 2, 64, 1, {"slopes": [40.0, 300.0, 3.0e4, 1.0e6]}),
    "very steep cap": ([500, 37], 3, 3, 128, 1, {"slopes": [40.0, 3.0e4, 1.0e6], "cap": 20.0}),
    "very steep both ways": ([300], 2, 1, 64, 0, {"slopes": [100.0, 1.0e5], "cap": 9.0}),
    "gathered scores, small heads": ([800], 4, 2, 64, 1, {"cap": 50.0, "std": 6.0}),
    "gathered scores, masks": ([800, 300], 2, 2, 64, 1, {"prefix": [70, 9], "std": 6.0}),
    "gathered scores": ([800], 2, 2, 128, 1, {"cap": 50.0, "std": 6.0}),
}


def _make(name):
    lengths, Hq, Hkv, D, causal, mods = CASES[name]
    seed = 1000 + sum(map(ord, name))
    c = inputs.make_cross(lengths, lengths, pad_to=4, Hq=Hq, Hkv=Hkv, D=D, cp_size=2, seed=seed)
    c["q"] = (c["q"].float() * mods.get("std", 1.5)).bfloat16()
    if "saturated" in mods:   # the scores lie on the first element: 5 x 7, spread by the other elements' share of them
        rng = np.random.default_rng(seed)
        n, hk = c["k"].shape[0], Hkv
        c["q"] *= 0.3
        c["q"][:, :, 0] = 16.0
        sign = torch.from_numpy(np.where(rng.random((n, hk)) < mods["saturated"], -1.0, 1.0))
        size = 35.0 + 5.0 * torch.from_numpy(rng.uniform(-1, 1, (n, hk)))
        c["k"][:, :, 0] = (sign * size * D ** 0.5 / 16).bfloat16()
    m = {"softcap": mods.get("cap", 0.0), "slopes": None, "doc_q": None, "doc_k": None, "prefix": None}
    if "slopes" in mods:
        m["slopes"] = np.array(mods["slopes"], np.float32)
    if "docs" in mods:
        m["doc_q"] = m["doc_k"] = _docs(mods["docs"], int(c["cu_q_pad"][-1]))
    if "prefix" in mods:
        m["prefix"] = np.array(mods["prefix"], np.int32)
    return c, m, causal, D ** -0.5


def _args(c):
    n = lambda x: c[x].float().numpy()  # noqa: E731
    return (n("q"), n("k"), n("v"), c["cu_q"], c["cu_kv"], c["cu_q_pad"], c["cu_kv_pad"]), n("do")


# ------------------------------------------------------------------ no GPU
def _bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().double().numpy()


def _rounded(c, m, causal, scale, mistake=None):
    """The gradients with P, dS, O and the results rounded to bf16, all else in
    64 bits, and one mistake."""
    (q, k, v, cu_q, cu_k, pad_q, pad_k), do = _args(c)
    q, k, v, do = (x.astype(np.float64) for x in (q, k, v, do))
    G = q.shape[1] // k.shape[1]
    out = {n: np.zeros_like(x) for n, x in (("o", q), ("dq", q), ("dk", k), ("dv", v))}
    for b in range(len(cu_q) - 1):
        lq, lk = int(cu_q[b + 1] - cu_q[b]), int(cu_k[b + 1] - cu_k[b])
        rq, rk = slice(int(pad_q[b]), int(pad_q[b]) + lq), slice(int(pad_k[b]), int(pad_k[b]) + lk)
        docs = (None, None) if m["doc_q"] is None else (m["doc_q"][rq], m["doc_k"][rk])
        see, at = so.visible(lq, lk, causal, None if m["prefix"] is None else int(m["prefix"][b]), *docs)
        for h in range(q.shape[1]):
            Q, K, V, dO = q[rq, h], k[rk, h // G], v[rk, h // G], do[rq, h]
            x = scale * (Q @ K.T)
            t = np.tanh(x / m["softcap"]) if m["softcap"] else 0 * x
            slope = float(m["slopes"][h]) if m["slopes"] is not None else 0.0
            y = (m["softcap"] * t if m["softcap"] else x) - slope * np.abs(at[:, None] - np.arange(lk))
            P, _ = so._softmax_rows(np.where(see, y, -np.inf))
            O = _bf16(_bf16(P) @ V)
            exact = sn.delta_corrected(see, slope, *docs) | (q.shape[2] == 64)
            if mistake == "Delta from O everywhere":
                exact[:] = False
            delta = np.where(exact, (dO * (P @ V)).sum(-1), (dO * O).sum(-1))
            delta_k = (dO * (P @ V)).sum(-1)
            if mistake == "Delta 2% off":
                delta, delta_k = 1.02 * delta, 1.02 * delta_k
            if mistake == "dK with Delta from O":
                delta_k = (dO * O).sum(-1)
            w = 1 - (0.98 if mistake == "0.98 tanh^2" else 1.0) * t * t
            if mistake == "1 - tanh^2 of a rounded tanh":
                w = 1 - t.astype(np.float32).astype(np.float64) ** 2
            if mistake == "a key too many":   # every row's first masked key
                first = np.where(see.any(1), see.argmax(1) - 1, -1)
                for i in np.flatnonzero(first >= 0):
                    P[i, first[i]] = 0.02 * P[i].max()
            sc = scale * (1.01 if mistake == "scale 1% off" else 1.0)
            dP = dO @ V.T
            out["o"][rq, h] = O
            out["dq"][rq, h] = sc * _bf16(P * (dP - delta[:, None]) * w) @ K
            out["dk"][rk, h // G] += sc * _bf16(P * (dP - delta_k[:, None]) * w).T @ Q
            out["dv"][rk, h // G] += _bf16(P).T @ dO
    return {n: _bf16(x) for n, x in out.items()}


def _worst(got, ref):
    return {n: max(sn.ratios(n, got[n], ref)) for n in ("o", "dq", "dk", "dv")}


@pytest.mark.parametrize("name", list(CASES))
def test_the_roundings_alone_keep_the_limits(name):
    c, m, causal, scale = _make(name)
    a, do = _args(c)
    ref = sn.model(*a, causal=causal, scale=scale, do=do, **m)
    assert max(_worst(_rounded(c, m, causal, scale), ref).values()) <= 1


def test_the_models_values_are_the_oracles():
    c, m, causal, scale = _make("documents both ways")
    a, do = _args(c)
    ref, orc = (f(*a, causal=causal, scale=scale, do=do, **m) for f in (sn.model, so.score))
    for n in ("o", "dq", "dk", "dv"):
        assert np.allclose(ref[n], orc[n], rtol=0, atol=1e-12)


@pytest.mark.parametrize("name,mistake,shows", [
    ("cap", "Delta 2% off", ("dq", "dk")), ("steep", "Delta 2% off", ("dq", "dk")),
    ("plain masks", "Delta 2% off", ("dq", "dk")), ("documents both ways", "Delta 2% off", ("dq", "dk")),
    ("steep", "Delta from O everywhere", ("dq",)), ("steep cap", "Delta from O everywhere", ("dq",)),
    ("documents of few", "Delta from O everywhere", ("dq",)),
    ("documents in wide tiles", "Delta from O everywhere", ("dq",)),
    ("gathered scores, small heads", "Delta from O everywhere", ("dq",)),
    ("gathered scores, masks", "Delta from O everywhere", ("dq",)),
    ("steep", "dK with Delta from O", ("dk",)), ("documents of few", "dK with Delta from O", ("dk",)),
    ("near the cap", "0.98 tanh^2", ("dq", "dk")),
    ("saturated", "1 - tanh^2 of a rounded tanh", ("dq", "dk")),
    ("saturated below", "1 - tanh^2 of a rounded tanh", ("dq", "dk")),
    ("documents in wide tiles", "a key too many", ("dv",)), ("gentle", "scale 1% off", ("dq", "dk"))])
def test_planted_mistakes_break_them(name, mistake, shows):
    c, m, causal, scale = _make(name)
    a, do = _args(c)
    ref = sn.model(*a, causal=causal, scale=scale, do=do, **m)
    got = _rounded(c, m, causal, scale, mistake)
    worst = _worst(got, ref)
    for n in shows:
        assert worst[n] > 1, (n, worst)


# ------------------------------------------------------------------ GPU
@pytest.mark.gpu
@pytest.mark.parametrize("kernel", [T.THD_FWD_KERNEL_SINGLE, T.THD_FWD_KERNEL_DUAL])
@pytest.mark.parametrize("name", [n for n in CASES if n.startswith("very steep")])
def test_lse_beside_far_larger_biases(thd_lib, name, kernel):
    """A row's lse against its scores' errors in score_oracle weighted by P: the
    biases of keys without weight count nothing."""
    c, m, causal, scale = _make(name)
    (q, k, v, cu, _, pad, _), _ = _args(c)
    g = lambda x: None if x is None else torch.from_numpy(x).cuda()  # noqa: E731
    off = [g(c[n]) for n in ("cu_q", "cu_kv", "cu_q_pad", "cu_kv_pad")]
    T.thd_test_select_fwd_kernel(kernel)
    try:
        _, lse, st = T.attn_score_fwd(c["q"].cuda(), c["k"].cuda(), c["v"].cuda(), *off, softcap=m["softcap"],
                                      dist_slopes=g(m["slopes"]), cp_size=2, causal=causal, softmax_scale=scale)
        T.check_status(st)
    finally:
        T.thd_test_select_fwd_kernel(0)
    q, k, D, G = q.astype(np.float64), k.astype(np.float64), q.shape[2], q.shape[1] // k.shape[1]
    for b in range(len(cu) - 1):
        rows = slice(int(pad[b]), int(pad[b] + cu[b + 1] - cu[b]))
        n = rows.stop - rows.start
        see, at = so.visible(n, n, causal, None, None, None)
        for h in range(q.shape[1]):
            Q, K = q[rows, h], k[rows, h // G]
            x = scale * Q @ K.T
            bias = float(m["slopes"][h]) * np.abs(at[:, None] - np.arange(n))
            y = (m["softcap"] * np.tanh(x / m["softcap"]) if m["softcap"] else x) - bias
            P, want = so._softmax_rows(np.where(see, y, -np.inf))
            dl = scale * D * 2.0 ** -24 * (np.abs(Q) @ np.abs(K).T) + m["softcap"] * 2.0 ** -20
            dl = dl + 2.0 ** -22 * (bias + np.abs(y))
            tol = (P * dl).sum(1) + 2.0 ** -20 + 2.0 ** -22 * np.abs(want)
            assert np.all(np.abs(lse[h, rows].double().cpu().numpy() - want) <= tol)


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_gradients_row_by_row(thd_lib, name):
    c, m, causal, scale = _make(name)
    a, do = _args(c)
    ref = sn.model(*a, causal=causal, scale=scale, do=do, **m)
    g = lambda x: None if x is None else torch.from_numpy(x).cuda()  # noqa: E731
    off = [g(c[n]) for n in ("cu_q", "cu_kv", "cu_q_pad", "cu_kv_pad")]
    d = {x: c[x].cuda() for x in ("q", "k", "v", "do")}
    kw = {"softcap": m["softcap"], "dist_slopes": g(m["slopes"]), "doc_q": g(m["doc_q"]), "doc_kv": g(m["doc_k"]),
          "prefix_len": g(m["prefix"]), "cp_size": 2, "causal": causal, "softmax_scale": scale}
    o, lse, st = T.attn_score_fwd(d["q"], d["k"], d["v"], *off, **kw)
    T.check_status(st)
    dq, dk, dv, st = T.attn_score_bwd(d["q"], d["k"], d["v"], o, lse, d["do"], *off, **kw)
    T.check_status(st)
    for n, x in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        row, head = sn.ratios(n, x.double().cpu().numpy(), ref)
        assert row <= 1 and head <= 1, f"{n}: a row at {row:.2f}, a head at {head:.2f} of its limit"
