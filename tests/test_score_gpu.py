"""Scored attention (thd_attn_score_fwd / _bwd): the refusals on the CPU, and on
the GPU parity with the fp64 oracle, forward on both forward kernels and
backward, over caps, distance biases, documents and prefixes alone and
together, all three causal modes, lengths from one token, rows that see
nothing, odd lengths, padding, shared key heads, both head sizes and cp 1-8.

Tolerances are the oracle's elementwise bounds (see score_oracle): the bf16
roundings of P, dS, O and the results, and fp32 score errors."""

import numpy as np
import pytest
import torch

from oracle import score_oracle as so
from packed_sequence_context_gb300 import inputs
from packed_sequence_context_gb300 import thd_attn as T

KERNELS = [T.THD_FWD_KERNEL_SINGLE, T.THD_FWD_KERNEL_DUAL]


# ------------------------------------------------------------------ refusals (no GPU)
def _fwd(**kw):
    a = dict(q=16, k=16, v=16, o=16, lse=16, cq=16, ck=16, pq=None, pk=None, B=2, Tq=192, Tk=192, Hq=2, Hkv=2, D=64,
             causal=1, scale=0.125, cp=2, pad=-1, cap=30.0, slopes=None, dq=None, dk=None, prefix=None, ws=256,
             wsb=1 << 30, st=16)
    a.update(kw)
    return T.thd_attn_score_fwd(*a.values(), stream=0)


def _bwd(**kw):
    a = dict(q=16, k=16, v=16, o=16, lse=16, do=16, gq=16, gk=16, gv=16, qr=192, kr=192, cq=16, ck=16, pq=None,
             pk=None, B=2, Tq=192, Tk=192, Hq=2, Hkv=2, D=64, causal=1, scale=0.125, cp=2, pad=-1, cap=30.0,
             slopes=None, dq=None, dk=None, prefix=None, ws=256, wsb=1 << 30, st=16)
    a.update(kw)
    return T.thd_attn_score_bwd(*a.values(), stream=0)


@pytest.mark.parametrize("kw", [
    {"q": None}, {"st": None}, {"q": 18}, {"cap": -1.0}, {"cap": float("inf")}, {"cap": float("nan")},
    {"cap": 1e-44}, {"cap": 1.5e11}, {"cap": 1e-14}, {"dq": 16}, {"dk": 16}, {"slopes": 18}, {"dq": 18, "dk": 16}, {"prefix": 17}, {"scale": 0.0},
    {"causal": 3}, {"pad": 2}, {"Hq": 3}, {"cp": 0}])
@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_refuses_bad_arguments(thd_lib, call, kw):
    assert call(**kw) == T.THD_ERR_INVALID_ARG


@pytest.mark.parametrize("call,bwd", [(_fwd, 0), (_bwd, 1)])
def test_refuses_head_sizes_and_small_workspaces(thd_lib, call, bwd):
    assert call(D=96) == T.THD_ERR_UNSUPPORTED
    for docs in (0, 1):
        n = T.thd_score_workspace_size(2, 192, 192, 2, 2, 64, 2, docs, bwd)
        assert n > T.thd_workspace_size(2, 192, 192, 2, 2, 64, 2, bwd)
        extra = {"dq": 16, "dk": 16} if docs else {}
        assert call(wsb=n - 1, **extra) == T.THD_ERR_WORKSPACE
        assert call(ws=8, wsb=n, **extra) == T.THD_ERR_WORKSPACE
    assert T.thd_score_workspace_size(2, 192, 192, 2, 2, 96, 2, 0, bwd) == 0
    assert "document" in T.thd_status_string(T.THD_DEV_ERR_DOC_ORDER)


def test_oracle_against_brute_force():
    """Four queries, four keys, every score by hand."""
    rng = np.random.default_rng(0)
    q, k, v = (rng.standard_normal((4, 1, 8)) for _ in range(3))
    cu = np.array([0, 4])
    doc = np.array([0, 0, 1, 1])
    r = so.score(q, k, v, cu, cu, cu, cu, causal=1, scale=0.5, softcap=2.0, slopes=[0.25], doc_q=doc, doc_k=doc,
                 prefix=[2])
    for i in range(4):
        js = [j for j in range(4) if doc[j] == doc[i] and (j <= i or j < 2)]
        y = [2.0 * np.tanh(0.5 * (q[i, 0] @ k[j, 0]) / 2.0) - 0.25 * abs(i - j) for j in js]
        e = np.exp(y)
        assert np.isclose(r["lse"][0, i], np.log(e.sum()))
        assert np.allclose(r["o"][i, 0], (e[:, None] * v[js, 0]).sum(0) / e.sum())


def test_oracle_gradients_against_differences():
    rng = np.random.default_rng(1)
    q, k, v, do = rng.standard_normal((6, 2, 8)), rng.standard_normal((6, 1, 8)), rng.standard_normal((6, 1, 8)), \
        rng.standard_normal((6, 2, 8))
    cu = np.array([0, 2, 6])
    kw = dict(causal=1, scale=0.4, softcap=1.5, slopes=[0.3, 0.1], prefix=[1, 2])
    r = so.score(q, k, v, cu, cu, cu, cu, do=do, **kw)
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        for at in [tuple(rng.integers(0, s) for s in x.shape) for _ in range(6)]:
            f = []
            for h in (1e-5, -1e-5):
                y = x.copy()
                y[at] += h
                a = {"dq": (y, k, v), "dk": (q, y, v), "dv": (q, k, y)}[name]
                f.append((so.score(*a, cu, cu, cu, cu, **kw)["o"] * do).sum())
            assert abs((f[0] - f[1]) / 2e-5 - r[name][at]) < 1e-7


# ------------------------------------------------------------------ GPU
def _docs(rng, lengths, pads, per):
    """Non-decreasing document numbers inside each sequence; pad rows hold junk."""
    out = np.full(int(pads[-1]), -7, np.int32)
    for b, n in enumerate(lengths):
        cut = np.cumsum(rng.random(n) < 1.0 / per) if n else np.zeros(0)
        out[pads[b]:pads[b] + n] = cut + rng.integers(-2, 2)
    return out


CASES = {
    # name: lengths q, lengths kv (None: the same), pad unit, cp, Hq, Hkv, D, causal, mods
    "cap": ([64, 128], None, 4, 2, 2, 2, 64, 1, {"cap": 5.0}),
    "cap long": ([700, 301, 1], None, 8, 4, 4, 2, 128, 1, {"cap": 20.0}),
    "bias": ([129, 130, 600], None, 16, 1, 4, 1, 128, 1, {"bias": True}),
    "bias all": ([257, 90], None, 12, 3, 2, 1, 64, 0, {"bias": True}),
    "bias bottom right": ([40, 300], [511, 300], 16, 2, 4, 4, 64, 2, {"bias": True}),
    "more queries than keys": ([400, 64], [90, 64], 16, 2, 2, 2, 128, 2, {"bias": True, "cap": 8.0}),
    "docs": ([1000], None, 16, 8, 4, 2, 128, 1, {"docs": 60}),
    "docs all": ([500, 333], None, 8, 2, 2, 2, 64, 0, {"docs": 200, "cap": 10.0}),
    "docs of one": ([200, 3], None, 4, 1, 2, 1, 64, 1, {"docs": 1}),
    "docs bottom right": ([300, 33], [900, 200], 12, 3, 2, 2, 128, 2, {"docs": 90, "bias": True}),
    "prefix": ([520, 260, 130], None, 8, 4, 4, 1, 64, 1, {"prefix": [300, 0, 1000]}),
    "prefix bias": ([400, 17], [400, 200], 8, 2, 2, 2, 128, 2, {"prefix": [-5, 150], "bias": True, "cap": 12.0}),
    "everything": ([900, 0, 77, 384], None, 24, 3, 8, 2, 128, 1,
                   {"cap": 15.0, "bias": True, "docs": 120, "prefix": [200, 3, 30, 384]}),
    "single tokens": ([1, 1, 2, 1], [130, 1, 300, 777], 2, 1, 4, 2, 64, 2, {"cap": 30.0, "bias": True}),
    "many short": ([0, 5, 64, 1, 33, 0, 2, 17] * 8, None, 4, 2, 2, 1, 64, 1, {"cap": 6.0, "docs": 9}),
    # caps past what needs no running maximum (55), scores in every form of tanh
    "large cap": ([300, 513], None, 8, 2, 4, 2, 128, 1, {"cap": 90.0}),
    "large cap bias": ([513, 70], None, 8, 2, 4, 2, 64, 1, {"cap": 70.0, "bias": True, "prefix": [60, 70]}),
    "three forms": ([640], None, 8, 2, 2, 2, 64, 1, {"cap": 10.0, "std": 4.0}),
    "three forms bias": ([640], None, 8, 2, 2, 2, 128, 0, {"cap": 10.0, "std": 4.0, "bias": True}),
    "growing bias": ([300, 200], None, 8, 2, 3, 1, 64, 1, {"cap": 9.0, "slopes": [-0.02, 0.0, 0.3]}),
    "growing bias both sides": ([100, 257], [300, 257], 16, 2, 3, 1, 128, 2,
                                {"cap": 9.0, "slopes": [-0.05, 0.01, -0.3], "docs": 40, "prefix": [90, 100]}),
    "far keys only": ([80, 40], [300, 200], 8, 2, 2, 2, 64, 0, {"cap": 20.0, "slopes": [3.0, 0.5], "docs": 30}),
    # many query heads to a key head: the key tiles are shared among work items
    "no keys": ([900, 64], [0, 64], 8, 2, 32, 1, 64, 2, {"cap": 9.0, "bias": True}),
    "no queries": ([0, 700], [300, 700], 8, 2, 32, 1, 64, 2, {"cap": 9.0, "prefix": [9, 80]}),
    "padded much": ([3, 129, 700], None, 512, 2, 24, 1, 128, 1, {"bias": True, "docs": 300}),
    "mask only": ([300, 200], None, 8, 2, 2, 2, 128, 1, {"prefix": [100, 50]}),
}


def _make(name, std=2.0):
    lq, lk, unit, cp, Hq, Hkv, D, causal, mods = CASES[name]
    std = mods.get("std", std)
    lk = lq if lk is None else lk
    seed = sum(map(ord, name))
    c = inputs.make_cross(lq, lk, pad_to=unit, Hq=Hq, Hkv=Hkv, D=D, cp_size=cp, seed=seed)
    rng = np.random.default_rng(seed)
    c["q"] = (c["q"].float() * std).bfloat16()
    m = {"softcap": mods.get("cap", 0.0), "slopes": None, "doc_q": None, "doc_k": None, "prefix": None}
    if mods.get("bias"):
        m["slopes"] = (2.0 ** (-6.0 * (np.arange(Hq) + 1) / Hq)).astype(np.float32)
    if "slopes" in mods:
        m["slopes"] = np.array(mods["slopes"], np.float32)
    if "docs" in mods:
        m["doc_k"] = _docs(rng, lk, c["cu_kv_pad"], mods["docs"])
        m["doc_q"] = m["doc_k"] if list(lq) == list(lk) else _docs(rng, lq, c["cu_q_pad"], mods["docs"])
    if "prefix" in mods:
        m["prefix"] = np.array(mods["prefix"], np.int32)
    return c, m, cp, causal, 1.0 / np.sqrt(D)


def _gpu(x):
    return None if x is None else torch.from_numpy(x).cuda() if isinstance(x, np.ndarray) else x.cuda()


def _offsets(c):
    return tuple(_gpu(c[n]) for n in ("cu_q", "cu_kv", "cu_q_pad", "cu_kv_pad"))


def _kw(m, cp, causal, scale):
    return {"softcap": m["softcap"], "dist_slopes": _gpu(m["slopes"]), "doc_q": _gpu(m["doc_q"]),
            "doc_kv": _gpu(m["doc_k"]), "prefix_len": _gpu(m["prefix"]), "cp_size": cp, "causal": causal,
            "softmax_scale": scale}


def _ref(c, m, causal, scale):
    n = lambda x: c[x].float().numpy()  # noqa: E731
    return so.score(n("q"), n("k"), n("v"), c["cu_q"], c["cu_kv"], c["cu_q_pad"], c["cu_kv_pad"], causal=causal,
                    scale=scale, do=n("do"), **m)


def _close(name, got, ref):
    g = got.detach().double().cpu().numpy()
    r, tol = ref[name], ref["tol_" + name]
    fin = np.isfinite(r)
    assert np.array_equal(np.isneginf(g), ~fin), f"{name}: rows that see nothing"
    err = np.abs(np.where(fin, g - np.where(fin, r, 0), 0))
    assert np.all(err <= tol), f"{name}: {(err - tol).max():.3e} over its bound of {tol[err > tol].max():.3e}"


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_matches_oracle(thd_lib, name):
    c, m, cp, causal, scale = _make(name)
    ref = _ref(c, m, causal, scale)
    d = {x: _gpu(c[x]) for x in ("q", "k", "v", "do")}
    off, kw = _offsets(c), _kw(m, cp, causal, scale)
    outs = []
    for kernel in KERNELS:
        T.thd_test_select_fwd_kernel(kernel)
        try:
            o, lse, st = T.attn_score_fwd(d["q"], d["k"], d["v"], *off, **kw)
            T.check_status(st)
        finally:
            T.thd_test_select_fwd_kernel(0)
        _close("o", o, ref)
        _close("lse", lse, ref)
        outs.append((o, lse))
    o, lse = outs[0]
    slack = 9
    full = {n: torch.full((d[s].shape[0] + slack, *d[s].shape[1:]), 3.0, dtype=torch.bfloat16, device="cuda")
            for n, s in (("dq", "q"), ("dk", "k"), ("dv", "v"))}
    dq, dk, dv, st = T.attn_score_bwd(d["q"], d["k"], d["v"], o, lse, d["do"], *off, **kw, **full,
                                      dq_rows=full["dq"].shape[0], dkv_rows=full["dk"].shape[0])
    T.check_status(st)
    for n, g in (("dq", dq), ("dk", dk), ("dv", dv)):
        assert not g[-slack:].any(), "slack rows are zero"
        _close(n, g[:-slack], ref)
    again = T.attn_score_bwd(d["q"], d["k"], d["v"], o, lse, d["do"], *off, **kw)
    for a, b in zip(again[:3], (dq, dk, dv)):
        assert torch.equal(a, b[:-slack]), "bit-reproducible"


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [0, 1, 2])
def test_without_modifications_it_is_plain_attention(thd_lib, causal):
    c, _, cp, _, scale = _make("cap long")
    d, off = {x: _gpu(c[x]) for x in ("q", "k", "v", "do")}, _offsets(c)
    a = T.attn_fwd(d["q"], d["k"], d["v"], *off, cp_size=cp, causal=causal, softmax_scale=scale)
    b = T.attn_score_fwd(d["q"], d["k"], d["v"], *off, cp_size=cp, causal=causal, softmax_scale=scale)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga = T.attn_bwd(d["q"], d["k"], d["v"], *a[:2], d["do"], *off, cp_size=cp, causal=causal, softmax_scale=scale)
    gb = T.attn_score_bwd(d["q"], d["k"], d["v"], *a[:2], d["do"], *off, cp_size=cp, causal=causal,
                          softmax_scale=scale)
    assert all(torch.equal(x, y) for x, y in zip(ga[:3], gb[:3]))


@pytest.mark.gpu
def test_the_ring_size_changes_no_bit(thd_lib):
    """Padded lengths every ring size divides: the same outputs and gradients."""
    c, m, _, causal, scale = _make("everything")   # padded to multiples of 24
    d, off = {x: _gpu(c[x]) for x in ("q", "k", "v", "do")}, _offsets(c)
    want = None
    for cp in (1, 2, 3, 4, 6, 12):
        kw = _kw(m, cp, causal, scale)
        o, lse, st = T.attn_score_fwd(d["q"], d["k"], d["v"], *off, **kw)
        T.check_status(st)
        g = T.attn_score_bwd(d["q"], d["k"], d["v"], o, lse, d["do"], *off, **kw)
        T.check_status(g[3])
        want = want or (o, lse, *g[:3])
        assert all(torch.equal(a, b) for a, b in zip(want, (o, lse, *g[:3])))


@pytest.mark.gpu
def test_documents_equal_separate_sequences(thd_lib):
    """Documents inside one sequence give what the same rows give as sequences
    of their own (on lengths that cp_size = 1 can split), bit for bit in dQ's
    inputs: same outputs up to the order of the tiles' sums."""
    lengths = [130, 512, 64, 300, 18]
    n = sum(lengths)
    g = torch.Generator().manual_seed(5)
    q, k, v, do = (torch.randn(n, 4, 64, generator=g).bfloat16().cuda() for _ in range(4))
    one = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    many = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")
    doc = torch.repeat_interleave(torch.arange(5, dtype=torch.int32), torch.tensor(lengths)).cuda()
    o1, l1, st = T.attn_score_fwd(q, k, v, one, one, doc_q=doc, doc_kv=doc, cp_size=4)
    T.check_status(st)
    o2, l2, st = T.attn_fwd(q, k, v, many, many)
    T.check_status(st)
    # O: both within (2^-8 + 2^-8) max|v| of the same number, and each rounded
    assert float((o1.float() - o2.float()).abs().max()) <= 4 * 2.0 ** -8 * float(v.float().abs().max())
    assert float((l1 - l2).abs().max()) <= 2.0 ** -16
    g1 = T.attn_score_bwd(q, k, v, o2, l2, do, one, one, doc_q=doc, doc_kv=doc, cp_size=4)
    g2 = T.attn_bwd(q, k, v, o2, l2, do, many, many)
    for a, b in zip(g1[:3], g2[:3]):
        assert float((a.float() - b.float()).norm()) <= 2.0 ** -7 * float(b.float().norm())


@pytest.mark.gpu
def test_far_positions_keep_their_bias(thd_lib):
    """A long sequence: positions up to 40,000, tiles far from the diagonal,
    a row's bias down to -40,000 x slope.  The nearest keys decide."""
    n, H, D = 40000, 1, 64
    g = torch.Generator().manual_seed(7)
    q, k, v = (torch.randn(n, H, D, generator=g).bfloat16() for _ in range(3))
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    slopes = torch.tensor([0.25], device="cuda")
    o, lse, st = T.attn_score_fwd(q.cuda(), k.cuda(), v.cuda(), cu, cu, dist_slopes=slopes, softcap=10.0, cp_size=4)
    T.check_status(st)
    for i in (0, 1, 127, 128, 20000, 39999):
        lo = max(0, i - 2000)    # e^(-500 + 20) of the rest: nothing
        r = so.score(q[i:i + 1].float().numpy(), k[lo:i + 1].float().numpy(), v[lo:i + 1].float().numpy(),
                     *(np.array([0, x]) for x in (1, i + 1 - lo, 1, i + 1 - lo)), causal=2, scale=D ** -0.5,
                     softcap=10.0, slopes=[0.25])
        assert np.all(np.abs(o[i].double().cpu().numpy() - r["o"][0]) <= r["tol_o"][0])
        assert np.all(np.abs(lse[:, i].double().cpu().numpy() - r["lse"][:, 0]) <= r["tol_lse"][:, 0])


@pytest.mark.gpu
def test_saturated_scores(thd_lib):
    """Scores of thousands: the cap holds them, tanh is 1, its derivative 0."""
    c, m, cp, causal, scale = _make("cap", std=500.0)
    ref = _ref(c, m, causal, scale)
    d, off, kw = {x: _gpu(c[x]) for x in ("q", "k", "v", "do")}, _offsets(c), _kw(m, cp, causal, scale)
    o, lse, st = T.attn_score_fwd(d["q"], d["k"], d["v"], *off, **kw)
    T.check_status(st)
    _close("o", o, ref)
    _close("lse", lse, ref)
    grads = T.attn_score_bwd(d["q"], d["k"], d["v"], o, lse, d["do"], *off, **kw)
    T.check_status(grads[3])
    for n, g in zip(("dq", "dk", "dv"), grads):
        _close(n, g, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [3.0e6, 1.0e9])
@pytest.mark.parametrize("kernel", KERNELS)
def test_a_cap_far_above_the_scores_changes_nothing(thd_lib, kernel, cap):
    """|x| / cap is below 1e-4: tanh departs from its argument by 1e-9 of it,
    and its polynomial's first coefficient by 7.8e-7 -- inside the uncapped
    bounds, whose D 2^-24 sum |q||k| is at least 3.8e-6 |x|."""
    c, m, cp, causal, scale = _make("cap")
    ref = _ref(c, {**m, "softcap": 0.0}, causal, scale)
    d, off, kw = {x: _gpu(c[x]) for x in ("q", "k", "v", "do")}, _offsets(c), _kw(m, cp, causal, scale)
    kw["softcap"] = cap
    T.thd_test_select_fwd_kernel(kernel)
    try:
        o, lse, st = T.attn_score_fwd(d["q"], d["k"], d["v"], *off, **kw)
        T.check_status(st)
    finally:
        T.thd_test_select_fwd_kernel(0)
    _close("o", o, ref)
    _close("lse", lse, ref)
    grads = T.attn_score_bwd(d["q"], d["k"], d["v"], o, lse, d["do"], *off, **kw)
    T.check_status(grads[3])
    for n, g in zip(("dq", "dk", "dv"), grads):
        _close(n, g, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", KERNELS)
def test_a_tiny_cap_and_queries_of_zero(thd_lib, kernel):
    """Coefficients past fp32 are not used, not even against scores of 0."""
    c, m, cp, causal, scale = _make("cap")
    m["softcap"] = 1e-9
    c["q"][::2] = 0
    ref = _ref(c, m, causal, scale)
    d, off, kw = {x: _gpu(c[x]) for x in ("q", "k", "v", "do")}, _offsets(c), _kw(m, cp, causal, scale)
    T.thd_test_select_fwd_kernel(kernel)
    try:
        o, lse, st = T.attn_score_fwd(d["q"], d["k"], d["v"], *off, **kw)
        T.check_status(st)
    finally:
        T.thd_test_select_fwd_kernel(0)
    _close("o", o, ref)
    _close("lse", lse, ref)
    d["q"].zero_()
    grads = T.attn_score_bwd(d["q"], d["k"], d["v"], o, lse, d["do"], *off, **kw)
    assert all(torch.isfinite(g.float()).all() for g in grads[:3])


@pytest.mark.gpu
@pytest.mark.parametrize("std", [0.1, 1.0, 100.0])
@pytest.mark.parametrize("kernel", KERNELS)
def test_a_nan_key_shows_in_the_rows_that_see_it(thd_lib, kernel, std):
    """In every form of tanh; rows before it and other heads' keys keep their
    numbers.  (A NaN on a row with a valid token is the caller's; it must not
    turn into plausible numbers.)"""
    c, m, cp, causal, scale = _make("cap", std=std)
    d, off, kw = {x: _gpu(c[x]) for x in ("q", "k", "v", "do")}, _offsets(c), _kw(m, cp, causal, scale)
    want, _, _ = T.attn_score_fwd(d["q"], d["k"], d["v"], *off, **kw)
    at = 70  # a position of the second sequence
    row = int(c["cu_kv_pad"][1]) + at
    d["k"][row, 0, 5] = float("nan")
    T.thd_test_select_fwd_kernel(kernel)
    try:
        o, lse, st = T.attn_score_fwd(d["q"], d["k"], d["v"], *off, **kw)
        T.check_status(st)
    finally:
        T.thd_test_select_fwd_kernel(0)
    see = slice(row, int(c["cu_q_pad"][1]) + 128)
    assert torch.isnan(o[see, 0].float()).all()
    other = o.clone()
    other[see, 0] = 0
    assert torch.isfinite(other.float()).all()
    assert float((other[:, 1].float() - want[:, 1].float()).abs().max()) <= 4 * 2.0 ** -8 * float(d["v"].float().abs().max())


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", KERNELS)
def test_decreasing_documents_are_refused_on_the_device(thd_lib, kernel):
    """Status 108, outputs untouched; numbers may fall between sequences and on
    pad rows; the same workspace then serves a valid call."""
    c, m, cp, causal, scale = _make("docs all")
    d, off, kw = {x: _gpu(c[x]) for x in ("q", "k", "v", "do")}, _offsets(c), _kw(m, cp, causal, scale)
    bad = m["doc_k"].copy()
    bad[77] = bad[76] - 1
    ws = torch.empty(T.thd_score_workspace_size(2, *[d[x].shape[0] for x in ("q", "k")], 2, 2, 64, cp, 1, 1),
                     dtype=torch.uint8, device="cuda")
    T.thd_test_select_fwd_kernel(kernel)
    try:
        for side in ("doc_q", "doc_kv"):
            o = torch.full_like(d["q"], 5.0)
            _, _, st = T.attn_score_fwd(d["q"], d["k"], d["v"], *off, **{**kw, side: _gpu(bad)}, out=o, workspace=ws)
            assert int(st.item()) == T.THD_DEV_ERR_DOC_ORDER and bool((o == 5.0).all())
            dq = torch.full_like(d["q"], 5.0)
            o2, l2, _ = T.attn_score_fwd(d["q"], d["k"], d["v"], *off, **kw)
            r = T.attn_score_bwd(d["q"], d["k"], d["v"], o2, l2, d["do"], *off, **{**kw, side: _gpu(bad)}, dq=dq,
                                 workspace=ws)
            assert int(r[3].item()) == T.THD_DEV_ERR_DOC_ORDER and bool((dq == 5.0).all())
        o3, l3, st = T.attn_score_fwd(d["q"], d["k"], d["v"], *off, **kw, workspace=ws)
        T.check_status(st)
        assert torch.equal(o3, o2) and torch.equal(l3, l2)
        # invalid offsets with documents: reported, nothing read through them
        cu = off[0].clone()
        cu[1] = -4
        _, _, st = T.attn_score_fwd(d["q"], d["k"], d["v"], cu, *off[1:], **kw, workspace=ws)
        assert int(st.item()) == T.THD_DEV_ERR_NOT_MONOTONE
    finally:
        T.thd_test_select_fwd_kernel(0)


@pytest.mark.gpu
def test_captured_in_a_graph(thd_lib):
    """Forward and backward captured once and replayed on new inputs, new
    documents, prefixes and slopes; an eager call in between."""
    c, m, cp, causal, scale = _make("everything")
    d, off, kw = {x: _gpu(c[x]) for x in ("q", "k", "v", "do")}, _offsets(c), _kw(m, cp, causal, scale)

    def step():
        o, lse, s1 = T.attn_score_fwd(d["q"], d["k"], d["v"], *off, **kw)
        return (o, lse, *T.attn_score_bwd(d["q"], d["k"], d["v"], o, lse, d["do"], *off, **kw), s1)

    step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = step()
    for _ in range(2):
        d["q"].mul_(-0.5)
        d["v"].add_(0.25)
        kw["doc_q"].floor_divide_(2)
        if kw["doc_kv"] is not kw["doc_q"]:
            kw["doc_kv"].floor_divide_(2)
        kw["prefix_len"].add_(7)
        kw["dist_slopes"].mul_(0.5)
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert int(out[5].item()) == 0 and int(out[6].item()) == 0
        for a, b in zip(out[:5], want[:5]):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_two_streams_at_once(thd_lib):
    """Two calls in flight with workspaces of their own."""
    c, m, cp, causal, scale = _make("everything")
    d, off, kw = {x: _gpu(c[x]) for x in ("q", "k", "v", "do")}, _offsets(c), _kw(m, cp, causal, scale)
    want = T.attn_score_fwd(d["q"], d["k"], d["v"], *off, **kw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append([T.attn_score_fwd(d["q"], d["k"], d["v"], *off, **kw) for _ in range(4)])
    torch.cuda.synchronize()
    for runs in got:
        for o, lse, st in runs:
            assert int(st.item()) == 0 and torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("fwd,kernel", [(KERNELS[0], T.THD_KERNEL_FWD), (KERNELS[1], T.THD_KERNEL_FWD),
                                        (KERNELS[0], T.THD_KERNEL_BWD_DQ), (KERNELS[0], T.THD_KERNEL_BWD)])
@pytest.mark.parametrize("cap", [0.0, 9.0])
def test_waits_end(thd_lib, cap, fwd, kernel):
    """The bounded wait of the scored kernels (their block sizes differ with a
    cap) runs out, the call reports it, its outputs stay as they were, and the
    next call is right."""
    c, m, cp, causal, scale = _make("bias all")
    m["softcap"] = cap
    d, off, kw = {x: _gpu(c[x]) for x in ("q", "k", "v", "do")}, _offsets(c), _kw(m, cp, causal, scale)
    T.thd_test_select_fwd_kernel(fwd)
    try:
        o, lse, _ = T.attn_score_fwd(d["q"], d["k"], d["v"], *off, **kw)
        outs = [torch.full_like(d[x], 7.0) for x in ("q", "k", "v")]
        assert T.thd_test_arm_stall(kernel) == T.THD_OK
        if kernel == T.THD_KERNEL_FWD:
            _, _, st = T.attn_score_fwd(d["q"], d["k"], d["v"], *off, **kw, out=outs[0])
            assert torch.all(outs[0] == 7.0)
        else:
            g = dict(zip(("dq", "dk", "dv"), outs))
            st = T.attn_score_bwd(d["q"], d["k"], d["v"], o, lse, d["do"], *off, **kw, **g)[3]
            assert torch.all(outs[1] == 7.0) and torch.all(outs[2] == 7.0)
            assert bool(torch.all(outs[0] == 7.0)) == (kernel == T.THD_KERNEL_BWD_DQ)
        assert int(st.item()) == T.THD_ERR_TIMEOUT
        o2, lse2, st = T.attn_score_fwd(d["q"], d["k"], d["v"], *off, **kw)
        T.check_status(st)
        assert torch.equal(o2, o) and torch.equal(lse2, lse)
    finally:
        T.thd_test_arm_stall(0)
        T.thd_test_select_fwd_kernel(0)


@pytest.mark.gpu
def test_elements_past_32_bits(thd_lib):
    """614,400 rows of 32 heads of 128, 2.5e9 elements: the last sequence, in a
    batch of 1200, gives what it gives alone, bit for bit (the forward kernel
    named, since the choice goes by the whole batch)."""
    B, L, Hq, Hkv, D = 1200, 512, 32, 2, 128
    n = B * L
    g = torch.Generator().manual_seed(3)
    kw = {"softcap": 30.0, "cp_size": 2, "dist_slopes": torch.full((Hq,), 0.01, device="cuda")}
    docs = torch.zeros(n, dtype=torch.int32, device="cuda")
    docs[-200:] = 1
    cu = torch.arange(0, n + 1, L, dtype=torch.int32, device="cuda")
    one = torch.tensor([0, L], dtype=torch.int32, device="cuda")
    last = {x: torch.randn(L, h, D, generator=g).bfloat16().cuda()
            for x, h in (("q", Hq), ("k", Hkv), ("v", Hkv), ("do", Hq))}
    d = {x: torch.zeros(n, *t.shape[1:], dtype=torch.bfloat16, device="cuda") for x, t in last.items()}
    for x, t in last.items():
        d[x][-L:] = t
    T.thd_test_select_fwd_kernel(T.THD_FWD_KERNEL_DUAL)
    try:
        o1, l1, st = T.attn_score_fwd(*(last[x] for x in "qkv"), one, one, doc_q=docs[-L:], doc_kv=docs[-L:], **kw)
        T.check_status(st)
        o, lse, st = T.attn_score_fwd(*(d[x] for x in "qkv"), cu, cu, doc_q=docs, doc_kv=docs, **kw)
        T.check_status(st)
    finally:
        T.thd_test_select_fwd_kernel(0)
    assert torch.equal(o[-L:], o1) and torch.equal(lse[:, -L:], l1)
    g1 = T.attn_score_bwd(*(last[x] for x in "qkv"), o1, l1, last["do"], one, one, doc_q=docs[-L:],
                          doc_kv=docs[-L:], **kw)
    ga = T.attn_score_bwd(*(d[x] for x in "qkv"), o, lse, d["do"], cu, cu, doc_q=docs, doc_kv=docs, **kw)
    T.check_status(ga[3])
    assert torch.equal(ga[0][-L:], g1[0])
    # dK, dV: a key tile's walk may be shared among work items when there are few of them, so the fp32 sums differ in
    # order (64 x 2^-24 of the terms) and each is rounded to bf16 (2^-8)
    for a, b in zip(ga[1:3], g1[1:3]):
        assert float((a[-L:].float() - b.float()).norm()) <= (2 * 2.0 ** -8 + 2.0 ** -14) * float(b.float().norm())


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,lengths", [(8, 1, 64, [2100, 900]), (4, 1, 128, [4000, 60]), (1, 1, 64, [4133])])
def test_shared_key_tiles(thd_lib, Hq, Hkv, D, lengths):
    """Few key tiles, each walked by several work items: the gradients, every
    score modification on, against the oracle; repeats are bit-identical; rows
    past the last sequence are zero."""
    c = inputs.make_cross(lengths, lengths, pad_to=8, Hq=Hq, Hkv=Hkv, D=D, cp_size=4, seed=9)
    rng = np.random.default_rng(10)
    m = {"softcap": 20.0, "slopes": (2.0 ** -(np.arange(Hq) + 3.0)).astype(np.float32), "prefix": None,
         "doc_k": _docs(rng, lengths, c["cu_kv_pad"], 1500)}
    m["doc_q"] = m["doc_k"]
    scale = D ** -0.5
    ref = _ref(c, m, 1, scale)
    d = {x: _gpu(c[x]) for x in ("q", "k", "v", "do")}
    off, kw = _offsets(c), _kw(m, 4, 1, scale)
    o, lse, st = T.attn_score_fwd(d["q"], d["k"], d["v"], *off, **kw)
    T.check_status(st)
    T.thd_profile_enable(T.THD_KERNEL_BWD_JOIN, 4)
    runs = [T.attn_score_bwd(d["q"], d["k"], d["v"], o, lse, d["do"], *off, **kw, dkv_rows=d["k"].shape[0] + 5)
            for _ in range(2)]
    assert len(T.thd_profile_read()) == 2
    T.thd_profile_enable(0, 0)
    for n, a, b in zip(("dq", "dk", "dv"), *runs):
        assert torch.equal(a, b)
        _close(n, a[:d["q" if n == "dq" else "k"].shape[0]], ref)
        if n != "dq":
            assert not a[-5:].any()
    # a workspace short of the shared tiles' room: shared less, or not at all
    t = d["q"].shape[0]
    for n in (T.thd_score_workspace_size(len(lengths), t, t, Hq, Hkv, D, 4, 1, 1) - 256, 300000):
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        less = T.attn_score_bwd(d["q"], d["k"], d["v"], o, lse, d["do"], *off, **kw, workspace=ws)
        T.check_status(less[3])
        for x, g in zip(("dq", "dk", "dv"), less):
            _close(x, g, ref)


@pytest.mark.gpu
def test_backwards_on_two_streams_and_in_a_graph(thd_lib):
    """Shared key tiles: two backward calls in flight, and a captured one, give
    what one alone gives; a refused batch leaves the gradients as they were."""
    c, m, cp, causal, scale = _make("padded much")
    d, off, kw = {x: _gpu(c[x]) for x in ("q", "k", "v", "do")}, _offsets(c), _kw(m, cp, causal, scale)
    o, lse, st = T.attn_score_fwd(d["q"], d["k"], d["v"], *off, **kw)
    T.check_status(st)
    call = lambda **more: T.attn_score_bwd(d["q"], d["k"], d["v"], o, lse, d["do"], *off, **{**kw, **more})  # noqa: E731
    T.thd_profile_enable(T.THD_KERNEL_BWD_JOIN, 4)
    want = call()
    assert len(T.thd_profile_read()) == 1
    T.thd_profile_enable(0, 0)
    torch.cuda.synchronize()
    got = []
    for s in [torch.cuda.Stream() for _ in range(2)]:
        with torch.cuda.stream(s):
            got += [call() for _ in range(3)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got.append(call())
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for g in got:
        assert int(g[3].item()) == 0 and all(torch.equal(a, b) for a, b in zip(g[:3], want[:3]))
    bad = kw["doc_q"].clone()
    bad[int(c["cu_q_pad"][2]) + 5] = -99
    outs = {x: torch.full_like(d[y], 7.0) for x, y in (("dq", "q"), ("dk", "k"), ("dv", "v"))}
    st = call(doc_q=bad, **outs)[3]
    assert int(st.item()) == T.THD_DEV_ERR_DOC_ORDER and all(torch.all(x == 7.0) for x in outs.values())


@pytest.mark.gpu
def test_helper_refuses_wrong_tensors(thd_lib):
    c, m, cp, causal, scale = _make("everything")
    d, off, kw = {x: _gpu(c[x]) for x in ("q", "k", "v", "do")}, _offsets(c), _kw(m, cp, causal, scale)
    before = T.thd_launch_count()
    for bad in ({"doc_q": kw["doc_q"].long()}, {"doc_q": kw["doc_q"][:-1]}, {"doc_kv": None},
                {"dist_slopes": kw["dist_slopes"].double()}, {"dist_slopes": kw["dist_slopes"][:2]},
                {"prefix_len": kw["prefix_len"][:2]}, {"prefix_len": kw["prefix_len"].cpu()},
                {"softcap": -1.0}, {"out": d["q"].float()}, {"causal": 5},
                {"workspace": torch.empty(1 << 24, dtype=torch.uint8)}):
        with pytest.raises(T.ThdError):
            T.attn_score_fwd(d["q"], d["k"], d["v"], *off, **{**kw, **bad})
    for q, k, v in ((d["q"].float(), d["k"], d["v"]), (d["q"], d["k"][:-1], d["v"]),
                    (d["q"].transpose(0, 1), d["k"], d["v"]), (d["q"].cpu(), d["k"], d["v"])):
        with pytest.raises(T.ThdError):
            T.attn_score_fwd(q, k, v, *off, **kw)
    assert T.thd_launch_count() == before


# ------------------------------------------------------------------ the run of operators as a training step uses them
@pytest.mark.gpu
def test_rope_attention_dropout_together(thd_lib):
    """q and k turned out of a fused projection, attended with a cap and
    documents, dropped out onto the residual; then the gradients all the way
    back into the fused projection's gradient, against fp64 on the same
    roundings (each operator's inputs are the library's own bf16 outputs, so
    each step is held to its own bound)."""
    from oracle import row_ops
    n, Hq, Hkv, D, cp = 600, 4, 2, 64, 4
    rng = np.random.default_rng(21)
    width = (Hq + 2 * Hkv) * D
    qkv = torch.from_numpy(rng.standard_normal((n, width))).bfloat16().cuda()
    res = torch.from_numpy(rng.standard_normal((n, Hq * D))).bfloat16().cuda()
    dout = torch.from_numpy(rng.standard_normal((n, Hq * D))).bfloat16().cuda()
    cut = lambda t: (t[:, :Hq * D].unflatten(1, (Hq, D)), t[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D)),  # noqa: E731
                     t[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D)))
    q0, k0, v0 = cut(qkv)
    v = v0.contiguous()
    inv, axis = 1e4 ** (-np.arange(32) / 32), np.repeat([0, 1, 2], [8, 12, 12]).astype(np.uint8)
    pos = torch.from_numpy(rng.integers(0, 600, (3, n)).astype(np.int32)).cuda()
    cu = torch.tensor([0, 248, n], dtype=torch.int32, device="cuda")
    doc = torch.from_numpy((np.arange(n) // 100).astype(np.int32)).cuda()
    state = torch.tensor([77, 5], dtype=torch.int64, device="cuda")
    kw = dict(softcap=20.0, doc_q=doc, doc_kv=doc, cp_size=cp)

    q, k = T.rope(q0, k0, pos, inv, axis)
    o, lse, s1 = T.attn_score_fwd(q, k, v, cu, cu, **kw)
    y = T.dropout_add(o.view(n, Hq * D), state, 0.1, residual=res)
    do = T.dropout_add(dout, state, 0.1).view(n, Hq, D)
    dqkv = torch.empty_like(qkv)
    dq0, dk0, dv0 = cut(dqkv)
    dq, dk, dv, s2 = T.attn_score_bwd(q, k, v, o, lse, do, cu, cu, **kw)
    T.rope(dq, dk, pos, inv, axis, inverse=True, q_out=dq0, k_out=dk0)
    dv0.copy_(dv)
    T.check_status(s1)
    T.check_status(s2)

    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    cun = cu.cpu().numpy()
    ref = so.score(f(q), f(k), f(v), cun, cun, cun, cun, causal=1, scale=D ** -0.5, softcap=20.0, doc_q=f(doc),
                   doc_k=f(doc), do=f(do))
    for name, g in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        _close(name, g, ref)
    for got, x, sign in ((q, q0, False), (k, k0, False), (dq0, dq, True), (dk0, dk, True)):
        r = row_ops.rope(f(x), pos.cpu().numpy(), inv, axis, inverse=sign)
        assert np.all(np.abs(f(got) - r) <= 2.0 ** -8 * np.abs(r) + 2.0 ** -18 * np.abs(f(x)).max())
    r, _ = row_ops.dropout_add(f(o).reshape(n, -1), f(res), np.arange(n), 0.1, 77, 5)
    assert np.all(np.abs(f(y) - r) <= 2.0 ** -8 * np.abs(r) + 2.0 ** -22 * (np.abs(f(o)).max() + 1))
    r, _ = row_ops.dropout_add(f(dout), None, np.arange(n), 0.1, 77, 5)
    assert np.all(np.abs(f(do).reshape(n, -1) - r) <= 2.0 ** -8 * np.abs(r) * (1 + 2.0 ** -10))
