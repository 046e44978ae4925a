"""Rotary positions with several axes (thd_rope): the refusals on the CPU, and
on the GPU parity with the fp64 oracle over head sizes, rotated sizes, both
pairings, both types, row strides (slices of a fused projection), alignments,
far and negative positions; the backward against the formula and against
differences; in place; captured in a graph.

Tolerance, per element with inputs (a, b) of its pair: the angle's rounding to
a 24-bit float of half turns and to 2^-24 turns (pi 2^-24 + 2 pi 2^-24), two
units in the last place of sine and cosine (2^-22) and three fp32 roundings:
below 2^-19 (|a| + |b|); then the rounding of the result, 2^-8 |y| in bf16."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import row_ops
from packed_sequence_context_gb300 import thd_attn as T


def _table(rot, parts, weave=False):
    half = rot // 2
    inv = 10000.0 ** (-np.arange(half) / half)
    if weave:
        axis = np.array([i % len(parts) for i in range(half)], np.uint8)
    else:
        axis = np.repeat(np.arange(len(parts)), parts).astype(np.uint8)
    return inv, axis


def _check(got, x, pos, inv, axis, dtype, **kw):
    x64 = x.detach().double().cpu().numpy()
    ref = row_ops.rope(x64, pos.cpu().numpy(), inv, axis, **kw)
    half = len(inv)
    mag = np.zeros_like(ref)
    for i in range(half):
        ia, ib = (2 * i, 2 * i + 1) if kw.get("adjacent") else (i, half + i)
        mag[:, :, ia] = mag[:, :, ib] = np.abs(x64[:, :, ia]) + np.abs(x64[:, :, ib])
    tol = 2.0 ** -19 * mag + (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24) * np.abs(ref)
    err = np.abs(got.detach().double().cpu().numpy() - ref)
    assert np.all(err <= tol), f"max excess {(err - tol).max():.3e}"


# ------------------------------------------------------------------ refusals (no GPU)
def _call(**kw):
    inv = (ctypes.c_double * 64)(*([0.5] * 64))
    axis = (ctypes.c_uint8 * 64)(*([0] * 64))
    a = dict(q_in=16, k_in=16, q_out=32, k_out=32, qs=256, ks=256, qos=256, kos=256, T=4, Hq=2, Hkv=2, D=128, rot=128,
             pos=16, n_axes=1, inv=ctypes.addressof(inv), axis=ctypes.addressof(axis), adjacent=0, inverse=0, dtype=0)
    tables = {"bad_inv": (ctypes.c_double * 64)(*([float("inf")] * 64)), "bad_axis": (ctypes.c_uint8 * 64)(*([3] * 64))}
    for k in list(kw):
        if k in tables:
            a["inv" if k == "bad_inv" else "axis"] = ctypes.addressof(tables[k])
            del kw[k]
    a.update(kw)
    return T.thd_rope(*a.values(), stream=0)


@pytest.mark.parametrize("kw", [
    {"q_in": None}, {"k_out": None}, {"pos": None}, {"pos": 18}, {"q_in": 17}, {"T": -1}, {"T": 1 << 31}, {"Hq": -1},
    {"Hq": 0, "Hkv": 0}, {"rot": 0}, {"rot": 63}, {"rot": 130}, {"n_axes": 0}, {"qs": 255}, {"kos": 128},
    {"q_out": 16, "qos": 512}, {"bad_inv": 1}, {"bad_axis": 1}, {"inv": None}, {"axis": None},
    {"dtype": 1, "q_in": 18}, {"Hq": (1 << 20) + 1, "qs": 1 << 30, "qos": 1 << 30}])
def test_refuses_bad_arguments(thd_lib, kw):
    assert _call(**kw) == T.THD_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [{"dtype": 2}, {"D": 1025, "rot": 64}, {"D": 0}, {"n_axes": 17},
                                {"D": 512, "rot": 258, "qs": 1024, "ks": 1024, "qos": 1024, "kos": 1024}])
def test_refuses_unsupported(thd_lib, kw):
    assert _call(**kw) == T.THD_ERR_UNSUPPORTED


def test_no_rows_is_no_launch(thd_lib):
    before = T.thd_launch_count()
    assert _call(T=0, q_in=None, k_in=None, q_out=None, k_out=None, pos=None) == T.THD_OK
    assert T.thd_launch_count() == before


def test_oracle_turns_a_known_pair():
    x = np.zeros((1, 1, 4))
    x[0, 0] = [1.0, 2.0, 3.0, 4.0]
    y = row_ops.rope(x, np.array([[1], [2]]), [np.pi / 2, np.pi / 2], [0, 1])
    assert np.allclose(y[0, 0], [-3.0, -2.0, 1.0, -4.0], atol=1e-12)
    y = row_ops.rope(x, np.array([[1], [2]]), [np.pi / 2, np.pi / 2], [0, 1], adjacent=True)
    assert np.allclose(y[0, 0], [-2.0, 1.0, -3.0, -4.0], atol=1e-12)


# ------------------------------------------------------------------ GPU
def _pos(rng, n, rows, far):
    return torch.from_numpy(rng.integers(-far, far, size=(n, rows), endpoint=True).astype(np.int32)).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("rows,Hq,Hkv,D,rot,parts", [
    (1, 1, 1, 64, 64, [32]), (7, 32, 8, 128, 128, [16, 24, 24]), (301, 3, 1, 64, 32, [8, 8]),
    (65, 5, 5, 128, 48, [4, 10, 10]), (33, 2, 2, 80, 80, [40]), (19, 4, 2, 66, 20, [3, 7]), (13, 1, 1, 5, 4, [1, 1]),
    (40, 16, 0, 256, 256, [64, 64]), (9, 2, 1, 1024, 16, [8]), (130, 1, 0, 16, 16, [2, 2, 2, 2]), (5, 70, 1, 8, 8, [4])])
def test_matches_oracle(thd_lib, dtype, adjacent, rows, Hq, Hkv, D, rot, parts):
    rng = np.random.default_rng(rows * 1000 + D)
    inv, axis = _table(rot, parts)
    pos = _pos(rng, len(parts), rows, 5000)
    q = torch.from_numpy(rng.standard_normal((rows, Hq, D))).to(dtype).cuda()
    k = torch.from_numpy(rng.standard_normal((rows, Hkv, D))).to(dtype).cuda() if Hkv else None
    for inverse in (False, True):
        qo, ko = T.rope(q, k, pos, inv, axis, adjacent=adjacent, inverse=inverse)
        torch.cuda.synchronize()
        _check(qo, q, pos, inv, axis, dtype, adjacent=adjacent, inverse=inverse)
        if Hkv:
            _check(ko, k, pos, inv, axis, dtype, adjacent=adjacent, inverse=inverse)


@pytest.mark.gpu
def test_far_and_negative_positions(thd_lib):
    """Exact reduction at any 32-bit position.  The fp64 oracle's own angle is
    off by up to 2^30 2^-53, far below the tolerance."""
    inv, axis = _table(128, [32, 32], weave=True)
    edge = [0, 1, -1, 131071, 1 << 20, (1 << 30) - 1, -(1 << 30)]
    pos = torch.tensor([edge, edge[::-1]], dtype=torch.int32, device="cuda")
    q = torch.randn(len(edge), 2, 128, device="cuda")
    qo, _ = T.rope(q, None, pos, inv, axis)
    torch.cuda.synchronize()
    _check(qo, q, pos, inv, axis, torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shift", [0, 1])
def test_slices_of_a_fused_projection_in_and_out(thd_lib, dtype, shift):
    """q and k read from one [T, (Hq + 2 Hkv) D] buffer and their gradients
    written into another; shift = 1 puts every row off the 16-byte grid.  The
    bytes between are left alone."""
    rows, Hq, Hkv, D = 77, 4, 2, 64
    width = (Hq + 2 * Hkv) * D + shift
    inv, axis = _table(D, [8, 12, 12])
    rng = np.random.default_rng(3)
    pos = _pos(rng, 3, rows, 1000)
    buf = torch.from_numpy(rng.standard_normal((rows, width))).to(dtype).cuda()
    out = torch.full_like(buf, 7.0)
    cut = lambda t: (t[:, shift:shift + Hq * D].unflatten(1, (Hq, D)),  # noqa: E731
                     t[:, shift + Hq * D:shift + (Hq + Hkv) * D].unflatten(1, (Hkv, D)))
    (q, k), (qo, ko) = cut(buf), cut(out)
    T.rope(q, k, pos, inv, axis, q_out=qo, k_out=ko)
    torch.cuda.synchronize()
    _check(qo, q, pos, inv, axis, dtype)
    _check(ko, k, pos, inv, axis, dtype)
    assert bool((out[:, shift + (Hq + Hkv) * D:] == 7.0).all()) and bool((out[:, :shift] == 7.0).all())
    # in place, through the same slices: the same bits
    T.rope(q, k, pos, inv, axis, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.gpu
def test_backward_is_the_gradient(thd_lib):
    """<rope(x), g> = <x, rope^-1(g)> (the formula), and against differences
    of a step h in fp32: the map is linear, so a difference is exact up to the
    rounding 2^-22 |y| / h of its two evaluations."""
    rows, H, D = 12, 2, 64
    inv, axis = _table(D, [10, 11, 11])
    rng = np.random.default_rng(9)
    pos = _pos(rng, 3, rows, 300)
    x, g = torch.randn(rows, H, D, device="cuda"), torch.randn(rows, H, D, device="cuda")
    y, _ = T.rope(x, None, pos, inv, axis)
    gx, _ = T.rope(g, None, pos, inv, axis, inverse=True)
    lhs, rhs = (y.double() * g.double()).sum(), (x.double() * gx.double()).sum()
    assert abs(float(lhs - rhs)) <= 2.0 ** -18 * float((x.double().abs() * 2 * g.double().abs().max()).sum())
    h = 0.5
    for t, hd, e in ((0, 0, 0), (3, 1, 31), (11, 0, 32), (5, 1, 63)):
        d = torch.zeros_like(x)
        d[t, hd, e] = h
        diff = (T.rope(x + d, None, pos, inv, axis)[0].double() - T.rope(x - d, None, pos, inv, axis)[0].double())
        num = float((diff * g.double()).sum()) / (2 * h)
        assert abs(num - float(gx[t, hd, e])) <= 2.0 ** -16 * 4 * float(g.abs().max())


@pytest.mark.gpu
def test_captured_in_a_graph_on_another_stream(thd_lib):
    inv, axis = _table(128, [16, 24, 24])
    rng = np.random.default_rng(4)
    pos = _pos(rng, 3, 50, 100)
    q, k = torch.randn(50, 4, 128, device="cuda").bfloat16(), torch.randn(50, 2, 128, device="cuda").bfloat16()
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        T.rope(q, k, pos, inv, axis, q_out=qo, k_out=ko)
    for step in (1, 2):
        pos += step
        q.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        _check(qo, q, pos, inv, axis, torch.bfloat16)
        _check(ko, k, pos, inv, axis, torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("D,rot", [(128, 128), (125, 62)])
def test_elements_past_32_bits(thd_lib, D, rot):
    """700,001 rows of 32 heads, in place: the last rows are what they are alone."""
    rows, H, n = 700001, 32, 5
    freq = 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    q = torch.zeros(rows, H, D, dtype=torch.bfloat16, device="cuda")
    q[-n:] = torch.randn(n, H, D, device="cuda").bfloat16()
    want, _ = T.rope(q[-n:].clone(), None, pos[-n:].clone(), freq)
    T.rope(q, None, pos, freq, q_out=q)
    assert torch.equal(q[-n:], want) and not q[:-n].any()


@pytest.mark.gpu
def test_helper_refuses_wrong_tensors(thd_lib):
    inv, axis = _table(64, [32])
    q = torch.zeros(4, 2, 64, device="cuda", dtype=torch.bfloat16)
    pos = torch.zeros(1, 4, device="cuda", dtype=torch.int32)
    bad = [(q, q[:3], pos, {}), (q, q.float(), pos, {}), (q, None, pos.long(), {}), (q, None, pos[:, :3], {}),
           (q, None, pos.cpu(), {}), (q.transpose(1, 2), None, pos, {}), (q, None, pos, {"q_out": q[:, :1]}),
           (q.cpu(), None, pos, {}), (q[..., ::2], None, pos, {})]
    before = T.thd_launch_count()
    for a, b, c, kw in bad:
        with pytest.raises(T.ThdError):
            T.rope(a, b, c, inv, axis, **kw)
    with pytest.raises(T.ThdError) as e:
        T.rope(q.half(), None, pos, inv, axis)
    assert e.value.code == T.THD_ERR_UNSUPPORTED
    assert T.thd_launch_count() == before
    qo, ko = T.rope(q[:0], q[:0], pos[:, :0].contiguous(), inv, axis)   # no rows
    assert qo.shape == (0, 2, 64) and T.thd_launch_count() == before
