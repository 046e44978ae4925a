"""Dropout from a counter-based generator plus the residual
(thd_dropout_add): published answers of the generator and the refusals on the
CPU, and on the GPU masks equal to the oracle's bit for bit, over shapes on and
off the 16-byte grid, types, row numbers, probabilities; a rank's shard draws
what the unsplit buffer draws; backward; infinities and NaN in dropped places;
a captured graph whose state advances.

Tolerance: x / (1 - p) and the sum are one fp32 rounding each (2^-24 of |x| s
and of the result, s = 1 / (1 - p), itself rounded to 2^-24), then the result's
own rounding: 2^-8 |y| in bf16, counted in fp32 already."""

import numpy as np
import pytest
import torch

from oracle import row_ops
from packed_sequence_context_gb300 import thd_attn as T


# ------------------------------------------------------------------ the generator (no GPU)
@pytest.mark.parametrize("counter,key,want", [
    ([0, 0, 0, 0], [0, 0], [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]),
    ([0xffffffff] * 4, [0xffffffff] * 2, [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]),
    ([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0],
     [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1])])
def test_oracle_generator_gives_the_published_answers(counter, key, want):
    got = row_ops.philox4x32([np.array([c], np.uint64) for c in counter], key)
    assert [int(w[0]) for w in got] == want


def test_oracle_bits_are_uniform():
    """Mean of n uniform 16-bit values: within 6 standard errors."""
    b = row_ops.dropout_bits(np.arange(500), 1000, 1234567, 89)
    n = b.size
    assert abs(b.mean() - 32767.5) < 6 * 65536 / np.sqrt(12 * n)
    assert len({int(v) for v in row_ops.dropout_bits([0, 1, 2], 8, 5, 6).ravel()}) > 20


@pytest.mark.parametrize("kw", [
    {"x": None}, {"out": None}, {"rng": None}, {"x": 17}, {"out": 17}, {"res": 17}, {"ids": 18}, {"rng": 20},
    {"T": -1}, {"C": -1}, {"T": 1 << 31}, {"C": 1 << 31}, {"p": -0.1}, {"p": 1.0}, {"p": 0.999999},
    {"p": float("nan")}, {"dtype": 1, "x": 18}])
def test_refuses_bad_arguments(thd_lib, kw):
    a = dict(x=16, res=None, out=16, T=4, C=8, ids=None, p=0.1, rng=16, dtype=0)
    a.update(kw)
    assert T.thd_dropout_add(*a.values(), stream=0) == T.THD_ERR_INVALID_ARG


def test_refuses_unknown_type_and_skips_empty(thd_lib):
    assert T.thd_dropout_add(16, None, 16, 4, 8, None, 0.1, 16, 2, stream=0) == T.THD_ERR_UNSUPPORTED
    before = T.thd_launch_count()
    assert T.thd_dropout_add(None, None, None, 0, 8, None, 0.1, None, 0, stream=0) == T.THD_OK
    assert T.thd_dropout_add(None, None, None, 8, 0, None, 0.1, None, 0, stream=0) == T.THD_OK
    assert T.thd_launch_count() == before


# ------------------------------------------------------------------ GPU
def _state(seed, offset):
    s = np.array([seed, offset], np.uint64).view(np.int64)
    return torch.from_numpy(s).cuda()


def _check(got, x, res, ids, p, seed, offset):
    ref, keep = row_ops.dropout_add(x.double().cpu().numpy(), None if res is None else res.double().cpu().numpy(),
                                    ids, p, seed, offset)
    xs = np.abs(x.double().cpu().numpy()) * 65536.0 / (65536 - np.rint(65536 * p))
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    tol = 2.0 ** -23 * xs + half * (1 + 2.0 ** -20) * np.abs(ref) + 2.0 ** -24 * np.abs(ref)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= tol), f"max excess {(err - tol).max():.3e}"
    if res is None:                                   # the mask itself, where x shows it
        assert np.array_equal(got.double().cpu().numpy() != 0, keep & (x.double().cpu().numpy() != 0))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,C,p", [(1, 1, 0.5), (192, 128, 0.1), (3, 5, 0.3), (33, 257, 0.25), (64, 264, 0.9),
                                      (1000, 72, 0.0), (7, 4096, 0.1), (129, 1111, 0.4), (2, 100003, 0.15)])
def test_matches_oracle(thd_lib, dtype, residual, rows, C, p):
    rng = np.random.default_rng(rows + C)
    x = torch.from_numpy(rng.standard_normal((rows, C))).to(dtype).cuda()
    res = torch.from_numpy(rng.standard_normal((rows, C))).to(dtype).cuda() if residual else None
    for ids in (None, rng.integers(-2 ** 31, 2 ** 31, size=rows).astype(np.int32)):
        t = None if ids is None else torch.from_numpy(ids).cuda()
        seed, offset = 0xfedcba9876543210, 0xffffffff00000001
        out = T.dropout_add(x, _state(seed, offset), p, residual=res, row_ids=t)
        torch.cuda.synchronize()
        _check(out, x, res, np.arange(rows) if ids is None else ids, p, seed, offset)


@pytest.mark.gpu
@pytest.mark.parametrize("C", [1, 2, 7, 9, 255, 256, 257, 511, 513, 1111])
@pytest.mark.parametrize("shift", [0, 1])
def test_odd_rows_in_bf16(thd_lib, C, shift):
    """Rows that start on odd elements (pairs straddle the groups of eight and
    the rows have elements without a partner), and tensors off the 4-byte grid;
    what lies around the output stays."""
    rows = 9
    rng = np.random.default_rng(C)
    base = torch.from_numpy(rng.standard_normal((2, rows * C + 2))).bfloat16().cuda()
    x, res = (base[i].clone()[shift:shift + rows * C].view(rows, C) for i in range(2))
    out = torch.full((rows * C + 2,), 9.0, dtype=torch.bfloat16, device="cuda")
    for r in (None, res):
        T.dropout_add(x, _state(21, 22), 0.4, residual=r, out=out[shift:shift + rows * C].view(rows, C))
        torch.cuda.synchronize()
        _check(out[shift:shift + rows * C].view(rows, C), x, r, np.arange(rows), 0.4, 21, 22)
        assert bool((out[:shift] == 9.0).all()) and bool((out[shift + rows * C:] == 9.0).all())


@pytest.mark.gpu
def test_off_the_grid_tensors_give_the_same_bits(thd_lib):
    """C a multiple of 8 but tensors off the 16-byte grid take the one-element
    path: the same bits; in place over x and over the residual as well."""
    rows, C = 31, 96
    base = torch.randn(2, rows * C + 1, device="cuda").bfloat16()
    x, res = base[0, 1:].view(rows, C), base[1, 1:].view(rows, C)
    xa, ra = x.clone(), res.clone()
    assert x.data_ptr() % 16 and not xa.data_ptr() % 16
    rng = _state(5, 6)
    want = T.dropout_add(xa, rng, 0.2, residual=ra)
    assert torch.equal(T.dropout_add(x, rng, 0.2, residual=res), want)
    T.dropout_add(xa, rng, 0.2, residual=ra, out=ra)
    T.dropout_add(x, rng, 0.2, residual=res, out=x)
    torch.cuda.synchronize()
    assert torch.equal(ra, want) and torch.equal(x, want)


@pytest.mark.gpu
def test_a_ranks_shard_draws_the_unsplit_mask(thd_lib):
    """Every rank's rows, gathered by the partition's token map and numbered
    by it, draw what the whole buffer draws at those rows."""
    cp, lengths, C = 4, [64, 200, 8], 128
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")
    n = int(cu[-1])
    part, st = T.cp_partition(cu, cp_size=cp, token_map_capacity=n)
    T.check_status(st)
    x, res = torch.randn(n, C, device="cuda").bfloat16(), torch.randn(n, C, device="cuda").bfloat16()
    rng = _state(11, 12)
    whole = T.dropout_add(x, rng, 0.3, residual=res)
    for r in range(cp):
        ids = part["token_map"][r * (n // cp):(r + 1) * (n // cp)]
        at = ids.long()
        assert torch.equal(T.dropout_add(x[at], rng, 0.3, residual=res[at], row_ids=ids), whole[at])


@pytest.mark.gpu
def test_backward_is_the_gradient(thd_lib):
    """dx = keep g / (1 - p): with the forward's state the same mask, and the
    difference quotient of <out, g> (linear in x: exact up to rounding)."""
    x, g = torch.randn(40, 56, device="cuda"), torch.randn(40, 56, device="cuda")
    rng = _state(3, 4)
    gx = T.dropout_add(g, rng, 0.35)
    torch.cuda.synchronize()
    _check(gx, g, None, np.arange(40), 0.35, 3, 4)
    for t, c in ((0, 0), (17, 33), (39, 55)):
        d = torch.zeros_like(x)
        d[t, c] = 1.0
        diff = T.dropout_add(x + d, rng, 0.35).double() - T.dropout_add(x - d, rng, 0.35).double()
        assert abs(float((diff * g.double()).sum()) / 2 - float(gx[t, c])) <= 2.0 ** -20 * 8 * float(g.abs().max())


@pytest.mark.gpu
@pytest.mark.parametrize("C", [64, 67])
def test_dropped_places_hide_infinities_and_nan(thd_lib, C):
    keep = row_ops.dropout_bits(np.arange(20), C, 8, 9) >= round(0.5 * 65536)
    x = np.where(keep, 1.0, np.where(np.arange(C) % 2 == 0, np.nan, np.inf))
    out = T.dropout_add(torch.from_numpy(x).float().cuda(), _state(8, 9), 0.5)
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), np.where(keep, 2.0, 0.0))


@pytest.mark.gpu
def test_a_captured_graph_draws_anew_when_its_state_advances(thd_lib):
    x = torch.ones(64, 128, device="cuda")
    rng, out = _state(1, 100), torch.empty(64, 128, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        T.dropout_add(x, rng, 0.5, out=out)
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        _check(out, x, None, np.arange(64), 0.5, 1, 100 + step)
        rng[1] += 1


@pytest.mark.gpu
@pytest.mark.parametrize("C", [32768, 32767])
def test_elements_past_32_bits(thd_lib, C):
    """70,001 rows, 2.3e9 elements: the last rows are what they are alone."""
    rows, n = 70001, 5
    rng = torch.tensor([11, 13], dtype=torch.int64, device="cuda")
    x = torch.zeros(rows, C, dtype=torch.bfloat16, device="cuda")
    x[-n:] = torch.randn(n, C, device="cuda").bfloat16()
    ids = torch.arange(rows, dtype=torch.int32, device="cuda")
    want = T.dropout_add(x[-n:].clone(), rng, 0.3, row_ids=ids[-n:].clone())
    out = T.dropout_add(x, rng, 0.3, out=x)
    assert torch.equal(out[-n:], want) and not out[:-n].any()


@pytest.mark.gpu
def test_helper_refuses_wrong_tensors(thd_lib):
    x = torch.zeros(8, 16, device="cuda", dtype=torch.bfloat16)
    rng, ids = _state(1, 2), torch.zeros(8, device="cuda", dtype=torch.int32)
    before = T.thd_launch_count()
    for kw in ({"residual": x.float()}, {"residual": x[:4]}, {"row_ids": ids.long()}, {"row_ids": ids[:7]},
               {"out": x.t()}, {"row_ids": ids.cpu()}, {"p": 1.0}, {"rng": rng[:1]}, {"rng": rng.int()},
               {"rng": rng.cpu()}, {"x": x.t()}, {"x": x.cpu()}):
        a = {"x": x, "rng": rng, "p": 0.1, **kw}
        with pytest.raises(T.ThdError):
            T.dropout_add(a.pop("x"), a.pop("rng"), a.pop("p"), **a)
    with pytest.raises(T.ThdError) as e:
        T.dropout_add(x.half(), rng, 0.1)
    assert e.value.code == T.THD_ERR_UNSUPPORTED and T.thd_launch_count() == before
    assert T.dropout_add(x[:0], rng, 0.1).shape == (0, 16) and T.thd_launch_count() == before
