"""The paged key-value cache on the GPU against the fp64 oracle: append, decode,
eviction, and a run of them together."""

import numpy as np
import pytest
import torch

from cache_testutil import FP8, Cache, same, slotwise
from oracle import cache_oracle as co
from packed_sequence_context_gb300 import thd_attn as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(thd_lib):
    return thd_lib


def _cuda(x, dtype=torch.int32):
    return None if x is None else torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def _np(t):
    return t.double().cpu().numpy()


def _status(st, want=0):
    torch.cuda.synchronize()
    assert int(st.item()) == want


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,old,page,Hkv,D,first", [
    ([1], [0], 16, 1, 64, False), ([1, 1, 1, 1, 1], [0, 15, 16, 17, 900], 16, 8, 128, True),
    ([0, 3, 0, 0, 70, 1, 0], [5, 0, 0, 64, 31, 8, 0], 1, 3, 64, False), ([513, 40], [0, 7], 24, 2, 128, True),
    ([300, 299, 1], [0, 1, 5], 7, 5, 64, True), ([2000], [100], 256, 16, 128, False)])
def test_append(new, old, page, Hkv, D, first, fp8):
    lens = np.array(new) + np.array(old)
    c = Cache(lens, page=page, Hkv=Hkv, D=D, fp8=fp8, heads_first=first, seed=len(new) + page)
    m, slack = sum(new), 3
    x = torch.randn(m + slack, 3 * Hkv * D, device="cuda").to(torch.bfloat16)
    x[: m // 2, Hkv * D] *= 2.0 ** 30              # rows of other sizes, zeros and the e4m3 format's edges
    if m > 2:
        x[1] = 0
        x[2, Hkv * D:] = 448.0
    k, v = x[:, Hkv * D:2 * Hkv * D].view(-1, Hkv, D), x[:, 2 * Hkv * D:].view(-1, Hkv, D)
    cu = np.concatenate([[0], np.cumsum(new)])
    seen = lens + 11
    before = c.host()
    ref, w, pos = co.append(before, _np(k), _np(v), cu, c.table_np, lens, seen, _np(c.weight), c.pos.cpu().numpy())
    st = T.cache_append(k, v, *c.args(), cu_seqlens=_cuda(cu), weight=c.weight, pos=c.pos, tokens_seen=_cuda(seen),
                        **c.exps())
    _status(st)
    got = c.host()
    for n in got:
        if got[n] is not None:
            assert same(got[n], ref[n]), n          # the slots that no row went to as well
    assert same(_np(c.weight), w) and same(c.pos.cpu().numpy(), pos)


def test_append_one_row_each_needs_no_offsets():
    c = Cache([4, 1, 33], Hkv=2, D=64, seed=3)
    k, v = (torch.randn(3, 2, 64, device="cuda").to(torch.bfloat16) for _ in range(2))
    ref, _, _ = co.append(c.host(), _np(k), _np(v), [0, 1, 2, 3], c.table_np, c.lens)
    _status(T.cache_append(k, v, *c.args()))
    assert same(c.host()["k"], ref["k"]) and same(c.host()["v"], ref["v"])


def test_append_marks_rows_that_are_no_numbers():
    c = Cache([3], Hkv=1, D=64, fp8=True, seed=4)
    k, v = (torch.randn(3, 1, 64, device="cuda").to(torch.bfloat16) for _ in range(2))
    k[0, 0, 63], v[1, 0, 0], k[2, 0, 5] = float("inf"), float("nan"), float("-inf")
    _status(T.cache_append(k, v, *c.args(), cu_seqlens=_cuda([0, 3]), **c.exps()))
    p, at = co.slots(c.table_np[0], 3, 16)
    assert list(c.host()["k_exp"][p, at, 0] == 255) == [True, False, True]
    assert list(c.host()["v_exp"][p, at, 0] == 255) == [False, True, False]
    q = torch.randn(1, 2, 64, device="cuda").to(torch.bfloat16)
    o, lse, st = T.attn_decode(q, *c.args(), **c.exps())
    _status(st)
    assert torch.isnan(o).all() and torch.isnan(lse).all()


def test_append_reports_and_leaves_out_what_has_no_slot():
    c = Cache([20, 20, 20, 20], page=4, Hkv=2, D=64, seed=5)
    before = c.host()
    table = c.table.clone()
    table[1, 4] = c.pages                          # past the cache
    kv_len = c.kv_len.clone()
    kv_len[2] = 10000                              # past the table
    kv_len[3] = 1                                  # fewer than the new rows
    k, v = (torch.randn(8, 2, 64, device="cuda").to(torch.bfloat16) for _ in range(2))
    st = T.cache_append(k, v, c.k, c.v, table, kv_len, cu_seqlens=_cuda([0, 2, 4, 6, 8]))
    _status(st, T.THD_DEV_ERR_KV_LEN)              # the larger of the two codes
    ref, _, _ = co.append(before, _np(k), _np(v), [0, 2, 2, 2, 2], c.table_np, c.lens)
    p, at = co.slots(c.table_np[3], 20, 4)         # sequence 3's second row has slot 0
    ref["k"][p[0], at[0]], ref["v"][p[0], at[0]] = _np(k)[7], _np(v)[7]
    assert same(c.host()["k"], ref["k"]) and same(c.host()["v"], ref["v"])
    st.zero_()
    T.cache_append(k, v, c.k, c.v, table, c.kv_len, cu_seqlens=_cuda([0, 2, 4, 6, 8]), dev_status=st)
    _status(st, T.THD_DEV_ERR_PAGE)
    T.cache_append(k, v, *c.args(), cu_seqlens=_cuda([0, 2, 4, 6, 8]), dev_status=st)
    _status(st, T.THD_DEV_ERR_PAGE)                # sticky
    for cu, code in (([1, 2, 4, 6, 8], T.THD_DEV_ERR_NONZERO_START), ([0, 4, 2, 6, 8], T.THD_DEV_ERR_NOT_MONOTONE),
                     ([0, 2, 4, 6, 9], T.THD_DEV_ERR_EXCEEDS_BUF)):
        _status(T.cache_append(k, v, *c.args(), cu_seqlens=_cuda(cu)), code)


# ------------------------------------------------------------------ decode
def _decode(c, q, *, cap=0.0, slopes=None, start=None, pos=False, seen=None, weight=False, scale=None):
    scale = (1.0 if not c.fp8 else 1 / 80) / np.sqrt(c.D) if scale is None else scale
    ref = co.decode(_np(q), c.host(), c.table_np, c.lens, scale=np.float32(scale), softcap=np.float32(cap), slopes=slopes,
                    start=start, pos=c.pos.cpu().numpy() if pos else None, seen=seen,
                    weight=_np(c.weight) if weight else None)
    wo = torch.full_like(c.weight, -7.0) if weight else None
    kw = dict(softmax_scale=scale, softcap=cap, dist_slopes=_cuda(slopes, torch.float32), kv_start=_cuda(start),
              pos=c.pos if pos else None, tokens_seen=_cuda(seen), **c.exps())
    o, lse, st = T.attn_decode(q, *c.args(), weight=c.weight if weight else None, weight_out=wo, **kw)
    _status(st)
    assert np.all(np.abs(_np(o) - ref["o"]) <= ref["tol_o"])
    inf = np.isinf(ref["lse"])
    assert same(_np(lse)[inf], ref["lse"][inf])
    assert np.all(np.abs(_np(lse)[~inf] - ref["lse"][~inf]) <= ref["tol_lse"][~inf])
    if weight:
        seen_slots = ref["tol_weight"] > 0
        assert np.all(_np(wo)[~seen_slots] == -7.0)
        assert np.all(np.abs(_np(wo) - ref["weight"])[seen_slots] <= ref["tol_weight"][seen_slots])
        inplace = c.weight.clone()
        o2, lse2, _ = T.attn_decode(q, *c.args(), weight=inplace, **kw)
        torch.cuda.synchronize()
        m = torch.from_numpy(seen_slots).cuda()
        assert torch.equal(inplace[m], wo[m]) and torch.equal(inplace[~m], c.weight[~m])
        assert torch.equal(o2, o) and torch.equal(lse2, lse)
    return o, lse


EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 700]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,Hkv,G,first", [(16, 2, 4, False), (1, 1, 8, True), (7, 3, 1, False), (64, 1, 16, True),
                                              (24, 2, 3, True), (100, 1, 32, False), (256, 1, 9, False), (8, 1, 40, True)])
def test_decode_lengths(page, Hkv, G, first, D, fp8):
    c = Cache(EDGES, page=page, Hkv=Hkv, D=D, fp8=fp8, heads_first=first, seed=page + G)
    q = torch.randn(len(EDGES), Hkv * G, D, device="cuda").to(torch.bfloat16)
    _decode(c, q, weight=G in (1, 3, 40))


@pytest.mark.parametrize("fp8,D,G,page", [(False, 128, 4, 64), (True, 64, 2, 24), (True, 128, 16, 32), (False, 64, 32, 16)])
def test_decode_long_shared_among_blocks(fp8, D, G, page):
    """One sequence over all blocks, short ones beside it, a rest that ends inside every unit."""
    c = Cache([3, 9001, 0, 70, 4097], page=page, Hkv=1, D=D, fp8=fp8, seed=9)
    q = torch.randn(5, G, D, device="cuda").to(torch.bfloat16) * 2
    _decode(c, q, weight=True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("cap,bias,docs,pos", [(30.0, False, False, False), (0.0, True, False, False), (0.0, True, False, True),
                                               (5.0, True, True, True), (0.0, False, True, False), (1e-3, False, False, False)])
def test_decode_scores(cap, bias, docs, pos, fp8):
    lens = [300, 1, 64, 129, 0, 1000]
    c = Cache(lens, page=16, Hkv=2, D=64, fp8=fp8, seed=21)
    q = torch.randn(6, 8, 64, device="cuda").to(torch.bfloat16) * 3
    slopes = (2.0 ** -np.arange(1, 9)).astype(np.float32) if bias else None
    start = [77, 0, 64, -5, 3, 999] if docs else None    # none, clamped, all hidden, one left
    _decode(c, q, cap=cap, slopes=slopes, start=start, pos=pos, seen=np.array(lens) + (1 << 20) if pos else None, weight=True)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_many_short_sequences(fp8):
    """More sequences than threads and items than blocks, empty ones among them."""
    lens = np.random.default_rng(3).integers(0, 90, 700)
    lens[:5] = lens[-3:] = lens[200:210] = 0
    c = Cache(lens, page=16, Hkv=2, D=64, fp8=fp8, seed=23)
    q = torch.randn(700, 4, 64, device="cuda").to(torch.bfloat16)
    _decode(c, q, start=np.random.default_rng(4).integers(-3, 80, 700), weight=True)


@pytest.mark.parametrize("fp8,G", [(False, 512), (True, 100), (False, 65)])
def test_decode_large_groups(fp8, G):
    c = Cache([700, 0, 65], page=16, Hkv=1, D=64, fp8=fp8, seed=25)
    q = torch.randn(3, G, 64, device="cuda").to(torch.bfloat16)
    _decode(c, q, weight=True)


def test_decode_one_table_row_for_all():
    """Beams of one prompt: the same pages, other lengths."""
    c = Cache([300], page=16, Hkv=2, D=64, seed=27)
    q = torch.randn(4, 4, 64, device="cuda").to(torch.bfloat16)
    n = _cuda([300, 17, 0, 250])
    o, lse, st = T.attn_decode(q, c.k, c.v, c.table.expand(4, -1), n)
    _status(st)
    want = T.attn_decode(q, c.k, c.v, c.table.repeat(4, 1), n)
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    ref = co.decode(_np(q), c.host(), np.repeat(c.table_np, 4, 0), [300, 17, 0, 250], scale=np.float32(0.125))
    assert np.all(np.abs(_np(o) - ref["o"]) <= ref["tol_o"])


def test_decode_two_streams_at_once():
    """Calls that overlap, each with its own workspace, next to one another's results."""
    cs = [Cache([4000, 123], page=16, Hkv=2, D=64, seed=s) for s in (81, 82)]
    q = torch.randn(2, 8, 64, device="cuda").to(torch.bfloat16)
    want = [T.attn_decode(q, *c.args()) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            got[i].append(T.attn_decode(q, *cs[i].args(), stream=st))
    torch.cuda.synchronize()
    for i in (0, 1):
        for o, lse, st in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1]) and int(st.item()) == 0


def test_decode_slices_and_strides():
    """q out of a fused projection, cache pools that are slices of larger tensors, a table wider than it is used."""
    c = Cache([100, 257], page=16, Hkv=2, D=64, seed=31, wide=40)
    x = torch.randn(2, 12 * 64, device="cuda").to(torch.bfloat16)
    q = x[:, :4 * 64].view(2, 4, 64)
    want = _decode(c, q.contiguous())
    both = torch.empty((c.pages, 2, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    both[:, 0], both[:, 1] = c.k, c.v
    o, lse, st = T.attn_decode(q, both[:, 0], both[:, 1], c.table[:, :20], c.kv_len)
    _status(st)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_decode_infinite_and_missing_scores():
    """A key of infinities makes its row NaN; a score of -inf takes no part."""
    c = Cache([70, 70], page=16, Hkv=1, D=64, seed=33)
    q = torch.ones(2, 1, 64, device="cuda", dtype=torch.bfloat16)
    c.k[c.table[0, 1], 3, 0, 0] = float("-inf")    # slot 19 of sequence 0: a score of -inf
    c.k[c.table[1, 1], 3, 0, 0] = float("inf")
    o, lse, st = T.attn_decode(q, *c.args())
    _status(st)
    h = c.host()
    p, at = co.slots(c.table_np[0], 70, 16)
    keep = np.arange(70) != 19
    s = h["k"][p, at, 0][keep].sum(-1) / 8
    w = np.exp(s - s.max())
    want = (w / w.sum()) @ h["v"][p, at, 0][keep]
    assert np.abs(_np(o)[0, 0] - want).max() <= 2.0 ** -7 * np.abs(h["v"][p, at, 0]).max()
    assert abs(float(lse[0, 0]) - (s.max() + np.log(w.sum()))) < 1e-4
    assert torch.isnan(o[1]).all() and torch.isnan(lse[0, 1])


def test_decode_values_of_very_different_scales():
    """Exponents from end to end: the row of the largest scale has little weight."""
    c = Cache([200], page=16, Hkv=1, D=64, fp8=True, seed=35, spread=50)
    q = torch.randn(1, 2, 64, device="cuda").to(torch.bfloat16)
    _decode(c, q, weight=True)


@pytest.mark.parametrize("size", [2.0 ** -100, 1e-20, 1e20, 2.0 ** 100])
def test_decode_e4m3_queries_of_any_size(size):
    c = Cache([150], page=16, Hkv=1, D=128, fp8=True, seed=36)
    q = (torch.randn(1, 8, 128, device="cuda") * size).to(torch.bfloat16)
    _decode(c, q, scale=float(1 / (80 * 11 * size)))


def test_decode_reports_bad_tables_and_lengths():
    c = Cache([40, 40, 40, 40], page=16, Hkv=1, D=64, seed=37)
    q = torch.randn(4, 2, 64, device="cuda").to(torch.bfloat16)
    good, _, st = T.attn_decode(q, *c.args())
    _status(st)
    for bad in (-1, c.pages, 2 ** 31 - 1, -2 ** 31):
        table = c.table.clone()
        table[1, 2] = bad
        o, _, st = T.attn_decode(q, c.k, c.v, table, c.kv_len)
        _status(st, T.THD_DEV_ERR_PAGE)
        assert torch.equal(o[[0, 2, 3]], good[[0, 2, 3]])
    for bad in (-1, 49, 2 ** 31 - 1):
        n = c.kv_len.clone()
        n[3] = bad
        o, lse, st = T.attn_decode(q, c.k, c.v, c.table, n, dev_status=st)
        _status(st, T.THD_DEV_ERR_KV_LEN)
        assert torch.equal(o[:3], good[:3]) and not o[3].any() and torch.isinf(lse[:, 3]).all()


def test_decode_repeats_bit_for_bit():
    c = Cache([5000, 31, 2500], page=32, Hkv=2, D=128, fp8=True, seed=39)
    q = torch.randn(3, 16, 128, device="cuda").to(torch.bfloat16)
    runs = [T.attn_decode(q, *c.args(), weight=c.weight, weight_out=torch.zeros_like(c.weight), **c.exps()) for _ in range(3)]
    torch.cuda.synchronize()
    for r in runs[1:]:
        assert torch.equal(r[0], runs[0][0]) and torch.equal(r[1], runs[0][1])


@pytest.mark.parametrize("fp8", [False, True])
def test_offsets_past_32_bits(fp8):
    """Pages that lie beyond 2^32 bytes and elements of their pool."""
    page, Hkv, D = 16, 8, 128
    pages = (1 << 33) // (page * Hkv * D * (1 if fp8 else 2)) + 5
    lens = np.array([40, 16], np.int32)
    table = np.array([[pages - 1, 3, pages - 3], [pages - 2, -1, -1]], np.int32)
    dt = FP8 if fp8 else torch.bfloat16
    kc, vc = (torch.empty((pages, page, Hkv, D), dtype=dt, device="cuda") for _ in range(2))
    small = Cache(lens, page=page, Hkv=Hkv, D=D, fp8=fp8, seed=41)   # the same rows in a small pool
    exps = {}
    if fp8:
        exps = {n: torch.empty((pages, page, Hkv), dtype=torch.uint8, device="cuda") for n in ("k_exp", "v_exp")}
    w, pos = torch.zeros((pages, page, Hkv), device="cuda"), torch.zeros((pages, page, Hkv), dtype=torch.int32, device="cuda")
    rows = {n: torch.randn(int(lens.sum()), Hkv, D, device="cuda").to(torch.bfloat16) for n in "kv"}
    cu = _cuda([0, 40, 56])
    big = (kc, vc, _cuda(table), small.kv_len)
    q = torch.randn(2, 16, D, device="cuda").to(torch.bfloat16)
    outs = []
    for args, e, weight, ps in ((big, exps, w, pos), (small.args(), small.exps() if fp8 else {}, torch.zeros_like(small.weight),
                                                      torch.zeros_like(small.pos))):
        _status(T.cache_append(rows["k"], rows["v"], *args, cu_seqlens=cu, weight=weight, pos=ps, **e))
        o, lse, st = T.attn_decode(q, *args, weight=weight, **e)
        _status(st)
        n, st = T.cache_evict(*args, weight, ps, small.kv_len, budget=20, recent=4, **e)
        _status(st)
        o2, lse2, st = T.attn_decode(q, args[0], args[1], args[2], n, **e)
        _status(st)
        outs.append((o, lse, o2, lse2, n))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ evict
def _evict(c, budget, sinks=0, recent=0, seen=None, in_place=True):
    seen = c.lens if seen is None else np.asarray(seen)
    w, pos, before = c.weight.cpu().numpy(), c.pos.cpu().numpy(), c.host()
    ref, rw, rp, rn = co.evict(before, c.table_np, c.lens, w, pos, seen, budget, sinks, recent)
    wo, po = (c.weight, c.pos) if in_place else (torch.full_like(c.weight, -3.0), torch.full_like(c.pos, -3))
    n, st = T.cache_evict(*c.args(), c.weight, c.pos, _cuda(seen), budget=budget, sinks=sinks, recent=recent,
                          weight_out=wo, pos_out=po, **c.exps())
    _status(st)
    got = c.host()
    for name in got:
        if got[name] is not None:
            assert same(got[name], ref[name]), name
    assert np.array_equal(n.cpu().numpy(), rn)
    if in_place:
        assert same(wo.cpu().numpy(), rw) and same(po.cpu().numpy(), rp)
        return
    assert same(c.weight.cpu().numpy(), w) and same(c.pos.cpu().numpy(), pos)
    kept = np.zeros(rw.shape, bool)
    for b, m in enumerate(rn):
        kept[co.slots(c.table_np[b], int(m), c.page)] = True
    assert same(wo.cpu().numpy(), np.where(kept, rw, -3.0)) and same(po.cpu().numpy(), np.where(kept, rp, -3))


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("fp8,D,page,Hkv,first", [(False, 128, 16, 2, True), (True, 64, 24, 3, False), (True, 128, 1, 1, True),
                                                  (False, 64, 64, 2, False)])
@pytest.mark.parametrize("budget", [1, 33, 256, 1000])
def test_evict(budget, fp8, D, page, Hkv, first, in_place):
    lens = [0, 1, 32, 33, 34, 256, 257, 999, 1000, 1001, 2500]
    c = Cache(lens, page=page, Hkv=Hkv, D=D, fp8=fp8, heads_first=first, seed=budget)
    r = np.random.default_rng(budget)
    # half the weights on a coarse grid: ties at the threshold
    w = r.random(c.weight.shape).astype(np.float32)
    w[r.random(w.shape) < 0.5] = 0.5
    c.weight.copy_(torch.from_numpy(w))
    c.pos.copy_(torch.from_numpy(r.integers(0, 2600, c.pos.shape).astype(np.int32)))
    _evict(c, budget, sinks=4, recent=budget // 3, seen=np.array(lens) + 50, in_place=in_place)


@pytest.mark.parametrize("kind", ["equal", "zeros", "special", "negative", "protected", "rising", "falling", "close"])
def test_evict_weights_of_every_kind(kind):
    lens, budget = [700, 5000], 300
    c = Cache(lens, page=16, Hkv=2, D=64, seed=51)
    r = np.random.default_rng(7)
    w = r.random(c.weight.shape).astype(np.float32)
    sinks, recent = 0, 0
    c.pos.zero_()
    if kind == "equal":
        w[:] = 0.25
    elif kind == "zeros":                          # +0 and -0 are equal
        w[:] = np.where(r.random(w.shape) < 0.5, 0.0, -0.0)
    elif kind == "special":
        x = r.integers(0, 6, w.shape)
        for i, v in enumerate((np.nan, np.inf, -np.inf, 1e-45, -1e-45)):
            w[x == i] = v
    elif kind == "negative":
        w = -w
    elif kind == "protected":                      # more than the budget holds: the lower slots
        recent = 400
        c.pos.copy_(torch.from_numpy(r.integers(0, 800, w.shape).astype(np.int32)))
    elif kind in ("rising", "falling"):
        for b, n in enumerate(lens):
            p, at = co.slots(c.table_np[b], n, 16)
            w[p, at] = (np.arange(n) if kind == "rising" else -np.arange(n))[:, None]
    else:                                          # neighbours in the last digit
        w = (np.float32(1.0).view(np.int32) + r.integers(0, 3, w.shape).astype(np.int32)).view(np.float32)
    c.weight.copy_(torch.from_numpy(w))
    _evict(c, budget, sinks=sinks, recent=recent, seen=[700, 790])


def test_evict_more_slots_than_a_cluster_holds():
    """Keys past what the blocks keep in shared memory are read again; one of the sequences is that long."""
    n = 8 * 40960 + 4321
    c = Cache([n, 50], page=64, Hkv=1, D=64, fp8=True, seed=53)
    _evict(c, 1500, recent=100, seen=[1 << 20, 1 << 20])


def test_evict_reports_bad_tables_and_lengths():
    c = Cache([40, 40, 40], page=16, Hkv=1, D=64, seed=55)
    before = c.host()
    table, n = c.table.clone(), c.kv_len.clone()
    table[1, 1] = c.pages + 7
    n[2] = 49
    new, st = T.cache_evict(c.k, c.v, table, n, c.weight, c.pos, c.kv_len, budget=20)
    _status(st, T.THD_DEV_ERR_KV_LEN)
    after = c.host()
    p, at = co.slots(c.table_np[2], 40, 16)
    assert same(after["k"][p, at], before["k"][p, at]) and int(new[0]) == 20
    _, st = T.cache_evict(c.k, c.v, table, c.kv_len, c.weight, c.pos, c.kv_len, budget=20)
    _status(st, T.THD_DEV_ERR_PAGE)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("captured", [False, True])
def test_a_run_of_decoding(fp8, captured):
    """Prompts go in, tokens follow one by one with rotary positions, weights add up, and caches are trimmed: eager,
    and with the token's step captured once and replayed while the lengths grow; every step against the oracle."""
    Hq, Hkv, D, page, B, budget = 4, 2, 64, 16, 3, 48
    r = np.random.default_rng(61)
    prompts = np.array([40, 7, 1], np.int32)
    steps, wide = 30, 8
    c = Cache([wide * page] * B, page=page, Hkv=Hkv, D=D, fp8=fp8, seed=62)    # the pool; nothing held yet
    c.weight.zero_(), c.pos.zero_()
    inv = 1e4 ** (-np.arange(D // 2) / (D // 2))
    kv_len, seen = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = np.concatenate([[0], np.cumsum(prompts)])
    k, v = (torch.randn(int(cu[-1]), Hkv, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    kv_len += _cuda(prompts)
    seen += _cuda(prompts)
    host, w, pos = co.append(c.host(), _np(k), _np(v), cu, c.table_np, prompts, prompts, _np(c.weight), c.pos.cpu().numpy())
    T.cache_append(k, v, c.k, c.v, c.table, kv_len, cu_seqlens=_cuda(cu), weight=c.weight, pos=c.pos, tokens_seen=seen,
                   dev_status=st, **c.exps())
    x = torch.empty((B, Hq + 2 * Hkv, D), dtype=torch.bfloat16, device="cuda")
    out = {}

    def step():
        kv_len.add_(1)
        seen.add_(1)
        q, kn = T.rope(x[:, :Hq], x[:, Hq:Hq + Hkv], (seen - 1), inv)
        T.cache_append(kn, x[:, Hq + Hkv:], c.k, c.v, c.table, kv_len, weight=c.weight, pos=c.pos, tokens_seen=seen,
                       dev_status=st, **c.exps())
        out["q"], out["k"] = q, kn
        out["o"], out["lse"], _ = T.attn_decode(q, c.k, c.v, c.table, kv_len, weight=c.weight, dev_status=st, **c.exps())
        new, _ = T.cache_evict(c.k, c.v, c.table, kv_len, c.weight, c.pos, seen, budget=budget, sinks=2, recent=10,
                               dev_status=st, **c.exps())
        kv_len.copy_(new)

    lens, count = prompts.copy(), prompts.copy()
    graph = None
    for i in range(steps):
        x.copy_(torch.from_numpy(r.standard_normal(x.shape).astype(np.float32)))
        if captured and graph is None:
            keep = [t.clone() for t in (kv_len, seen, c.k, c.v, c.weight, c.pos)]
            keep += [t.clone() for t in (c.k_exp, c.v_exp)] if fp8 else []
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                step()
            torch.cuda.current_stream().wait_stream(s)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            for t, old in zip((kv_len, seen, c.k, c.v, c.weight, c.pos, c.k_exp, c.v_exp), keep):
                t.copy_(old)
        if captured:
            graph.replay()
        else:
            step()
        _status(st)
        lens, count = lens + 1, count + 1
        host, w, pos = co.append(host, _np(out["k"]), _np(x[:, Hq + Hkv:]), np.arange(B + 1), c.table_np, lens, count, w, pos)
        ref = co.decode(_np(out["q"]), host, c.table_np, lens, scale=1 / np.sqrt(D), weight=w)
        assert np.all(np.abs(_np(out["o"]) - ref["o"]) <= ref["tol_o"]) and np.all(np.abs(_np(out["lse"]) - ref["lse"]) <= ref["tol_lse"])
        # the trim goes by the kernel's own sums (they differ from the oracle's by roundings): before it, they are near
        host, w2, pos, lens2 = co.evict(host, c.table_np, lens, ref["weight"], pos, count, budget, 2, 10)
        got_w = _np(c.weight)
        for b in range(B):
            p, at = co.slots(c.table_np[b], int(lens2[b]), page)
            assert np.all(np.abs(got_w[p, at] - w2[p, at]) <= 1e-4)
            assert np.array_equal(c.pos.cpu().numpy()[p, at], pos[p, at])
        w, lens = got_w, lens2
        assert np.array_equal(kv_len.cpu().numpy(), lens)
        for n, t in c.host().items():
            if t is not None:
                for b in range(B):
                    p, at = co.slots(c.table_np[b], int(lens[b]), page)
                    assert same(t[p, at], host[n][p, at])


def test_ranks_caches_merge():
    """A sequence's slots on two caches: the outputs merged by log-sum-exp are those of one cache."""
    c = Cache([500], page=16, Hkv=2, D=64, seed=71)
    q = torch.randn(1, 4, 64, device="cuda").to(torch.bfloat16)
    want, lse, _ = T.attn_decode(q, *c.args())
    n = _cuda([208])
    o1, l1, _ = T.attn_decode(q, c.k, c.v, c.table, n)
    o2, l2, _ = T.attn_decode(q, c.k, c.v, c.table[:, 13:].contiguous(), c.kv_len - 208)
    acc, lacc = o1.float(), l1.clone()
    T.lse_merge_bf16(acc, lacc, o2, l2)
    torch.cuda.synchronize()
    # the parts' and the whole's roundings to bf16
    assert (acc - want.float()).abs().max() <= 3 * 2.0 ** -8 * o1.float().abs().max().clamp(min=1) and (lacc - lse).abs().max() < 1e-5


def test_another_stream():
    """A busy stream's calls, with the current stream making tensors meanwhile."""
    c = Cache([3000, 60], page=16, Hkv=2, D=64, seed=73)
    q = torch.randn(2, 8, 64, device="cuda").to(torch.bfloat16)
    want = T.attn_decode(q, *c.args(), weight=c.weight, weight_out=torch.zeros_like(c.weight))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    wo = torch.zeros_like(c.weight)
    side.wait_stream(torch.cuda.current_stream())
    got = T.attn_decode(q.clone(), *c.args(), weight=c.weight, weight_out=wo, stream=side)
    junk = [torch.full((n,), 0x3f, dtype=torch.uint8, device="cuda")
            for n in [T.thd_decode_workspace_size(2, 8, 2, 64, c.table.shape[1] * 16, 1)] * 3]
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and int(got[2].item()) == 0
    del junk
