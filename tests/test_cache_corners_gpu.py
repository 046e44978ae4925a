"""Corners of the paged cache: bad pages of sequences that nothing leaves; values of zeros in 8 bits;
more protected tokens than a budget holds; documents and eviction;
tables much wider than the sequences; weights that lie close together."""

import numpy as np
import pytest
import torch

from cache_testutil import Cache, same
from oracle import cache_oracle as co
from packed_sequence_context_gb300 import thd_attn as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(thd_lib):
    return thd_lib


def _cuda(x, dtype=torch.int32):
    return None if x is None else torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def _status(st, want=0):
    torch.cuda.synchronize()
    assert int(st.item()) == want


@pytest.mark.parametrize("n", [1, 19, 20])
@pytest.mark.parametrize("bad", [-1, 2 ** 31 - 1])
def test_evict_reports_a_bad_page_where_nothing_leaves(n, bad):
    """A sequence within the budget: its numbers cannot go to the other arrays, and the status says so."""
    c = Cache([45, n, 20], page=16, Hkv=2, D=64, seed=3)
    table = c.table.clone()
    table[1, (n - 1) // 16] = bad
    before, w, pos = c.host(), c.weight.cpu().numpy(), c.pos.cpu().numpy()
    for name in ("weight", "pos"):                 # each array alone, then both
        wo = torch.full_like(c.weight, -3.0) if name == "weight" else c.weight.clone()
        po = torch.full_like(c.pos, -3) if name == "pos" else c.pos.clone()
        k, v = c.k.clone(), c.v.clone()
        _, st = T.cache_evict(k, v, table, c.kv_len, wo if name == "pos" else c.weight, po if name == "weight" else c.pos,
                              c.kv_len, budget=20, weight_out=wo, pos_out=po)
        _status(st, T.THD_DEV_ERR_PAGE)
    wo, po = torch.full_like(c.weight, -3.0), torch.full_like(c.pos, -3)
    new, st = T.cache_evict(c.k, c.v, table, c.kv_len, c.weight, c.pos, c.kv_len, budget=20, weight_out=wo, pos_out=po)
    _status(st, T.THD_DEV_ERR_PAGE)
    assert new.tolist() == [20, n, 20]
    ref, rw, rp, _ = co.evict(before, c.table_np, c.lens, w, pos, c.lens, 20)
    for b in (0, 2):                               # the others
        p, at = co.slots(c.table_np[b], 20, 16)
        assert same(c.host()["k"][p, at], ref["k"][p, at]) and same(c.host()["v"][p, at], ref["v"][p, at])
        assert same(wo.cpu().numpy()[p, at], rw[p, at]) and same(po.cpu().numpy()[p, at], rp[p, at])


# ------------------------------------------------------------------ rows of zeros among 8-bit values
def _check(c, q, scale, **kw):
    """attn_decode of an 8-bit cache against the oracle and its bounds."""
    ref = co.decode(q.double().cpu().numpy(), c.host(), c.table_np, c.lens, scale=np.float32(scale), **kw)
    o, lse, st = T.attn_decode(q, *c.args(), softmax_scale=scale, **c.exps())
    _status(st)
    assert np.all(np.abs(o.double().cpu().numpy() - ref["o"]) <= ref["tol_o"])
    assert np.all(np.abs(lse.double().cpu().numpy() - ref["lse"]) <= ref["tol_lse"])
    return o, ref


@pytest.mark.parametrize("D,G", [(64, 1), (64, 16), (64, 32), (128, 8), (128, 16), (128, 32)])
@pytest.mark.parametrize("zeros,size,near", [([0], 1e-2, 14.0), ([5, 69], 1e-8, 0.0), (list(range(64)), 1e-3, 9.0),
                                             ([130], 2.0 ** -50, 3.0), (list(range(0, 150, 2)), 1e-2, 12.0)])
def test_zero_values_of_a_strong_key_hide_nothing(zeros, size, near, D, G):
    """Keys that take most of the weight and whose values are zeros, next to small values: what is left of those shows."""
    n = 150
    c = Cache([n], page=16, Hkv=1, D=D, fp8=True, seed=7)
    k = torch.randn(n, 1, D, device="cuda") * 0.1
    k[zeros] = 1.0                                 # q . k = D for a query of ones
    v = torch.randn(n, 1, D, device="cuda") * size
    v[zeros] = 0
    v[zeros[-1], 0, ::3] = -0.0
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    _status(T.cache_append(k, v, *c.args(), cu_seqlens=_cuda([0, n]), **c.exps()))
    q = torch.ones(1, G, D, device="cuda", dtype=torch.bfloat16) + torch.randn(1, G, D, device="cuda").to(torch.bfloat16) / 64
    o, ref = _check(c, q, near / D if near else 1e-6)
    assert (o.float().abs().amax(-1) > 0).all()    # the rest has e^-14 of the weight at least
    # whatever scale the rows of zeros carry, as another program may have stored them
    p, at = co.slots(c.table_np[0], n, 16)
    for e in (15, 200, 254):
        c.v_exp[_cuda(p[zeros], torch.int64), _cuda(at[zeros], torch.int64)] = e
        _check(c, q, near / D if near else 1e-6)


def test_zero_values_alone():
    """Nothing but zeros, also in some warps' and blocks' shares only; one row that is no number stays so."""
    n = 5000
    c = Cache([n, 40], page=24, Hkv=2, D=128, fp8=True, seed=8)
    p, at = co.slots(c.table_np[0], n, 24)
    zero = slice(700, 4100)
    c.v.view(torch.uint8)[_cuda(p[zero], torch.int64), _cuda(at[zero], torch.int64)] = 0
    c.v_exp[_cuda(p[zero], torch.int64), _cuda(at[zero], torch.int64)] = 220
    p1, at1 = co.slots(c.table_np[1], 40, 24)
    c.v.view(torch.uint8)[_cuda(p1, torch.int64), _cuda(at1, torch.int64)] = 0x80
    q = torch.randn(2, 8, 128, device="cuda").to(torch.bfloat16)
    o, _ = _check(c, q, 1 / 900)
    assert not o[1].any()
    c.v_exp[int(p1[17]), int(at1[17]), 0] = 255    # zeros marked as no numbers
    o, _, st = T.attn_decode(q, *c.args(), softmax_scale=1 / 900, **c.exps())
    _status(st)
    assert torch.isnan(o[1, :4]).all() and not o[1, 4:].any() and not torch.isnan(o[0]).any()


# ------------------------------------------------------------------ more protected tokens than the budget holds
def _trim(c, w, pos, seen, budget, **kw):
    """cache_evict in place against the oracle; the kept slots' numbers."""
    c.weight.copy_(torch.from_numpy(w)), c.pos.copy_(torch.from_numpy(pos))
    ref, rw, rp, rn = co.evict(c.host(), c.table_np, c.lens, w, pos, seen, budget, kw.get("sinks", 0), kw.get("recent", 0))
    new, st = T.cache_evict(*c.args(), c.weight, c.pos, _cuda(seen), budget=budget, **kw, **c.exps())
    _status(st)
    assert same(c.host()["k"], ref["k"]) and same(c.host()["v"], ref["v"]) and np.array_equal(new.cpu().numpy(), rn)
    assert same(c.weight.cpu().numpy(), rw) and same(c.pos.cpu().numpy(), rp)
    return [rp[co.slots(c.table_np[b], int(n), c.page)] for b, n in enumerate(rn)]


def _numbered(c, r, seen, mixed):
    """Every held slot's token, by slot or in no order."""
    pos = np.full(c.pos.shape, -1, np.int32)
    for b, n in enumerate(c.lens):
        p, at = co.slots(c.table_np[b], int(n), c.page)
        for g in range(c.Hkv):
            x = seen[b] - n + np.arange(n)
            pos[p, at, g] = r.permutation(x) if mixed else x
    return pos


@pytest.mark.parametrize("mixed", [False, True])
@pytest.mark.parametrize("sinks,recent,budget", [(4, 300, 256), (0, 2000, 100), (10, 5, 8), (3, 1, 1), (0, 40, 40), (700, 0, 64),
                                                 (2 ** 31 - 1, 0, 33), (0, 2 ** 31 - 1, 33)])
def test_evict_keeps_the_newest(sinks, recent, budget, mixed):
    c = Cache([700, 41, 5000, 9000], page=16, Hkv=2, D=64, seed=budget)
    r = np.random.default_rng(budget)
    seen = c.lens + np.array([0, 3, 100, 1 << 20])
    pos = _numbered(c, r, seen, mixed)
    w = r.random(c.weight.shape).astype(np.float32)
    w[r.random(w.shape) < 0.2] = np.inf            # no weight outranks them
    left = _trim(c, w, pos, seen, budget, sinks=sinks, recent=recent)
    for b, p in enumerate(left):
        if len(p) == budget and recent >= 1:       # the token that was just appended, and all that are protected like it
            for g in range(2):
                want = np.arange(seen[b] - min(budget, recent, int(c.lens[b])), seen[b])
                assert np.isin(want, p[:, g]).all()


def test_evict_ages_that_count_alike():
    """Numbers past tokens_seen, and ages at the end of what is told apart: the lower slots."""
    c = Cache([900], page=16, Hkv=2, D=64, seed=11)
    r = np.random.default_rng(12)
    seen = np.array([1 << 30], np.int32)
    age = r.choice([-5, -1, 0, 1, 255, 256, 65535, 65536, (1 << 23) - 3, (1 << 23) - 2, (1 << 23) - 1, 1 << 23, 1 << 29], c.pos.shape)
    pos = (int(seen[0]) - 1 - age).astype(np.int32)
    for budget in (20, 200, 500, 800):
        _trim(c, r.random(c.weight.shape).astype(np.float32), pos, seen, budget, recent=2 ** 31 - 1)


# ------------------------------------------------------------------ documents in a cache that is trimmed
@pytest.mark.parametrize("fp8", [False, True])
def test_documents_and_eviction(fp8):
    """What no later token may see leaves first, marked by NaN; then decoding needs no kv_start, and sees what the
    document's own cache, trimmed alike, would show."""
    lens, start, budget, recent = np.array([900, 300, 130, 64], np.int32), np.array([400, 0, 66, 0], np.int32), 64, 16
    c = Cache(lens, page=16, Hkv=2, D=64, fp8=fp8, seed=13)
    r = np.random.default_rng(14)
    c.pos.copy_(torch.from_numpy(_numbered(c, r, lens, False)))
    q = torch.randn(4, 8, 64, device="cuda").to(torch.bfloat16)
    scale = 1 / 640 if fp8 else 0.125
    w = c.weight.cpu().numpy()
    for b in range(4):                             # by the table and the starts, as a program does it
        p, at = co.slots(c.table_np[b], int(start[b]), 16)
        w[p, at] = np.nan
    host, pos = c.host(), c.pos.cpu().numpy()
    c.weight.copy_(torch.from_numpy(w))
    new, st = T.cache_evict(*c.args(), c.weight, c.pos, c.kv_len, budget=budget, recent=recent, **c.exps())
    _status(st)
    got = c.pos.cpu().numpy()
    for b in range(4):
        p, at = co.slots(c.table_np[b], int(new[b]), 16)
        assert (got[p, at] >= start[b]).all()      # the document's tokens alone
    o, lse, st = T.attn_decode(q, c.k, c.v, c.table, new, softmax_scale=scale, **c.exps())
    _status(st)
    # the document's slots alone, numbered from its first, in pages of one slot
    for b in range(4):
        n = int(lens[b] - start[b])
        p, at = (x[start[b]:] for x in co.slots(c.table_np[b], int(lens[b]), 16))
        doc = {k: None if x is None else x[p, at][:, None] for k, x in host.items()}
        table = np.arange(n)[None]
        doc, dw, dp, m = co.evict(doc, table, [n], w[p, at][:, None], pos[p, at][:, None], [int(lens[b])], budget, 0, recent)
        ref = co.decode(q[b:b + 1].double().cpu().numpy(), doc, table, m, scale=np.float32(scale))
        assert np.all(np.abs(o[b:b + 1].double().cpu().numpy() - ref["o"]) <= ref["tol_o"])
        assert np.all(np.abs(lse[:, b:b + 1].double().cpu().numpy() - ref["lse"]) <= ref["tol_lse"])
        p2, at2 = co.slots(c.table_np[b], int(new[b]), 16)
        for g in range(2):
            assert sorted(got[p2, at2, g]) == sorted(dp[:int(m[0]), 0, g])


# ------------------------------------------------------------------ tables for sequences that may come
@pytest.mark.parametrize("slots,Hkv,lens", [(131072, 16, [2000, 0, 1, 512, 513, 2100] * 3), (1 << 20, 2, [9000, 511, 600]),
                                            (40000, 4, [700, 3000] * 20)])
def test_tables_far_wider_than_the_sequences(slots, Hkv, lens):
    """Grids and shared memory go by the table's width, work by the lengths: results as with a tight table."""
    wide = Cache(lens, page=16, Hkv=Hkv, D=64, seed=15, wide=slots // 16)
    r = np.random.default_rng(16)
    w, pos = r.random(wide.weight.shape).astype(np.float32), _numbered(wide, r, wide.lens, True)
    wide.weight.copy_(torch.from_numpy(w)), wide.pos.copy_(torch.from_numpy(pos))
    tight = wide.table[:, :-(-max(lens) // 16)].contiguous()
    q = torch.randn(len(lens), 2 * Hkv, 64, device="cuda").to(torch.bfloat16)
    outs = []
    for table in (tight, wide.table):
        wo = torch.full_like(wide.weight, -3.0)
        o, lse, st = T.attn_decode(q, wide.k, wide.v, table, wide.kv_len, weight=wide.weight, weight_out=wo)
        _status(st)
        outs.append((o, lse, wo))
    # (the cut goes by the lengths, and so does the order of sums)
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    _trim(wide, w, pos, wide.lens, 512, sinks=2, recent=100)


# ------------------------------------------------------------------ weights that lie close together
@pytest.mark.parametrize("close", [2, 7, 8, 127, 128, 129, 130, 500, 1024, 1025, 3000])
def test_evict_close_weights(close):
    """Around the threshold `close` weights with the same upper half, half of them kept; some equal, spread over the slots."""
    lens, budget = [9000, 5200], 2048
    c = Cache(lens, page=16, Hkv=2, D=64, seed=close)
    r = np.random.default_rng(close)
    w = np.zeros(c.weight.shape, np.float32)
    low = np.float32(1.0).view(np.int32)
    for b, n in enumerate(lens):
        p, at = co.slots(c.table_np[b], n, 16)
        for g in range(2):
            near = (low + r.integers(0, 1 << 16, close) // (1 << (4 * g)) * (1 << (4 * g))).astype(np.int32).view(np.float32)
            above = budget - close // 2 if close // 2 < budget else 0
            x = np.concatenate([r.uniform(2, 60, above), near, r.uniform(0.01, 0.9, n - above - close)])
            w[p, at, g] = r.permutation(x)
    _trim(c, w, _numbered(c, r, c.lens, True), c.lens, budget)
