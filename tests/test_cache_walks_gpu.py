"""The paged cache's kernels in their steady state: blocks that walk many units of
several items, warps that refill their rings, joins with several heads a block,
appends of many rows a block.  Against plain forms in 64 bits, everywhere."""

import numpy as np
import pytest
import torch

import cache_plain64 as plain
from cache_testutil import FP8, layout, slotwise
from packed_sequence_context_gb300 import thd_attn as T

pytestmark = pytest.mark.gpu

MOST_BLOCKS = 512                                  # of a decode launch, on any GPU


@pytest.fixture(scope="module", autouse=True)
def _lib(thd_lib):
    return thd_lib


def _i32(x):
    return None if x is None else torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _status(st, want=0):
    torch.cuda.synchronize()
    assert int(st.item()) == want


class Pool:
    """A cache of random rows made on the device; what no sequence holds is NaN."""

    def __init__(self, lens, page, Hkv, D, fp8, first, seed):
        self.rng = r = np.random.default_rng(seed)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.lens, self.page, self.fp8 = np.asarray(lens, np.int32), page, fp8
        self.table_np, pages = layout(r, lens, page)
        self.table, self.kv_len = _i32(self.table_np), _i32(self.lens)
        held = torch.zeros((pages, page), dtype=torch.bool, device="cuda")
        for b, n in enumerate(self.lens):
            held[plain.places(self.table[b], int(n), page)] = True
        make = lambda dt, tail=(): slotwise(pages, page, Hkv, dt, first, tail=tail)  # noqa: E731
        self.exps = {}
        for name in ("k", "v"):
            x = make(FP8 if fp8 else torch.bfloat16, (D,))
            for p0 in range(0, pages, 256):        # (a piece at a time: the numbers are fp32 at first)
                y = torch.randn(x[p0:p0 + 256].shape, generator=g, device="cuda") * (80 if fp8 else 1)
                x[p0:p0 + 256] = y.clamp_(-448, 448).to(x.dtype)
            if fp8:
                x.view(torch.uint8)[~held] = 0x7f
                e = make(torch.uint8)
                s = 3 if name == "v" else 1
                e.copy_(torch.randint(121 - s, 122 + s, e.shape, generator=g, device="cuda", dtype=torch.uint8))
                e[~held] = 255
                self.exps[name + "_exp"] = e
            else:
                x[~held] = float("nan")
            setattr(self, name, x)
        self.weight = make(torch.float32)
        self.weight.copy_(torch.rand(self.weight.shape, generator=g, device="cuda"))
        self.pos = make(torch.int32)
        self.pos.copy_(torch.randint(0, 1 << 14, self.pos.shape, generator=g, device="cuda", dtype=torch.int32))

    def args(self):
        return self.k, self.v, self.table, self.kv_len


def _ragged(seed, seqs, lo, hi):
    n = np.random.default_rng(seed).integers(lo, hi + 1, seqs)
    n[seqs // 3], n[seqs // 2], n[-1] = 0, 1, 0    # nothing, and next to nothing, in the middle
    return n


# every page size: smaller than a tile of rows, odd, larger; every form of a work item (8, 16, 32 heads) with both
# widths and types; bias, cap, documents and weights among them
WALKS = [
    # fp8, D, G, Hkv, page, heads_first, seqs, lo, hi, what
    (False, 64, 8, 4, 24, False, 60, 1200, 3000, ""), (False, 64, 16, 6, 8, True, 40, 1500, 3000, "w"),
    (False, 64, 32, 8, 64, False, 40, 1500, 3000, "d"), (False, 128, 8, 4, 16, True, 60, 1200, 3000, "wd"),
    (False, 128, 16, 4, 100, False, 60, 1200, 3000, "c"), (False, 128, 32, 8, 7, True, 40, 1500, 3000, "wb"),
    (True, 64, 8, 4, 16, False, 60, 1200, 3000, "wcbd"), (True, 64, 16, 6, 40, True, 40, 1500, 3000, ""),
    (True, 64, 32, 8, 24, True, 40, 1500, 3000, "w"), (True, 128, 8, 4, 64, True, 60, 1200, 3000, "b"),
    (True, 128, 16, 4, 1, False, 60, 1200, 3000, "d"), (True, 128, 32, 8, 32, False, 40, 1500, 3000, "wcbd"),
    # several runs of heads an item, one head each, few kv heads, uneven lengths
    (False, 128, 40, 4, 128, False, 40, 1500, 3000, "w"), (True, 128, 3, 5, 256, False, 40, 2000, 4000, "w"),
    (False, 64, 1, 16, 64, True, 40, 1000, 2000, "wd"), (True, 64, 20, 4, 24, False, 64, 1, 6000, "b"),
]


@pytest.mark.parametrize("fp8,D,G,Hkv,page,first,seqs,lo,hi,what", WALKS)
def test_decode_walks(fp8, D, G, Hkv, page, first, seqs, lo, hi, what):
    lens = _ragged(D + G, seqs, lo, hi)
    heads = 8 if G <= 8 else 16 if G <= 16 else 32
    runs = -(-G // heads)
    start = None
    if "d" in what:
        start = np.random.default_rng(1).integers(-2, np.maximum(lens // 3, 1))
        start[5] = lens[5]                         # all hidden
    seen = [max(0, n - (0 if start is None else max(0, start[b]))) for b, n in enumerate(lens)]
    units = sum(-(-n // 64) for n in seen) * Hkv * runs
    # a block's share: several units of 64 slots for each of its four warps, so that stages are filled again, and the
    # end of one item and the beginning of the next in many
    assert units >= 8 * MOST_BLOCKS and units / (seqs * Hkv * runs) >= 8
    items = seqs * Hkv * runs
    assert items >= 160
    c = Pool(lens, page, Hkv, D, fp8, first, seed=D + G + page)
    q = torch.randn(seqs, Hkv * G, D, device="cuda").to(torch.bfloat16)
    scale = float(np.float32((1 / 80 if fp8 else 1) * D ** -0.5))
    cap = 20.0 if "c" in what else 0.0
    slopes = torch.exp2(-8.0 * torch.arange(1, Hkv * G + 1, device="cuda") / (Hkv * G)) if "b" in what else None
    kw = dict(pos=c.pos, seen=list(lens + (1 << 14))) if "b" in what else {}
    ref = plain.decode(q, c.k, c.v, c.table, lens, scale=scale, softcap=cap, slopes=slopes, start=start,
                       weight=c.weight if "w" in what else None, **c.exps, **kw)
    ws = torch.full((T.thd_decode_workspace_size(seqs, Hkv * G, Hkv, D, c.table.shape[1] * page, "w" in what),), 0xff,
                    dtype=torch.uint8, device="cuda")
    outs = []
    for fill in (0xff, 0x3f):                      # what a workspace held before shows in no bit
        ws.fill_(fill)
        wo = torch.full_like(c.weight, -7.0) if "w" in what else None
        o, lse, st = T.attn_decode(q, *c.args(), softmax_scale=scale, softcap=cap, dist_slopes=slopes, kv_start=_i32(start),
                                   pos=c.pos if kw else None, tokens_seen=_i32(kw["seen"]) if kw else None, workspace=ws,
                                   weight=c.weight if "w" in what else None, weight_out=wo, **c.exps)
        _status(st)
        outs.append((o, lse, wo))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert ((o.double() - ref["o"]).abs() <= ref["tol_o"]).all()
    inf = torch.isinf(ref["lse"])
    assert inf.any() and torch.equal(lse.double()[inf], ref["lse"][inf])
    assert ((lse.double() - ref["lse"]).abs() <= ref["tol_lse"])[~inf].all()
    if "w" in what:
        assert torch.equal(outs[0][2], outs[1][2])
        m = ref["tol_weight"] > 0
        assert (wo[~m] == -7.0).all()
        assert ((wo.double() - ref["weight"]).abs() <= ref["tol_weight"])[m].all()


@pytest.mark.parametrize("fp8,G", [(False, 4), (True, 32)])
def test_decode_one_long_sequence(fp8, G):
    """Every block inside one item, several times around its ring."""
    n = 262144 + 37
    assert -(-n // 64) >= 8 * MOST_BLOCKS
    c = Pool([n, 0, 3], 48, 1, 64, fp8, False, seed=5)
    q = torch.randn(3, G, 64, device="cuda").to(torch.bfloat16)
    scale = 1 / 640 if fp8 else 0.125
    ref = plain.decode(q, c.k, c.v, c.table, [n, 0, 3], scale=scale, **c.exps)
    o, lse, st = T.attn_decode(q, *c.args(), softmax_scale=scale, **c.exps)
    _status(st)
    assert ((o.double() - ref["o"]).abs() <= ref["tol_o"]).all()
    assert ((lse.double() - ref["lse"]).abs() <= ref["tol_lse"])[:, [0, 2]].all() and torch.isinf(lse[:, 1]).all()


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows,Hkv,D,page,first,per", [
    (2433, 3, 128, 16, False, 4), (5000, 5, 64, 24, True, 2), (5001, 16, 128, 64, True, 900), (17003, 16, 128, 1, False, 3),
    (30011, 7, 64, 100, False, 40), (160003, 1, 64, 32, True, 2000)])
def test_append_many_rows_a_block(rows, Hkv, D, page, first, per, fp8):
    """Blocks with several rows of several sequences: the offsets' order, sequences of no row, the end of the last
    sequence, a last block that is not full; a row whose page is bad keeps to itself."""
    a_block = -(-rows // (16 * torch.cuda.get_device_properties(0).multi_processor_count))
    assert a_block >= 2
    r = np.random.default_rng(rows)
    new = []
    while sum(new) < rows - 50:
        new.append(int(r.integers(0, per + 1)))
    m = sum(new)
    assert m < rows + per
    B = len(new)
    old = r.integers(0, 40, B)
    lens = np.array(new) + old
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    table_np, pages = layout(r, lens, page)
    make = lambda dt, tail=(): slotwise(pages, page, Hkv, dt, first, tail=tail)  # noqa: E731
    kc, vc = (make(FP8 if fp8 else torch.bfloat16, (D,)) for _ in range(2))
    ke, ve = (make(torch.uint8) if fp8 else None for _ in range(2))
    w, pos = make(torch.float32), make(torch.int32)
    for t in (kc, vc, ke, ve):
        if t is not None:
            t.view(torch.uint8).fill_(0x2a)        # what no row goes to stays
    w.fill_(-3.0), pos.fill_(-3)
    total = m + 61                                 # rows behind the last sequence
    x = torch.randn(total, 3 * Hkv * D, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-40, 40, (total, 1), generator=g, device="cuda").float())
    x = x.to(torch.bfloat16)
    x[::97, Hkv * D:] = 0
    x[5::1013, 2 * Hkv * D + 3] = float("nan")
    k, v = x[:, Hkv * D:2 * Hkv * D].view(total, Hkv, D), x[:, 2 * Hkv * D:].view(total, Hkv, D)
    cu = np.concatenate([[0], np.cumsum(new)])
    seen = lens + 9
    table = _i32(table_np)
    want = plain.append(k, v, cu, table, lens, page, fp8=fp8, seen=seen)
    # bad pages, one inside the walk and one in the last sequence that has rows
    bad = torch.zeros(m, dtype=torch.bool, device="cuda")
    last = max(b for b in range(B) if new[b])
    mid = next(b for b in range(B // 2, B) if new[b])
    broken = table.clone()
    for b in {mid, last}:
        i = (int(lens[b]) - 1) // page
        broken[b, i] = pages + 3 if b == mid else -2
        t = torch.arange(m, device="cuda")
        j = int(lens[b]) - (int(cu[b + 1]) - t)
        bad |= (t >= int(cu[b])) & (t < int(cu[b + 1])) & (j // page == i)
    exps = {"k_exp": ke, "v_exp": ve} if fp8 else {}
    arrays = [t for t in (kc, vc, ke, ve, w, pos) if t is not None]
    untouched = [t.clone() for t in arrays]
    for tab, left in ((broken, bad), (table, torch.zeros_like(bad))):
        st = T.cache_append(k, v, kc, vc, tab, _i32(lens), cu_seqlens=_i32(cu), weight=w, pos=pos, tokens_seen=_i32(seen), **exps)
        _status(st, T.THD_DEV_ERR_PAGE if left.any() else 0)
        p, at = want["p"][~left], want["at"][~left]
        want_of = [want["k"], want["v"]] + ([want["k_exp"], want["v_exp"]] if fp8 else [])
        want_of += [torch.zeros(m, Hkv, device="cuda"), want["pos"].to(torch.int32)[:, None].expand(m, Hkv)]
        raw = lambda t: t.view(torch.uint8) if t.dtype is FP8 else t.view(torch.int16) if t.dtype is torch.bfloat16 else t  # noqa: E731
        for t, y, z in zip(arrays, want_of, untouched):
            ref = raw(z).clone()
            ref[p, at] = raw(y.contiguous())[~left]
            nan = torch.zeros((), dtype=torch.bool, device="cuda")
            if t.dtype is FP8:                     # (NaN has several codes)
                nan = ((ref & 0x7f) == 0x7f) & ((raw(t) & 0x7f) == 0x7f)
            elif t.dtype is torch.bfloat16:
                nan = ((ref & 0x7fff) > 0x7f80) & ((raw(t) & 0x7fff) > 0x7f80)
            assert (nan | (raw(t) == ref)).all()
