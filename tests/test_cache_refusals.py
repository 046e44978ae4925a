"""What the cache's calls refuse before any launch: the C entries by their
arguments, the helpers by their tensors; and where the helpers allocate.  No
GPU."""

import copy

import pytest
import torch

from packed_sequence_context_gb300 import thd_attn as T
from test_row_refusals import FakeLib, lib  # noqa: F401
from test_streams import FakeStream, _tensors, fakes  # noqa: F401


# ------------------------------------------------------------------ C entries
def _kv(**over):
    c = T.KvCache(k=256, v=256, block_table=16, kv_len=16, num_pages=10, table_stride=4, page_size=16, max_pages=4, B=2,
                  Hkv=2, D=64, dtype=T.THD_DTYPE_BF16)
    c.kv_stride[:] = (2048, 128, 64)
    for n, v in over.items():
        if n.endswith("stride") and n != "table_stride":
            getattr(c, n)[:] = v
        else:
            setattr(c, n, v)
    return c


BAD = [({"k": 0}, 1), ({"v": None}, 1), ({"k": 264}, 1), ({"block_table": 0}, 1), ({"kv_len": 18}, 1), ({"num_pages": 0}, 1),
       ({"num_pages": 1 << 31}, 1), ({"page_size": 0}, 1), ({"max_pages": 0}, 1), ({"B": 0}, 1), ({"B": 1 << 24}, 1),
       ({"Hkv": 0}, 1), ({"table_stride": 3}, 1), ({"D": 96}, 2), ({"dtype": T.THD_DTYPE_FP32}, 2),
       ({"page_size": 1 << 29}, 2), ({"kv_stride": (2048, 124, 64)}, 1), ({"kv_stride": (-2048, 128, 64)}, 1),
       ({"k_exp": 16}, 1), ({"dtype": T.THD_DTYPE_E4M3}, 1), ({"dtype": T.THD_DTYPE_E4M3, "k_exp": 16}, 1),
       ({"dtype": T.THD_DTYPE_E4M3, "k_exp": 16, "v_exp": 16, "kv_stride": (2048, 128, 72)}, 1), ({"weight_stride": (-1, 1, 1)}, 1)]


def _append(c=None, **o):
    a = dict(k=256, v=256, ks=128, vs=128, T=2, cu=None, w=None, pos=None, seen=None, st=16) | o
    return T.thd_cache_append(c or _kv(), a["k"], a["v"], a["ks"], a["vs"], a["T"], a["cu"], a["w"], a["pos"], a["seen"],
                              a["st"], stream=0)


def _decode(c=None, **o):
    a = dict(q=256, qs=256, o=256, lse=16, Hq=4, scale=0.1, cap=0.0, slopes=None, start=None, pos=None, seen=None, wi=None,
             wo=None, ws=256, n=1 << 30, st=16) | o
    return T.thd_attn_decode(c or _kv(), a["q"], a["qs"], a["o"], a["lse"], a["Hq"], a["scale"], a["cap"], a["slopes"],
                             a["start"], a["pos"], a["seen"], a["wi"], a["wo"], a["ws"], a["n"], a["st"], stream=0)


def _evict(c=None, **o):
    a = dict(wi=16, wo=16, pi=16, po=16, seen=16, budget=8, sinks=0, recent=0, new=32, ws=256, n=1 << 30, st=16) | o
    return T.thd_cache_evict(c or _kv(), a["wi"], a["wo"], a["pi"], a["po"], a["seen"], a["budget"], a["sinks"], a["recent"],
                             a["new"], a["ws"], a["n"], a["st"], stream=0)


@pytest.mark.parametrize("over,code", BAD, ids=lambda x: str(x))
def test_caches(thd_lib, over, code):
    n = T.thd_launch_count()
    assert [f(_kv(**over)) for f in (_append, _decode, _evict)] == [code] * 3
    assert T.thd_launch_count() == n


@pytest.mark.parametrize("f,over,code", [
    (_append, {"k": None}, 1), (_append, {"k": 264}, 1), (_append, {"T": 3}, 1), (_append, {"T": -1}, 1), (_append, {"ks": 120}, 1),
    (_append, {"vs": 132}, 1), (_append, {"st": None}, 1), (_append, {"st": 18}, 1), (_append, {"pos": 2}, 1),
    (_append, {"T": 1 << 31, "cu": 16}, 1),
    (_decode, {"q": None}, 1), (_decode, {"q": 258}, 1), (_decode, {"qs": 128}, 1), (_decode, {"qs": 257}, 1), (_decode, {"o": 264}, 1),
    (_decode, {"lse": None}, 1), (_decode, {"Hq": 3}, 1), (_decode, {"Hq": 0}, 1), (_decode, {"Hq": 2 * 513}, 2),
    (_decode, {"scale": 0.0}, 1), (_decode, {"scale": -1.0}, 1), (_decode, {"scale": float("nan")}, 1),
    (_decode, {"scale": 3e38}, 1), (_decode, {"cap": -1.0}, 1), (_decode, {"cap": float("inf")}, 1), (_decode, {"cap": 3e38}, 1),
    (_decode, {"scale": 1e-20, "cap": 1e30}, 1), (_decode, {"scale": 1e30, "cap": 1e-20}, 1), (_decode, {"wi": 16}, 1),
    (_decode, {"wo": 16}, 1), (_decode, {"st": None}, 1), (_decode, {"ws": None}, 5), (_decode, {"ws": 264}, 5),
    (_decode, {"n": 100}, 5), (_decode, {"slopes": 2}, 1), (_decode, {"start": 2}, 1),
    (_evict, {"wi": None}, 1), (_evict, {"wo": None}, 1), (_evict, {"pi": None}, 1), (_evict, {"po": 2}, 1), (_evict, {"seen": None}, 1),
    (_evict, {"budget": 0}, 1), (_evict, {"budget": -5}, 1), (_evict, {"sinks": -1}, 1), (_evict, {"recent": -1}, 1),
    (_evict, {"new": None}, 1), (_evict, {"new": 16}, 1), (_evict, {"ws": 128}, 5), (_evict, {"n": 10}, 5), (_evict, {"st": None}, 1)],
    ids=lambda x: getattr(x, "__name__", str(x)))
def test_arguments(thd_lib, f, over, code):
    n = T.thd_launch_count()
    assert f(**over) == code
    assert T.thd_launch_count() == n


def test_no_cache_and_no_rows(thd_lib):
    assert T.thd_cache_append(None, 256, 256, 128, 128, 2, None, None, None, None, 16, stream=0) == T.THD_ERR_INVALID_ARG
    assert _append(T=0, cu=16, k=None, v=None) == T.THD_OK


def test_workspaces(thd_lib):
    f = T.thd_decode_workspace_size
    assert 0 < f(4, 32, 8, 128, 4096, 0) < f(4, 32, 8, 128, 4096, 1)
    assert f(4, 32, 8, 128, 4096, 1) >= 4 * 32 * 4096 * 4
    for bad in ((0, 32, 8, 128, 64), (4, 30, 8, 128, 64), (4, 32, 8, 96, 64), (4, 32, 8, 128, 0), (4, 32, 8, 128, (1 << 30) + 1),
                (4, 513, 1, 128, 64), (4, 0, 8, 64, 64)):
        assert f(*bad, 0) == 0
    g = T.thd_evict_workspace_size
    assert g(4, 8, 4096, 1000) >= 4 * 8 * 1000 * 8 and g(4, 8, 4096, 5000) > 0
    assert g(0, 8, 4096, 10) == g(4, 0, 4096, 10) == g(4, 8, 0, 10) == g(4, 8, 4096, 0) == 0


def test_new_codes_have_texts(thd_lib):
    for code in (T.THD_DEV_ERR_PAGE, T.THD_DEV_ERR_KV_LEN):
        assert T.thd_status_string(code) != "unknown status"


# ------------------------------------------------------------------ helpers
def _ok(fp8=False):
    """Arguments of the three helpers that they take."""
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    z = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    cache = {"k_cache": z(6, 4, 2, 64, dtype=dt), "v_cache": z(6, 4, 2, 64, dtype=dt), "block_table": i(3, 2), "kv_len": i(3)}
    exps = {n: z(6, 4, 2, dtype=torch.uint8) if fp8 else None for n in ("k_exp", "v_exp")}
    bf = lambda *s: z(*s, dtype=torch.bfloat16)  # noqa: E731
    return {
        "append": (T.cache_append, {"k": bf(5, 2, 64), "v": bf(5, 2, 64), **cache, "cu_seqlens": i(4), **exps, "weight": z(6, 4, 2),
                                    "pos": i(6, 4, 2), "tokens_seen": i(3), "dev_status": i(1)}),
        "decode": (T.attn_decode, {"q": bf(3, 4, 64), **cache, **exps, "dist_slopes": z(4), "kv_start": i(3), "pos": i(6, 4, 2),
                                   "tokens_seen": i(3), "weight": z(6, 4, 2), "weight_out": z(6, 4, 2), "out": bf(3, 4, 64),
                                   "lse": z(4, 3), "dev_status": i(1)}),
        "evict": (T.cache_evict, {**cache, "weight": z(6, 4, 2), "pos": i(6, 4, 2), "tokens_seen": i(3), "budget": 3, **exps,
                                  "weight_out": z(6, 4, 2), "pos_out": i(6, 4, 2), "new_len": i(3), "dev_status": i(1)}),
    }


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", ["append", "decode", "evict"])
def test_helpers_take_what_fits(lib, name, fp8):  # noqa: F811
    f, kw = _ok(fp8)[name]
    f(**kw)
    # the other order in memory, and slices
    kw = dict(kw)
    for n in ("k_cache", "v_cache"):
        kw[n] = torch.zeros((6, 2, 4, 64), dtype=kw[n].dtype).transpose(1, 2)
    kw["block_table"] = torch.zeros((3, 9), dtype=torch.int32)[:, 2:4]
    f(**kw)
    assert len([n for n, _ in lib.calls if not n.endswith("_size")]) == 2


def _wrong():
    """(helper, argument, a change that has to be refused)"""
    for name, (_, kw) in _ok(True).items():
        for arg, t in kw.items():
            if not isinstance(t, torch.Tensor):
                continue
            changes = {"type": t.double() if t.dtype != torch.int32 else t.long(), "dimensions": t[None].contiguous(),
                       "size": torch.zeros([s + 1 for s in t.shape], dtype=t.dtype)}
            if arg in ("block_table", "k_cache", "v_cache"):
                changes["layout"] = torch.zeros((*t.shape[:-1], 2 * t.shape[-1]), dtype=t.dtype)[..., ::2]
            for what, x in changes.items():
                yield name, arg, what, x


@pytest.mark.parametrize("name,arg,what,x", list(_wrong()), ids=lambda x: "" if isinstance(x, torch.Tensor) else str(x))
def test_helpers_refuse(lib, name, arg, what, x):  # noqa: F811
    f, kw = _ok(True)[name]
    with pytest.raises(T.ThdError) as e:
        f(**{**kw, arg: x})
    assert e.value.code in (T.THD_ERR_INVALID_ARG, T.THD_ERR_UNSUPPORTED)
    assert not [n for n, _ in lib.calls if not n.endswith("_size")]


@pytest.mark.parametrize("name", ["append", "decode", "evict"])
def test_helpers_refuse_missing_or_needless_exponents(lib, name):  # noqa: F811
    f, kw = _ok(True)[name]
    with pytest.raises(T.ThdError):
        f(**{**kw, "v_exp": None})
    f, kw = _ok(False)[name]
    with pytest.raises(T.ThdError):
        f(**{**kw, "k_exp": torch.zeros((6, 4, 2), dtype=torch.uint8), "v_exp": torch.zeros((6, 4, 2), dtype=torch.uint8)})
    assert not [n for n, _ in lib.calls if not n.endswith("_size")]


@pytest.mark.parametrize("name", ["append", "decode", "evict"])
def test_helpers_allocate_from_the_launch_stream(fakes, name):  # noqa: F811
    lib_, made, recorded = fakes
    f, kw = _ok(True)[name]
    kw = copy.copy(kw)
    for n in ("dev_status", "out", "lse", "new_len"):
        kw.pop(n, None)
    made.clear()
    out = _tensors(f(**kw, stream=FakeStream(64)))
    assert [a[-1] for n, a in lib_.calls if not n.endswith("_size")] == [64]
    assert made and all(h == 64 for h, _ in made)
    for t in out:
        assert recorded.get(t.data_ptr()) == {0}
    for t in kw.values():
        if isinstance(t, torch.Tensor):
            assert recorded.get(t.data_ptr()) == {64}


def test_the_helpers_bytes_are_the_struct(lib, thd_lib):  # noqa: F811
    """What the helpers pack is thd_kv_cache, field by field."""
    import ctypes
    _, kw = _ok(True)["append"]
    kw["k_cache"], kw["v_cache"] = (torch.zeros((6, 2, 4, 64), dtype=torch.float8_e4m3fn).transpose(1, 2) for _ in range(2))
    kw["block_table"] = torch.zeros((3, 9), dtype=torch.int32)[:, 2:4]
    raw = T._cache("x", *(kw[n] for n in ("k_cache", "v_cache", "block_table", "kv_len", "k_exp", "v_exp", "weight")), None,
                   kw["pos"], None)[0]
    assert len(raw) == ctypes.sizeof(T.KvCache)
    c = T.KvCache.from_buffer_copy(raw)
    for field, arg in (("k", "k_cache"), ("v", "v_cache"), ("k_exp", "k_exp"), ("v_exp", "v_exp"), ("block_table", "block_table"),
                       ("kv_len", "kv_len")):
        assert getattr(c, field) == kw[arg].data_ptr(), field
    assert (c.num_pages, c.table_stride, c.page_size, c.max_pages, c.B, c.Hkv, c.D, c.dtype) == (6, 9, 4, 2, 3, 2, 64, T.THD_DTYPE_E4M3)
    assert list(c.kv_stride) == [512, 64, 256] and list(c.exp_stride) == [8, 2, 1] == list(c.weight_stride) == list(c.pos_stride)


def test_dimensions_of_size_one_may_carry_any_stride(lib):  # noqa: F811
    f, kw = _ok(False)["append"]
    one = lambda dt, *tail: torch.zeros((6, 4, 1, *tail), dtype=dt).as_strided((6, 4, 1, *tail), (256, 64, 3, 1)[:3 + len(tail)])  # noqa: E731
    kw = {**kw, "k": kw["k"][:, :1].contiguous(), "v": kw["v"][:, :1].contiguous(), "k_cache": one(torch.bfloat16, 64),
          "v_cache": torch.zeros((6, 4, 1, 64), dtype=torch.bfloat16), "weight": None, "pos": None}
    f(**kw)
    c = T.KvCache.from_buffer_copy(lib.calls[-1][1][0])
    assert list(c.kv_stride) == [256, 64, 0]


def test_one_table_row_for_all(lib):  # noqa: F811
    f, kw = _ok(False)["decode"]
    f(**{**kw, "block_table": torch.zeros((1, 2), dtype=torch.int32).expand(3, 2)})
    assert T.KvCache.from_buffer_copy(lib.calls[-1][1][0]).table_stride == 0
