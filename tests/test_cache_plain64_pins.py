"""The cache's plain forms without loops against the oracle's."""

import numpy as np
import pytest
import torch

import cache_plain64 as plain
from oracle import cache_oracle as co

FP8 = torch.float8_e4m3fn


def _cache(rng, pages, page, Hkv, D, fp8):
    x = [torch.from_numpy(rng.standard_normal((pages, page, Hkv, D)) * (80 if fp8 else 1)).float().clamp(-448, 448) for _ in "kv"]
    e = [torch.from_numpy(rng.integers(118, 125, (pages, page, Hkv)).astype(np.uint8)) if fp8 else None for _ in "kv"]
    return [t.to(FP8 if fp8 else torch.bfloat16) for t in x], e


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("everything", [False, True])
def test_decode(fp8, everything):
    r = np.random.default_rng(3)
    B, Hkv, G, D, page, pages = 4, 2, 3, 8, 5, 40
    (k, v), (ke, ve) = _cache(r, pages, page, Hkv, D, fp8)
    table = torch.from_numpy(r.permutation(pages)[:B * 8].reshape(B, 8).astype(np.int32))
    lens = [37, 0, 1, 20]
    q = torch.from_numpy(r.standard_normal((B, Hkv * G, D))).to(torch.bfloat16)
    v.view(torch.uint8)[table[0, 1], 2] = 0
    kw = {}
    if everything:
        kw = dict(softcap=4.0, slopes=np.array([.5, .25, .1, 0, .3, .2], np.float32), start=[12, 0, 5, -3], seen=[100, 9, 8, 90])
    pos = r.integers(0, 90, (pages, page, Hkv))
    w = r.random((pages, page, Hkv))
    host = {"k": k.double().numpy(), "v": v.double().numpy(), "k_exp": ke and None, "v_exp": None} if not fp8 else \
        {"k": k.double().numpy(), "v": v.double().numpy(), "k_exp": ke.numpy().astype(int), "v_exp": ve.numpy().astype(int)}
    want = co.decode(q.double().numpy(), host, table.numpy(), lens, scale=0.01, pos=pos if everything else None, weight=w, **kw)
    if everything:
        kw["slopes"] = torch.from_numpy(kw["slopes"])
    got = plain.decode(q, k, v, table, lens, scale=0.01, pos=torch.from_numpy(pos) if everything else None,
                       weight=torch.from_numpy(w), k_exp=ke, v_exp=ve, **kw)
    for n in want:
        assert np.allclose(got[n].numpy(), want[n], rtol=1e-9, atol=1e-15), n


@pytest.mark.parametrize("fp8", [False, True])
def test_append(fp8):
    r = np.random.default_rng(4)
    Hkv, D, page, pages = 3, 16, 4, 30
    new, lens, seen = [0, 5, 1, 0, 12], [3, 7, 1, 0, 13], [3, 9, 4, 0, 20]
    cu = np.concatenate([[0], np.cumsum(new)])
    table = torch.from_numpy(r.permutation(pages)[:25].reshape(5, 5).astype(np.int32))
    k, v = (torch.from_numpy(r.standard_normal((20, Hkv, D)) * 2.0 ** r.integers(-70, 60, (20, Hkv, 1))).to(torch.bfloat16) for _ in "kv")
    k[3], k[4, 1, 2], v[7, 0, 0] = 0, float("inf"), float("nan")
    zero = lambda dt=np.float64, *s: np.zeros((pages, page, Hkv, *s), dt)  # noqa: E731
    cache = {"k": zero(np.float64, D), "v": zero(np.float64, D), "k_exp": zero(int) if fp8 else None, "v_exp": zero(int) if fp8 else None}
    want, _, pos = co.append(cache, k.double().numpy(), v.double().numpy(), cu, table.numpy(), lens, seen, zero(), zero(int))
    got = plain.append(k, v, cu, table, lens, page, fp8=fp8, seen=seen)
    p, at = got["p"].numpy(), got["at"].numpy()
    for n in ("k", "v"):
        assert np.array_equal(got[n].double().numpy(), want[n][p, at], equal_nan=True)
        if fp8:
            assert np.array_equal(got[n + "_exp"].numpy(), want[n + "_exp"][p, at])
    assert np.array_equal(np.broadcast_to(got["pos"].numpy()[:, None], pos[p, at].shape), pos[p, at])
