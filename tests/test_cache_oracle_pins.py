"""The cache's oracles against hand-made values and against the other oracles."""

import numpy as np
import pytest
import torch

from oracle import cache_oracle as co
from oracle import score_oracle as so


def test_e4m3_numbers_are_torchs():
    codes = np.arange(127, dtype=np.uint8)
    assert np.array_equal(torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy(), co.E4M3)
    x = np.random.default_rng(1).uniform(-448, 448, 20000)
    x[:127], x[127:253] = co.E4M3, (co.E4M3[1:] + co.E4M3[:-1]) / 2        # the numbers and the ties
    got = torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(co.to_e4m3(x.astype(np.float32)), got)


@pytest.mark.parametrize("row,e", [([0.0, 0.0], 127), ([448.0, 1.0], 127), ([449.0, 0.0], 128), ([-896.0, 3.0], 128),
                                   ([224.0, 1.0], 126), ([225.0, 1.0], 127), ([1.0, -0.5], 119), ([2.0 ** -60, 0.0], 67),
                                   ([np.inf, 1.0], 255), ([np.nan, 1.0], 255), ([1.75, 0], 119), ([1.76, 0], 120)])
def test_row_exponent(row, e):
    assert co.row_exponent(np.array(row)) == e


def test_decode_is_a_sequences_last_row():
    r = np.random.default_rng(2)
    n, Hq, Hkv, D, page = 37, 4, 2, 8, 5
    k, v, q = r.standard_normal((n, Hkv, D)), r.standard_normal((n, Hkv, D)), r.standard_normal((n, Hq, D))
    table = np.array([[3, 0, 7, 1, 2, 9, 4, 8]])
    cache = {"k": np.zeros((10, page, Hkv, D)), "v": np.zeros((10, page, Hkv, D)), "k_exp": None, "v_exp": None}
    cache, w, pos = co.append(cache, k, v, [0, n], table, [n], weight=np.ones((10, page, Hkv)),
                              pos=np.zeros((10, page, Hkv), int))
    p, at = co.slots(table[0], n, page)
    assert np.array_equal(pos[p, at, 1], np.arange(n)) and not w[p, at].any() and w.sum() == (50 - n) * Hkv
    slopes = np.array([0.5, 0.25, 0.1, 0.0])
    doc = np.repeat([0, 1], [12, 25])
    cu = np.array([0, n])
    ref = so.score(q, k, v, cu, cu, cu, cu, causal=1, scale=0.3, softcap=4.0, slopes=slopes, doc_q=doc, doc_k=doc)
    got = co.decode(q[-1:], cache, table, [n], scale=0.3, softcap=4.0, slopes=slopes, start=[12], pos=pos, weight=w * 0)
    assert np.allclose(got["o"][0], ref["o"][-1], atol=1e-12) and np.allclose(got["lse"][:, 0], ref["lse"][:, -1], atol=1e-12)
    assert np.allclose(got["weight"][p, at].sum(), Hq) and not got["weight"][p[:12], at[:12]].any()


def test_evict_by_hand():
    page, n = 2, 7
    table = np.array([[2, 0, 1, 3]])
    k = np.zeros((4, page, 1, 1))
    p, at = co.slots(table[0], n, page)
    k[p, at, 0, 0] = np.arange(n)
    cache = {"k": k, "v": 10 * k, "k_exp": None, "v_exp": None}
    w, pos = np.zeros((4, page, 1)), np.zeros((4, page, 1), int)
    w[p, at, 0] = [5, 1, 0, 3, 3, 3, 9]          # ties at 3: slots 3 and 4 stay, 5 goes
    pos[p, at, 0] = [4, 6, 0, 5, 7, 8, 9]        # slot 2 holds the first token: kept
    out, wo, po, m = co.evict(cache, table, [n], w, pos, [10], 5, sinks=1)
    assert list(out["k"][p, at, 0, 0][:5]) == [0, 6, 2, 3, 4] and list(out["v"][p, at, 0, 0][:5]) == [0, 60, 20, 30, 40]
    assert list(wo[p, at, 0][:5]) == [5, 9, 0, 3, 3] and list(po[p, at, 0][:5]) == [4, 9, 0, 5, 7] and list(m) == [5]
    out, *_ , m = co.evict(cache, table, [n], w, pos, [10], 7)
    assert np.array_equal(out["k"], k) and list(m) == [7]
