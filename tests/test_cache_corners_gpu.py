"""Corners of the paged cache: bad pages of sequences that nothing leaves."""

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
