"""Arrays that are broadcast along pages, slots or heads: taken where a call only
reads them, or writes one number for all heads; refused where it writes more."""

import numpy as np
import pytest
import torch

from packed_sequence_context_gb300 import thd_attn as T
from test_cache_refusals import _append, _decode, _evict, _kv

E4M3 = {"dtype": T.THD_DTYPE_E4M3, "k_exp": 16, "v_exp": 16}
FULL = {"kv_stride": (2048, 128, 64), "exp_stride": (32, 2, 1), "weight_stride": (32, 2, 1), "pos_stride": (32, 2, 1)}


@pytest.mark.parametrize("at", [0, 1, 2])
@pytest.mark.parametrize("f,over,array,kw", [
    (_append, {}, "kv_stride", {}), (_append, E4M3, "exp_stride", {}), (_decode, {}, "weight_stride", {"wi": 16, "wo": 16}),
    (_evict, {}, "kv_stride", {}), (_evict, E4M3, "exp_stride", {}), (_evict, {}, "weight_stride", {}), (_evict, {}, "pos_stride", {})])
def test_written_arrays_that_share_places(thd_lib, f, over, array, kw, at):
    s = list(FULL[array])
    s[at] = 0
    n = T.thd_launch_count()
    assert f(_kv(**{**FULL, **over, array: s}), **kw) == T.THD_ERR_INVALID_ARG
    assert T.thd_launch_count() == n


@pytest.mark.gpu
def test_one_number_for_all_heads(thd_lib):
    """pos as an expanded array: set by append, read by decode's distances; and dimensions of one element with stride 0."""
    r = np.random.default_rng(5)
    pages, page, Hkv, D, n = 7, 16, 4, 64, 70
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    kc, vc = (torch.zeros(pages, page, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table, kv_len = i32(r.permutation(pages)[None, :5]), i32([n])
    k, v = (torch.randn(n, Hkv, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    one = torch.full((pages, page, 1), -1, dtype=torch.int32, device="cuda")
    each = torch.full((pages, page, Hkv), -1, dtype=torch.int32, device="cuda")
    q = torch.randn(1, 8, D, device="cuda").to(torch.bfloat16)
    slopes = torch.rand(8, device="cuda")
    outs = []
    for pos in (one.expand(-1, -1, Hkv), each):
        st = T.cache_append(k, v, kc, vc, table, kv_len, cu_seqlens=i32([0, n]), pos=pos, tokens_seen=i32([n + 30]))
        o, lse, _ = T.attn_decode(q, kc, vc, table, kv_len, dist_slopes=slopes, pos=pos, tokens_seen=i32([n + 30]), dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        outs.append((o, lse))
    assert torch.equal(one.expand(-1, -1, Hkv), each)
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    w = torch.zeros(pages, page, Hkv, device="cuda")
    with pytest.raises(T.ThdError):
        T.cache_evict(kc, vc, table, kv_len, w, one.expand(-1, -1, Hkv), i32([n + 30]), budget=32)
