"""Scored attention under a cap that bounds the scores: P without a running
maximum reaches from 2^-80 to 2^80, and v may hold 0 and magnitudes from 2^-40
to 2^30.  Every score at -cap against the smallest values, and at +cap against
the largest, 40,000 keys of one sign (the row sum's largest products)."""

import numpy as np
import pytest
import torch

from packed_sequence_context_gb300 import thd_attn as T


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", [T.THD_FWD_KERNEL_SINGLE, T.THD_FWD_KERNEL_DUAL])
@pytest.mark.parametrize("sign,exponent", [(-1.0, -40), (1.0, 29)])
def test_values_at_both_ends(thd_lib, kernel, sign, exponent):
    n, D, cap = 40000, 64, 55.0
    g = torch.Generator().manual_seed(11)
    q = torch.full((n, 1, D), 16.0).bfloat16()
    k = torch.full((n, 1, D), 16.0 * sign).bfloat16()     # x = 2048: tanh is 1 to the last bit
    v = ((1 + torch.rand(n, 1, D, generator=g)) * 2.0 ** exponent).bfloat16()
    v[:, :, 0] = 0
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    T.thd_test_select_fwd_kernel(kernel)
    try:
        o, lse, st = T.attn_score_fwd(q.cuda(), k.cuda(), v.cuda(), cu, cu, softcap=cap, cp_size=4)
        T.check_status(st)
    finally:
        T.thd_test_select_fwd_kernel(0)
    want = torch.cumsum(v.double(), 0) / torch.arange(1, n + 1, dtype=torch.float64)[:, None, None]
    # every P is the same number, rounded to bf16 once (2^-8); 40,000 additions in fp32 (at most n 2^-24); O's
    # rounding (2^-8)
    err = (o.double().cpu() - want).abs()
    assert torch.all(err <= (2 * 2.0 ** -8 + n * 2.0 ** -24 + 2.0 ** -16) * want)
    assert not o[:, :, 0].any()
    lse_want = sign * cap + np.log(np.arange(1, n + 1))
    # the score (cap 2^-20) and the sum's logarithm
    assert np.abs(lse.double().cpu().numpy()[0] - lse_want).max() <= cap * 2.0 ** -20 + 2.0 ** -15

