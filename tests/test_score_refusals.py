"""Scales and caps of scored attention that are floats themselves but not in the
log2 units the kernels take them in: refused on the host (they would turn scores
of 0 into NaN)."""

import pytest
from test_score_gpu import _bwd, _fwd

from packed_sequence_context_gb300 import thd_attn as T


@pytest.mark.parametrize("kw", [{"cap": 3e38, "scale": 1e30}, {"cap": 2.4e38, "scale": 2.4e38}, {"cap": 0.0, "scale": 3e38,
                                "prefix": 16}, {"cap": 1e30, "scale": 3e38}])
@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_refuses_what_overflows_in_log2_units(thd_lib, call, kw):
    assert call(**kw) == T.THD_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [{"cap": 2e38, "scale": 1e30}, {"cap": 0.0, "scale": 2e38, "prefix": 16}])
@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_takes_what_does_not(thd_lib, call, kw):
    assert call(wsb=0, **kw) == T.THD_ERR_WORKSPACE   # past the checks of the scores
