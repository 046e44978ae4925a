"""What the helpers rope and dropout_add refuse before any launch: tensors of
other dimensions, and axis numbers that do not fit the table's bytes.  On the
CPU, with the library and the device check replaced."""

import numpy as np
import pytest
import torch

from packed_sequence_context_gb300 import thd_attn as T


class FakeLib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def lib(monkeypatch):
    fake = FakeLib()
    monkeypatch.setattr(T, "lib", lambda: fake)
    monkeypatch.setattr(T, "thd_status_string", lambda code: str(code))
    monkeypatch.setattr(T, "_current", lambda where, t: t.get_device())
    monkeypatch.setattr(T, "_s", lambda stream: 0)
    return fake


def _rope(axis_of=None, q=(4, 2, 8), k=(4, 1, 8), pos=(2, 4)):
    q, k = torch.zeros(q, dtype=torch.bfloat16), torch.zeros(k, dtype=torch.bfloat16)
    return T.rope(q, k, torch.zeros(pos, dtype=torch.int32), np.ones(4), axis_of)


@pytest.mark.parametrize("axis_of", [[0, 1, 256, 1], [0, -1, 0, 0], [0, 2, 0, 0], [0.5, 1, 0, 0], np.array([0, 1, 257, 0]),
                                     np.array([0, 1, -256, 0], np.int32), [0, 1, 0], [[0, 1, 0, 1]], ["0"] * 4,
                                     [float("nan"), 0, 0, 0]])
def test_axis_numbers(lib, axis_of):
    with pytest.raises(T.ThdError) as e:
        _rope(axis_of)
    assert e.value.code == T.THD_ERR_INVALID_ARG and not lib.calls


@pytest.mark.parametrize("axis_of", [None, [0, 1, 0, 1], np.array([1, 1, 0, 0]), np.array([1.0, 1, 0, 0]),
                                     [True, False, True, True], np.zeros(4, np.uint8)])
def test_axis_numbers_that_fit(lib, axis_of):
    _rope(axis_of)
    assert len(lib.calls) == 1


@pytest.mark.parametrize("shapes", [{"q": (4, 16)}, {"q": (16,)}, {"q": (1, 4, 2, 8)}, {"k": (4, 8)}, {"k": (4,)},
                                    {"pos": (1, 2, 4)}, {"pos": ()}, {"pos": (2, 1, 4)}])
def test_dimensions(lib, shapes):
    with pytest.raises(T.ThdError) as e:
        _rope(**shapes)
    assert e.value.code == T.THD_ERR_INVALID_ARG and not lib.calls


def test_dropout_of_a_number(lib):
    with pytest.raises(T.ThdError) as e:
        T.dropout_add(torch.tensor(1.0), torch.zeros(2, dtype=torch.int64), 0.5)
    assert e.value.code == T.THD_ERR_INVALID_ARG and not lib.calls


@pytest.mark.parametrize("name", ["q", "k", "v", "o", "dout", "lse"])
@pytest.mark.parametrize("shape", [(), (8,), (8, 64), (1, 8, 2, 64)])
@pytest.mark.parametrize("bwd", [False, True])
def test_scored_attention_of_other_dimensions(lib, bwd, name, shape):
    t = {"q": (8, 2, 64), "k": (8, 1, 64), "v": (8, 1, 64), "o": (8, 2, 64), "dout": (8, 2, 64), "lse": (2, 8)}
    if name == "lse" and len(shape) == 2:
        shape = (8, 2)
    t[name] = shape
    t = {n: torch.zeros(s, dtype=torch.float32 if n == "lse" else torch.bfloat16) for n, s in t.items()}
    cu = torch.tensor([0, 8], dtype=torch.int32)
    with pytest.raises(T.ThdError) as e:
        if bwd:
            T.attn_score_bwd(*(t[n] for n in ("q", "k", "v", "o", "lse", "dout")), cu, cu, softcap=5.0)
        else:
            T.attn_score_fwd(t["q"], t["k"], t["v"], cu, cu, softcap=5.0, out=t["o"], lse=t["lse"],
                             dev_status=None if name != "dout" else torch.zeros(2, dtype=torch.int32))
    assert e.value.code == T.THD_ERR_INVALID_ARG and not lib.calls
