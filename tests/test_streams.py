"""Helpers called with ``stream=``: everything they allocate has to come from
that stream's memory.  A workspace from the current stream's would be free for
the current stream's next tensor as soon as the helper returns, while the
kernels on the other stream still read the schedule and the row extents in it;
an output from there may still be in use by what the current stream was given
before.

On the CPU: the library and torch's streams are fakes, and every allocation is
recorded with the stream that is current at the time.  On the GPU: a busy
stream's call, with tensors made and filled on the current stream meanwhile."""

import numpy as np
import pytest
import torch

from packed_sequence_context_gb300 import inputs
from packed_sequence_context_gb300 import thd_attn as T


# ------------------------------------------------------------------ no GPU
class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle

    def __eq__(self, other):
        return isinstance(other, FakeStream) and other.cuda_stream == self.cuda_stream

    __hash__ = None


class FakeLib:
    """Every entry point answers THD_OK (or a size) and leaves its arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 4096 if name.endswith("_size") else 0
        return call


@pytest.fixture
def fakes(monkeypatch):
    """(library, allocations [(handle, shape)], {data_ptr: handles recorded on it})"""
    lib, made, recorded = FakeLib(), [], {}
    current = [FakeStream(0)]

    class Entered:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            current.append(self.s)

        def __exit__(self, *_):
            current.pop()

    def record(t, s):
        recorded.setdefault(t.data_ptr(), set()).add(s.cuda_stream)

    monkeypatch.setattr(T, "lib", lambda: lib)
    monkeypatch.setattr(T, "_current", lambda where, t: t.get_device())
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", Entered)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: FakeStream(0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", FakeStream)
    monkeypatch.setattr(torch.Tensor, "record_stream", record)
    for name in ("empty", "zeros", "empty_like"):
        real = getattr(torch, name)

        def alloc(*a, _real=real, **kw):
            t = _real(*a, **kw)
            made.append((current[-1].cuda_stream, t))
            return t
        monkeypatch.setattr(torch, name, alloc)
    new_empty = torch.Tensor.new_empty

    def new(self, *a, **kw):
        t = new_empty(self, *a, **kw)
        made.append((current[-1].cuda_stream, t))
        return t
    monkeypatch.setattr(torch.Tensor, "new_empty", new)
    return lib, made, recorded


def _calls():
    """name -> (call(stream), the inputs it reads)"""
    n, D = 8, 64
    rows = lambda h: torch.ones(n, h, D, dtype=torch.bfloat16)  # noqa: E731
    q, k, v, o, do = rows(2), rows(1), rows(1), rows(2), rows(2)
    lse = torch.ones(2, n)
    cu = torch.tensor([0, n], dtype=torch.int32)
    doc = torch.ones(n, dtype=torch.int32)
    shard = lambda h: torch.ones(2, n // 2, h, D, dtype=torch.bfloat16)  # noqa: E731
    sq, sk, so, sdo = shard(2), shard(2), shard(2), shard(2)
    x, rng = torch.ones(n, 16), torch.ones(2, dtype=torch.int64)
    pos = torch.ones(n, dtype=torch.int32)
    a2a = {"cp_size": 2, "a2a_size": 2}
    return {
        "attn_fwd": (lambda s: T.attn_fwd(q, k, v, cu, cu, stream=s), (q, k, v, cu)),
        "attn_fwd_step": (lambda s: T.attn_fwd_step(q, k, v, cu, cu, step=0, stream=s), (q, k, v, cu)),
        "attn_fwd_step_bf16": (lambda s: T.attn_fwd_step_bf16(q, k, v, cu, cu, step=0, stream=s), (q, k, v, cu)),
        "attn_bwd": (lambda s: T.attn_bwd(q, k, v, o, lse, do, cu, cu, stream=s), (q, k, v, o, lse, do, cu)),
        "attn_score_fwd": (lambda s: T.attn_score_fwd(q, k, v, cu, cu, doc_q=doc, doc_kv=doc, stream=s),
                           (q, k, v, cu, doc)),
        "attn_score_bwd": (lambda s: T.attn_score_bwd(q, k, v, o, lse, do, cu, cu, doc_q=doc, doc_kv=doc, stream=s),
                           (q, k, v, o, lse, do, cu, doc)),
        "cp_partition": (lambda s: T.cp_partition(cu, cp_size=2, token_map_capacity=n, stream=s), (cu,)),
        "cp_a2a": (lambda s: T.cp_a2a(sq, cu, direction=T.THD_A2A_TO_GROUPS, stream=s, **a2a), (sq, cu)),
        "attn_fwd_a2a": (lambda s: T.attn_fwd_a2a(sq, sk, sk, cu, cu, stream=s, **a2a), (sq, sk, cu)),
        "attn_bwd_a2a": (lambda s: T.attn_bwd_a2a(sq, sk, sk, so, lse, sdo, cu, cu, stream=s, **a2a),
                         (sq, sk, so, lse, sdo, cu)),
        "rope": (lambda s: T.rope(q, k, pos, np.ones(4), stream=s), (q, k, pos)),
        "dropout_add": (lambda s: T.dropout_add(x, rng, 0.5, residual=x, row_ids=doc, stream=s), (x, rng, doc)),
    }


def _tensors(out):
    if isinstance(out, torch.Tensor):
        return [out]
    if isinstance(out, dict):
        return [t for t in out.values() if t is not None]
    return [t for item in out for t in _tensors(item)] if isinstance(out, tuple) else []


@pytest.mark.parametrize("name", list(_calls()))
def test_allocates_from_the_launch_stream(fakes, name):
    lib, made, recorded = fakes
    call, ins = _calls()[name]
    made.clear()
    out = _tensors(call(FakeStream(64)))
    launches = [a for n, a in lib.calls if not n.endswith("_size")]
    assert [a[-1] for a in launches] == [64]
    assert made and all(handle == 64 for handle, _ in made), "allocated where the kernels do not run"
    # outputs come back to the caller's stream, inputs are read on the other: both are kept until it is done
    for t in out:
        assert recorded.get(t.data_ptr()) == {0}
    for t in ins:
        assert recorded.get(t.data_ptr()) == {64}


@pytest.mark.parametrize("handle,where", [(0, 0), (1, 0), (64, 64)])
@pytest.mark.parametrize("name", ["attn_score_fwd", "rope"])
def test_a_raw_handle_names_a_stream_too(fakes, name, handle, where):
    """0 and 1 (the legacy default stream) are the default stream."""
    lib, made, _ = fakes
    call, _ = _calls()[name]
    made.clear()
    call(handle)
    assert [a[-1] for n, a in lib.calls if not n.endswith("_size")] == [handle]
    assert made and all(h == where for h, _ in made)


@pytest.mark.parametrize("name", list(_calls()))
def test_without_a_stream_nothing_is_recorded(fakes, name):
    lib, made, recorded = fakes
    T_s = T._s
    T._s = lambda stream: 0 if stream is None else T_s(stream)
    try:
        call, _ = _calls()[name]
        made.clear()
        call(None)
        call(FakeStream(0))   # the current one
    finally:
        T._s = T_s
    assert made and all(h == 0 for h, _ in made) and not recorded


# ------------------------------------------------------------------ GPU
@pytest.mark.gpu
@pytest.mark.parametrize("by_handle", [False, True])
def test_a_busy_stream_keeps_its_buffers(thd_lib, by_handle):
    """The call waits on its stream behind other work; meanwhile the current
    stream makes and fills tensors of the workspace's and the outputs' sizes,
    and the call's own temporary inputs are gone."""
    lengths = [300, 513]
    c = inputs.make_cross(lengths, lengths, pad_to=8, Hq=4, Hkv=2, D=64, cp_size=2, seed=3)
    d = {x: c[x].cuda() for x in ("q", "k", "v", "do")}
    off = [torch.from_numpy(c[n]).cuda() for n in ("cu_q", "cu_kv", "cu_q_pad", "cu_kv_pad")]
    doc = torch.zeros(d["q"].shape[0], dtype=torch.int32, device="cuda")
    kw = dict(softcap=20.0, cp_size=2)
    want = T.attn_score_fwd(d["q"], d["k"], d["v"], *off, doc_q=doc, doc_kv=doc, **kw)
    wantg = T.attn_score_bwd(d["q"], d["k"], d["v"], *want[:2], d["do"], *off, doc_q=doc, doc_kv=doc, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    arg = side.cuda_stream if by_handle else side
    t = d["q"].shape[0]
    sizes = [T.thd_score_workspace_size(2, t, t, 4, 2, 64, 2, 1, b) for b in (0, 1)]
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)   # about 10 ms, then it ends
        own = [doc.clone(), doc.clone()] if by_handle else None
        q = [d["q"] if by_handle else d["q"].clone()]
        side.wait_stream(torch.cuda.current_stream())
        got = T.attn_score_fwd(q.pop(), d["k"], d["v"], *off,
                               doc_q=own[0] if own else doc, doc_kv=own[1] if own else doc, stream=arg, **kw)
        g = T.attn_score_bwd(d["q"], d["k"], d["v"], *want[:2], d["do"], *off, doc_q=doc, doc_kv=doc, stream=arg, **kw)
        junk = [torch.full((n,), 0x3f, dtype=torch.uint8, device="cuda") for n in sizes * 2]
        junk += [torch.full_like(d["q"], 9.0) for _ in range(4)]
        torch.cuda.synchronize()
        for a, b in zip(got[:2] + g[:3], want[:2] + wantg[:3]):
            assert torch.equal(a, b)
        assert int(got[2].item()) == 0 and int(g[3].item()) == 0
        del junk
