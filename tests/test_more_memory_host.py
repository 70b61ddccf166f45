"""Where the differential attention's and the fused norm's calls take their own memory from,
on the host (no GPU).

Scratch and outputs of a call on another stream than the current one come from that stream;
the outputs are also kept for the current one, the scratch is free again behind the kernels.
Stand-ins take the place of the streams, the device memory and the library's launches.
"""
import contextlib

import pytest
import torch

from block_sparse_attention_nablat_gb300 import nabla as N

CURRENT, SIDE = 111, 222
B, S, h, D = 1, 640, 2, 64


class OnDevice(torch.Tensor):
    """Host memory that says it is on cuda:0."""
    device = property(lambda self: torch.device("cuda", 0))
    is_cuda = True
    kept = {}  # data_ptr -> the streams it was recorded on

    def record_stream(self, stream):
        OnDevice.kept.setdefault(self.data_ptr(), []).append(stream.cuda_stream)


class FakeStream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle


class Library:
    """The real library's sizes; launches are recorded."""

    def __init__(self, lib):
        self.lib, self.calls = lib, []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.lib, name)
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def made(monkeypatch):
    """The allocations of a call: [(tensor, stream it came from)], and the library."""
    try:
        real = N.load()
    except RuntimeError:
        import __graft_entry__

        __graft_entry__.build()
        real = N.load()
    lib, active, made, empty = Library(real), [CURRENT], [], torch.empty

    def fake_empty(*size, device=None, **kw):
        t = empty(*size, **kw).as_subclass(OnDevice)
        made.append((t, active[-1]))
        return t

    @contextlib.contextmanager
    def on(stream):
        active.append(stream.cuda_stream)
        yield
        active.pop()

    OnDevice.kept.clear()
    monkeypatch.setattr(torch, "empty", fake_empty)
    monkeypatch.setattr(torch, "empty_like",
                        lambda t, **kw: fake_empty(t.shape, dtype=t.dtype))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: FakeStream(CURRENT))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: CURRENT, raising=False)
    monkeypatch.setattr(torch.cuda, "ExternalStream", FakeStream)
    monkeypatch.setattr(N, "load", lambda: lib)
    return made, lib


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


def calls():
    """Every entry point that allocates, with none of its outputs given."""
    q, k, v, o, o2, g = (t(B, S, h, D) for _ in range(6))
    lam, lse = t(h, dtype=torch.float32), t(B, h, 2, S, dtype=torch.float32)
    one = t(B, 1, h, D)  # few rows: the forward splits its states, with scratch
    x, u, ds, dy, m, w = (*(t(B, S, 256) for _ in range(4)), t(B, 256), t(256))
    norm = dict(gate=m, scale=m, shift=m, weight=w, post_weight=w, post_norm="rms")
    return {
        "block_norm": lambda s: N.nabla_block_norm(x, u, stream=s, **norm),
        "block_norm_bwd": lambda s: N.nabla_block_norm_bwd(x, u, ds, dy, stream=s, **norm),
        "diff_attn_fwd": lambda s: N.nabla_diff_attn_fwd(one, k, v, lam, stream=s),
        "diff_attn_fwd_lse": lambda s: N.nabla_diff_attn_fwd_lse(one, k, v, lam, stream=s),
        "diff_attn_bwd": lambda s: N.nabla_diff_attn_bwd(q, k, v, lam, o, o2, lse, g, stream=s),
    }


OUTPUTS = {"block_norm": 2, "block_norm_bwd": 7, "diff_attn_fwd": 1, "diff_attn_fwd_lse": 3,
           "diff_attn_bwd": 4}


def returned(x):
    return {y.data_ptr() for y in (x if isinstance(x, (tuple, list)) else [x]) if y is not None}


@pytest.mark.parametrize("name", list(OUTPUTS))
@pytest.mark.parametrize("stream", [FakeStream(SIDE), SIDE], ids=["object", "handle"])
def test_memory_of_a_call_on_another_stream(made, name, stream):
    allocated, lib = made
    outs = returned(calls()[name](stream))
    (_, args), = lib.calls
    assert args[-1] == SIDE
    assert allocated and all(at == SIDE for _, at in allocated)
    own = {x.data_ptr() for x, _ in allocated}
    assert len(outs) == OUTPUTS[name]
    assert outs <= own and all(OnDevice.kept[p] == [CURRENT] for p in outs)
    assert len(own - outs) == (name != "block_norm")
    assert all(p not in OnDevice.kept for p in own - outs)


@pytest.mark.parametrize("name", list(OUTPUTS))
@pytest.mark.parametrize("stream", [FakeStream(CURRENT), CURRENT, None],
                         ids=["object", "handle", "none"])
def test_memory_of_a_call_on_the_current_stream(made, name, stream):
    allocated, lib = made
    calls()[name](stream)
    assert lib.calls[0][1][-1] == CURRENT
    assert allocated and all(at == CURRENT for _, at in allocated) and not OnDevice.kept
