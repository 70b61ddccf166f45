"""What a call allocates itself when it is given a stream, on the host (no GPU).

The caching allocator reuses a freed block in the order of the stream that it was
allocated on.  So the scratch and the outputs of a call on another stream than the
current one have to come from that stream, and the outputs, which the caller goes on
using, have to be kept for the current stream too.  Stand-ins take the place of the
streams, the device memory and the library's launches.
"""
import contextlib

import pytest
import torch

from block_sparse_attention_nablat_gb300 import nabla as N

CURRENT, SIDE = 111, 222
B, S, h, D = 1, 1024, 2, 64
s1 = S // 64


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
    monkeypatch.setattr(torch, "empty_like", lambda t: fake_empty(t.shape, dtype=t.dtype))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: FakeStream(CURRENT))
    monkeypatch.setattr(torch.cuda, "ExternalStream", FakeStream)
    monkeypatch.setattr(N, "load", lambda: lib)
    return made, lib


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)


def calls():
    """Every entry point that allocates, with none of its outputs given."""
    q, k, v, o, g = (t(B, S, h, D) for _ in range(5))
    nb, inds = t(B, h, s1, dtype=torch.int32), t(B, h, s1, s1, dtype=torch.int32)
    sta, w = t(s1, s1, dtype=torch.uint8), t(D)
    lse = t(B, h, S, dtype=torch.float32)
    one = t(B, 1, h, D)  # few rows: the forward splits its states, with scratch
    return {
        "build_mask": lambda s: N.nabla_build_mask(q, k, sta, 0.9, stream=s),
        "build_mask_topk": lambda s: N.nabla_build_mask_topk(q, k, 0.1, stream=s),
        "attn_fwd": lambda s: N.nabla_attn_fwd(q, k, v, nb, inds, stream=s),
        "attn_fwd_lse": lambda s: N.nabla_attn_fwd_lse(q, k, v, nb, inds, stream=s),
        "attn_bwd": lambda s: N.nabla_attn_bwd(q, k, v, o, g, nb, inds, stream=s),
        "sta_mask": lambda s: N.nabla_sta_mask(4, 2, 2, 1, 1, 1, device="cuda:0", stream=s),
        "flatten": lambda s: N.nabla_fractal_flatten(t(1, 2, 16, 16, 2, 64), 8, stream=s),
        "unflatten": lambda s: N.nabla_fractal_unflatten(t(1, 512, 2, 64), 2, 16, 16, 8, stream=s),
        "qk_norm_rope": lambda s: N.nabla_qk_norm_rope(q, k, w, w, stream=s),
        "qk_norm_rope_bwd": lambda s: N.nabla_qk_norm_rope_bwd(q, k, w, w, o, g, stream=s),
        "cross_attn_fwd": lambda s: N.nabla_cross_attn_fwd(one, k, v, stream=s),
        "cross_attn_fwd_lse": lambda s: N.nabla_cross_attn_fwd_lse(one, k, v, stream=s),
        "cross_attn_bwd": lambda s: N.nabla_cross_attn_bwd(q, k, v, o, lse, g, stream=s),
    }


SCRATCH = {"build_mask", "build_mask_topk", "attn_bwd", "qk_norm_rope_bwd", "cross_attn_fwd",
           "cross_attn_fwd_lse", "cross_attn_bwd"}


def returned(x):
    return {y.data_ptr() for y in (x if isinstance(x, (tuple, list)) else [x]) if y is not None}


@pytest.mark.parametrize("name", list(calls()))
@pytest.mark.parametrize("stream", [FakeStream(SIDE), SIDE], ids=["object", "handle"])
def test_memory_of_a_call_on_another_stream(made, name, stream):
    allocated, lib = made
    outs = returned(calls()[name](stream))
    (_, args), = lib.calls
    assert args[-1] == SIDE
    assert allocated and all(at == SIDE for _, at in allocated)
    own = {x.data_ptr() for x, _ in allocated}
    assert outs <= own and all(OnDevice.kept[p] == [CURRENT] for p in outs)
    assert len(own - outs) == (1 if name in SCRATCH else 0)
    assert all(p not in OnDevice.kept for p in own - outs)  # free again behind the kernels


@pytest.mark.parametrize("name", list(calls()))
@pytest.mark.parametrize("stream", [FakeStream(CURRENT), CURRENT], ids=["object", "handle"])
def test_memory_of_a_call_on_the_current_stream(made, name, stream):
    allocated, lib = made
    calls()[name](stream)
    assert lib.calls[0][1][-1] == CURRENT
    assert allocated and all(at == CURRENT for _, at in allocated) and not OnDevice.kept
