"""Refusals of the gated sum with adaptive norm, on the host (no GPU): the C ABI's checks of
addresses, strides and sizes (nothing is launched), and the binding's checks of tensors."""
import ctypes

import pytest
import torch

from block_sparse_attention_nablat_gb300 import nabla as N

INVALID = 1
M = 1 << 20  # 16-byte aligned addresses far apart; never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    try:
        return N.load()
    except RuntimeError:
        import __graft_entry__

        __graft_entry__.build()
        return N.load()


def st(batch, token):
    return ctypes.byref(N._Strides(batch, token, 0))


def fwd(lib, **kw):
    a = dict(x=M, x_st=None, u=2 * M, u_st=None, dt=1, B=2, S=8, C=64, norm=2, post=1, w=3 * M,
             pw=3 * M + 512, wdt=1, gate=4 * M, gate_st=64, scale=5 * M, scale_st=64, shift=6 * M,
             shift_st=64, mdt=0, rows=2, rs=1.0, eps=1e-6, xo=7 * M, xo_st=None, y=8 * M,
             y_st=None, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.nabla_block_norm(*a.values())


def bwd(lib, **kw):
    a = dict(s=M, s_st=None, u=2 * M, u_st=None, dsum=9 * M, dsum_st=None, dy=10 * M, dy_st=None,
             dt=1, B=2, S=8, C=64, norm=2, post=1, w=3 * M, pw=3 * M + 512, wdt=1, gate=4 * M,
             gate_st=64, scale=5 * M, scale_st=64, mdt=0, rows=2, rs=1.0, eps=1e-6, dx=7 * M,
             dx_st=None, du=8 * M, du_st=None, dgate=11 * M, dscale=12 * M, dshift=13 * M,
             dw=14 * M, dpw=15 * M, ws=16 * M, ws_bytes=1 << 30, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.nabla_block_norm_bwd(*a.values())


BOTH = [dict(dt=2), dict(wdt=7), dict(mdt=-1), dict(B=0), dict(S=0), dict(C=0), dict(C=60),
        dict(C=8200), dict(norm=3), dict(norm=-1), dict(post=3), dict(rows=0), dict(rows=3),
        dict(rs=NAN), dict(rs=INF), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(w=3 * M + 8),
        dict(pw=3 * M + 4), dict(gate=4 * M + 4), dict(gate_st=60), dict(scale_st=66),
        dict(scale=5 * M + 8), dict(post=0), dict(u=None), dict(u=2 * M + 2),
        dict(u_st=st(8 * 64, 60)), dict(u_st=st(7 * 64, 64)), dict(B=2 ** 31 - 1, S=2 ** 31 - 1)]
FWD = [dict(x=None), dict(x=M + 8), dict(x_st=st(8 * 64, 68)), dict(xo=None), dict(y=None),
       dict(norm=0), dict(norm=0, y=None), dict(xo=M, xo_st=st(9 * 64, 64)), dict(xo=M + 16),
       dict(xo=2 * M), dict(y=M), dict(y=2 * M), dict(y=7 * M), dict(y=3 * M), dict(xo=4 * M),
       dict(y=5 * M + 256), dict(xo=3 * M + 512), dict(shift_st=32), dict(shift=6 * M + 4),
       dict(y=6 * M), dict(xo_st=st(8 * 64, 64 - 8)), dict(y_st=st(0, 64))]
BWD = [dict(s=None), dict(dy=None), dict(norm=0), dict(s=M + 8), dict(dy=10 * M + 4),
       dict(dsum=9 * M + 8), dict(dx=M), dict(dx=2 * M), dict(dx=10 * M), dict(du=7 * M),
       dict(du=9 * M), dict(du=2 * M), dict(dx=9 * M + 16), dict(dx=9 * M, dx_st=st(9 * 64, 64)),
       dict(dx=4 * M), dict(du=3 * M), dict(dgate=4 * M), dict(dgate=11 * M + 4),
       dict(dscale=11 * M), dict(dshift=12 * M + 256), dict(dw=3 * M), dict(dw=15 * M),
       dict(dpw=7 * M), dict(dshift=10 * M), dict(ws=None), dict(ws=16 * M + 16),
       dict(ws_bytes=4096)]


@pytest.mark.parametrize("bad", BOTH + FWD, ids=str)
def test_forward_refuses(lib, bad):
    assert fwd(lib, **bad) == INVALID


@pytest.mark.parametrize("bad", BOTH + BWD, ids=str)
def test_backward_refuses(lib, bad):
    if "u" in bad and bad["u"] is None:  # without u: nothing that needs it
        assert bwd(lib, u=None, post=0, pw=None, dgate=None, dpw=3) == INVALID
        assert bwd(lib, u=None, post=0, pw=None, dpw=None) == INVALID  # dgate
    assert bwd(lib, **bad) == INVALID


def test_more_that_is_refused(lib):
    assert fwd(lib, u=None, xo=None, post=0, pw=None) == INVALID             # a gate
    assert fwd(lib, u=None, xo=None, gate=None, pw=None) == INVALID          # a post norm
    assert fwd(lib, norm=0, y=None, w=None, scale=None) == INVALID           # a shift
    assert bwd(lib, post=0, pw=None) == INVALID                              # dpost_weight
    none = dict(dx=None, du=None, dgate=None, dscale=None, dshift=None, dw=None, dpw=None)
    assert bwd(lib, **none) == INVALID                                       # nothing wanted
    assert bwd(lib, norm=0, s=None, dy=None, w=None, scale=None, dscale=None, dshift=None,
               dw=None, dsum=None) == INVALID                                # nothing upstream


def test_modulations_whose_extent_wraps_are_refused(lib):
    """2^30 rows 2^34 elements apart: 2^64 elements, 0 if their number is taken modulo that."""
    far = dict(B=1, S=1 << 30, C=8, rows=1 << 30, mdt=1, u=None, post=0, w=None, pw=None,
               gate=None, scale=None)
    assert fwd(lib, xo=None, x=1 << 50, y=2 << 50, shift=3 << 50, shift_st=1 << 34,
               **far) == INVALID
    far.update(scale=3 << 50, scale_st=1 << 34)
    assert bwd(lib, s=1 << 50, dy=2 << 50, dsum=None, dx=4 << 50, du=None, dgate=None, dscale=None,
               dshift=None, dw=None, dpw=None, **far) == INVALID


def test_workspace(lib):
    size = lib.nabla_block_norm_bwd_workspace_bytes
    assert size(1, 1000, 60) == size(0, 8, 64) == size(1, 1, 8200) == 0
    for shape in ((1, 1, 8), (2, 32768, 2048), (16, 1, 8192), (1, 2000000, 64)):
        assert 0 < size(*shape) < 1 << 28 and size(*shape) % 256 == 0
    assert bwd(lib, ws_bytes=size(2, 8, 64) - 1) == INVALID


def tensors(C=64, B=2, S=6):
    x, u = torch.zeros(B, S, C), torch.zeros(B, S, C)
    return x, u, torch.zeros(B, C), torch.zeros(C)


def test_binding_refuses(lib):
    x, u, m, w = tensors()
    cases = [
        ((x, u[:, :5]), {}, "u must be"), ((x[0], None), {}, r"\[B, S, C\]"),
        ((x, u.bfloat16()), {}, "u must be torch.float32"),
        ((x, u.transpose(1, 2).contiguous().transpose(1, 2)), {}, "columns of u"),
        ((x, u[:, :1].expand(2, 6, 64)), {}, "rows of u must not overlap"),
        ((x, u), dict(norm="batch"), "norm must be"), ((x, u), dict(post_norm=1), "post_norm"),
        ((x, u), dict(norm=None, scale=m), "need a norm"), ((x, None), dict(norm=None), "nothing"),
        ((x, u), dict(post_weight=w), "needs a post_norm"), ((x, None), dict(gate=m), "need u"),
        ((x, None), dict(x_out=u), "x_out without u"), ((x, u), dict(norm=None, y=x), "y without"),
        ((x, u), dict(weight=w[:32]), "weight"), ((x, u), dict(gate=m[:1]), "gate must be"),
        ((x, u), dict(gate=torch.zeros(2, 4, 64)), "m dividing 6"),
        ((x, u), dict(gate=torch.zeros(64, 2).t()), "columns of gate"),
        ((x, u), dict(gate=torch.zeros(2, 5, 64)[:, :3]), "equally far apart"),
        ((x, u), dict(gate=m, scale=m.bfloat16()), "scale must be"),
        ((x, u), dict(gate=m, shift=w), "shift must be"),
        ((x, u), dict(weight=w.double(), gate=m), "unsupported dtype"),
        ((x, u), dict(), "CUDA device"),
    ]
    for args, kw, text in cases:
        with pytest.raises((ValueError, TypeError), match=text):
            N.nabla_block_norm(*args, **kw)


def test_binding_backward_refuses(lib):
    x, u, m, w = tensors()
    cases = [
        ((x, u, x, None), {}, "dy is needed"), ((None, u, None, None), dict(norm=None), "dsum"),
        ((x, u, x[:1], x), {}, "dsum must be"), ((x, u, x, x), dict(dx=x[:, :3]), "dx must be"),
        ((x, None, x, x), dict(du=u), "du without u"), ((x, None, x, x), dict(gate=m), "need u"),
        ((x, u, x, x), dict(workspace=torch.zeros(8, 8).t()), "workspace"),
        ((x, u, x, x), {}, "CUDA device"),
    ]
    for args, kw, text in cases:
        with pytest.raises(ValueError, match=text):
            N.nabla_block_norm_bwd(*args, **kw)
