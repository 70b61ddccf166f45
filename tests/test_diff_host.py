"""Refusals of the differential attention, on the host (no GPU): the C ABI's checks of
addresses, strides and sizes (nothing is launched), the workspaces, and the binding's checks."""
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


def st(batch, token, head=64):
    return ctypes.byref(N._Strides(batch, token, head))


def fwd(lib, **kw):
    a = dict(q=M, q_st=None, k=2 * M, k_st=None, v=3 * M, v_st=None, dt=1, B=2, Sq=8, Sk=10, h=4,
             hk=2, D=64, lam=4 * M, lam_n=4, kv_len=5 * M, scale=0.1, o=6 * M, o2=7 * M, lse=8 * M,
             ws=16 * M, ws_bytes=1 << 30, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.nabla_diff_attn_fwd(*a.values())


def bwd(lib, **kw):
    a = dict(q=M, q_st=None, k=2 * M, k_st=None, v=3 * M, v_st=None, o=6 * M, o_st=None, o2=7 * M,
             o2_st=None, lse=8 * M, dout=9 * M, dout_st=None, dt=1, B=2, Sq=8, Sk=10, h=4, hk=2,
             D=64, lam=4 * M, lam_n=4, kv_len=5 * M, scale=0.1, dq=10 * M, dk=11 * M, dv=12 * M,
             dlam=13 * M, ws=16 * M, ws_bytes=1 << 30, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.nabla_diff_attn_bwd(*a.values())


BOTH = [dict(q=None), dict(k=2 * M + 8), dict(v=None), dict(dt=3), dict(B=0), dict(Sq=0),
        dict(Sk=0), dict(h=0), dict(hk=0), dict(hk=3), dict(h=130, hk=2), dict(D=32), dict(D=256),
        dict(lam=None), dict(lam=4 * M + 2), dict(lam_n=0), dict(lam_n=2), dict(kv_len=5 * M + 1),
        dict(scale=NAN), dict(scale=INF), dict(q_st=st(8 * 256, 252)), dict(q_st=st(7 * 256, 256)),
        dict(k_st=st(10 * 128, 128, 60)), dict(v_st=st(10 * 128, -128)),
        dict(Sq=2 ** 30 + 1), dict(B=2 ** 20, Sq=2 ** 20), dict(ws=16 * M + 8, Sk=9000, B=1, Sq=1),
        dict(ws=None, Sk=9000, B=1, Sq=1), dict(ws_bytes=64, Sk=9000, B=1, Sq=1)]
FWD = [dict(o=None), dict(o=6 * M + 8), dict(o2=7 * M + 4), dict(lse=8 * M + 2), dict(o=M),
       dict(o2=2 * M), dict(lse=3 * M), dict(o=5 * M), dict(o2=6 * M), dict(lse=7 * M),
       dict(o=4 * M), dict(lse=6 * M + 64)]
BWD = [dict(o=None), dict(o2=None), dict(lse=None), dict(dout=None), dict(dq=None), dict(dk=None),
       dict(dv=None), dict(dlam=None), dict(dlam=13 * M + 2), dict(dq=10 * M + 8),
       dict(o2_st=st(8 * 256, 250)), dict(dout=9 * M + 2), dict(dq=M), dict(dk=9 * M),
       dict(dv=11 * M), dict(dlam=4 * M), dict(dlam=8 * M), dict(dq=7 * M), dict(dk=6 * M),
       dict(dlam=12 * M), dict(dv=5 * M), dict(lse=8 * M + 1)]


@pytest.mark.parametrize("bad", BOTH + FWD, ids=str)
def test_forward_refuses(lib, bad):
    assert fwd(lib, **bad) == INVALID


@pytest.mark.parametrize("bad", BOTH + BWD, ids=str)
def test_backward_refuses(lib, bad):
    assert bwd(lib, **bad) == INVALID


def test_workspaces(lib):
    f, b = lib.nabla_diff_attn_fwd_workspace_bytes, lib.nabla_diff_attn_bwd_workspace_bytes
    for bad in ((1, 0, 1, 1, 1, 1, 64), (1, 1, 1, 1, 1, 1, 96), (2, 1, 1, 1, 1, 1, 64),
                (0, 1, 1, 1, 3, 2, 64)):
        assert f(*bad) == b(*bad) == 0
    assert f(1, 2, 32768, 512, 12, 12, 128) == 0         # many rows: no runs
    n = f(1, 1, 1, 8192, 2, 2, 128)                      # few: runs of 256 states
    assert n == 32 * 2 * 2 * 129 * 4
    for dt in (0, 1):
        assert b(dt, 2, 100, 300, 6, 2, 128) >= 5 * 2 * 2 * 6 * 64 * 4
        assert bwd(lib, dt=dt, ws_bytes=b(dt, 2, 8, 10, 4, 2, 64) - 1) == INVALID


def test_binding_refuses(lib):
    q, k, lam = torch.zeros(2, 5, 4, 64), torch.zeros(2, 7, 2, 64), torch.zeros(4)
    lse = torch.zeros(2, 4, 2, 5)
    forward = [
        ((q[0], k, k, lam), {}, r"q must be"), ((q, k, k[:, :6], lam), {}, "v must be"),
        ((q, k.bfloat16(), k, lam), {}, "k must be torch.float32"),
        ((q, k, k, lam[:3]), {}, "lam must be"), ((q, k, k, lam.view(2, 2)), {}, "lam must be"),
        ((q, k, k, lam.double()), {}, "lam must be torch.float32"),
        ((q, k, k, lam), dict(kv_len=torch.zeros(3, dtype=torch.int32)), "kv_len"),
        ((q, k, k, lam), dict(kv_len=torch.zeros(2)), "kv_len must be torch.int32"),
        ((q, k, k, lam), dict(o=q[:1]), "o holds"), ((q, k, k, lam), {}, "CUDA device"),
    ]
    for args, kw, text in forward:
        with pytest.raises(ValueError, match=text):
            N.nabla_diff_attn_fwd(*args, **kw)
    with pytest.raises(ValueError, match="lse holds"):
        N.nabla_diff_attn_fwd_lse(q, k, k, lam, lse=lse[:, :, 0].contiguous())
    with pytest.raises(ValueError, match="o2 must be"):
        N.nabla_diff_attn_fwd_lse(q, k, k, lam, o2=q.bfloat16())
    backward = [
        ((q[:, :4], q, lse, q), {}, "o must be"), ((q, q.bfloat16(), lse, q), {}, "o2 must be"),
        ((q, q, lse[:1], q), {}, "lse holds"), ((q, q, lse, q[:1]), {}, "dout must be"),
        ((q, q, lse, torch.zeros(1).expand(q.shape)), {}, "columns of dout|must not overlap"),
        ((q, q, lse, q), dict(dlam=lam[:2]), "dlam holds"), ((q, q, lse, q), {}, "CUDA device"),
    ]
    for args, kw, text in backward:
        with pytest.raises(ValueError, match=text):
            N.nabla_diff_attn_bwd(q, k, k, lam, *args, **kw)
