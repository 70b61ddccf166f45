"""Refusals of the cross attention on the host (no GPU): the C ABI's checks of addresses,
strides and sizes (nothing is launched), and the binding's checks of tensors."""
import ctypes

import pytest
import torch

from block_sparse_attention_nablat_gb300 import nabla as N

INVALID = 1
M = 1 << 24  # 256-byte aligned addresses far apart; never dereferenced


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


SHAPE = dict(dt=1, B=2, Sq=8, Sk=2048, h=4, hk=2, D=64)


def fwd(lib, **kw):
    a = dict(q=M, q_st=None, k=2 * M, k_st=None, v=3 * M, v_st=None, **SHAPE, kv_len=4 * M,
             scale=0.125, o=5 * M, lse=6 * M, ws=7 * M, ws_bytes=1 << 23, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.nabla_cross_attn_fwd(*a.values())


def bwd(lib, **kw):
    a = dict(q=M, q_st=None, k=2 * M, k_st=None, v=3 * M, v_st=None, o=5 * M, o_st=None,
             lse=6 * M, dout=8 * M, dout_st=None, **SHAPE, kv_len=4 * M, scale=0.125, dq=9 * M,
             dk=10 * M, dv=11 * M, ws=7 * M, ws_bytes=1 << 23, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.nabla_cross_attn_bwd(*a.values())


BAD = [dict(q=None), dict(k=None), dict(v=None), dict(q=M + 8), dict(k=2 * M + 2),
       dict(v=3 * M + 4), dict(dt=2), dict(B=0), dict(Sq=0), dict(Sk=0), dict(Sk=-1), dict(h=0),
       dict(hk=0), dict(hk=3), dict(h=130), dict(D=32), dict(D=96), dict(kv_len=4 * M + 2),
       dict(scale=float("nan")), dict(scale=float("inf")), dict(Sq=2 ** 30 + 1),
       dict(Sk=2 ** 30 + 1), dict(q_st=st(8 * 256, 255)), dict(q_st=st(7 * 256, 256)),
       dict(k_st=st(2048 * 128, 127)), dict(v_st=st(2047 * 128, 128)), dict(v_st=st(0, 128)),
       dict(k_st=st(2048 * 128, 64, 2047 * 64)), dict(ws=None), dict(ws=7 * M + 16),
       dict(ws_bytes=64), dict(B=2 ** 31 - 1)]


@pytest.mark.parametrize("kw", BAD, ids=lambda kw: "-".join(kw))
def test_bad_arguments(lib, kw):
    assert fwd(lib, **kw) == INVALID
    assert bwd(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(o=None), dict(o=5 * M + 8), dict(lse=6 * M + 2), dict(o=M),
                                dict(o=2 * M + 4096), dict(lse=3 * M), dict(lse=5 * M + 256),
                                dict(o=4 * M)], ids=lambda kw: "-".join(kw))
def test_bad_outputs(lib, kw):
    assert fwd(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(o=None), dict(lse=None), dict(dout=None), dict(dq=None),
                                dict(dk=None), dict(dv=None), dict(o=5 * M + 8),
                                dict(dout=8 * M + 2), dict(dq=9 * M + 4), dict(dk=2 * M),
                                dict(dv=10 * M), dict(dq=M + 256), dict(dq=8 * M), dict(dk=6 * M),
                                dict(o_st=st(8 * 256, 128)), dict(dout_st=st(8 * 256, 256, 32))],
                         ids=lambda kw: "-".join(kw))
def test_bad_gradient_arguments(lib, kw):
    assert bwd(lib, **kw) == INVALID


def test_workspace_bytes(lib):
    f, b = lib.nabla_cross_attn_fwd_workspace_bytes, lib.nabla_cross_attn_bwd_workspace_bytes
    assert f(1, 1, 32768, 512, 24, 24, 128) == 0      # enough rows: nothing is split
    assert f(1, 2, 1, 4096, 8, 2, 128) > 0            # one token against long states
    assert f(0, 2, 1, 4096, 8, 2, 128) > 0            # in fp32 too
    assert f(0, 1, 32768, 512, 24, 24, 128) == 0
    assert b(1, 1, 32768, 512, 24, 24, 128) >= 2 * 24 * 32768 * 4
    for bad in [(2, 1, 8, 8, 2, 2, 64), (1, 0, 8, 8, 2, 2, 64), (1, 1, 8, 8, 3, 2, 64),
                (1, 1, 8, 8, 2, 2, 80)]:
        assert f(*bad) == 0 and b(*bad) == 0


def tensors(dtype=torch.bfloat16):
    q = torch.zeros(2, 8, 4, 64, dtype=dtype)
    kv = torch.zeros(2, 70, 2, 2, 64, dtype=dtype)
    return q, kv[:, :, 0], kv[:, :, 1], torch.tensor([70, 3], dtype=torch.int32)


def test_binding_passes_good_tensors_up_to_the_device_check():
    for dtype in (torch.bfloat16, torch.float32):
        q, k, v, n = tensors(dtype)
        lse = torch.zeros(2, 4, 8)
        heads = q.transpose(1, 2).contiguous().transpose(1, 2)
        for call in (lambda: N.nabla_cross_attn_fwd(q, k, v),
                     lambda: N.nabla_cross_attn_fwd(heads, k, v, kv_len=n),
                     lambda: N.nabla_cross_attn_fwd_lse(q, k, v, n, 0.3),
                     lambda: N.nabla_cross_attn_bwd(q, k, v, heads, lse, q.clone(), n)):
            with pytest.raises(ValueError, match="CUDA device"):
                call()


def test_binding_refuses():
    q, k, v, n = tensors()
    lse = torch.zeros(2, 4, 8)
    for match, call in [
        ("q must be", lambda: N.nabla_cross_attn_fwd(q[0], k, v)),
        ("v must be", lambda: N.nabla_cross_attn_fwd(q, k, v[:, :60])),
        ("k must be", lambda: N.nabla_cross_attn_fwd(q, k[:1], v)),
        ("k must be torch.bfloat16", lambda: N.nabla_cross_attn_fwd(q, k.float(), v)),
        ("unsupported dtype", lambda: N.nabla_cross_attn_fwd(q.half(), k.half(), v.half())),
        ("v is on meta", lambda: N.nabla_cross_attn_fwd(q, k, v.to("meta"))),
        ("must not overlap", lambda: N.nabla_cross_attn_fwd(q, k[:1].expand(2, 70, 2, 64), v)),
        ("lie together", lambda: N.nabla_cross_attn_fwd(
            q.transpose(2, 3).contiguous().transpose(2, 3), k, v)),
        ("kv_len must be", lambda: N.nabla_cross_attn_fwd(q, k, v, n[:1])),
        ("kv_len must be torch.int32", lambda: N.nabla_cross_attn_fwd(q, k, v, n.long())),
        ("o must be torch.bfloat16", lambda: N.nabla_cross_attn_fwd(q, k, v, n, o=q.float())),
        ("o holds", lambda: N.nabla_cross_attn_fwd(q, k, v, n, o=q[:1].clone())),
        ("lse holds", lambda: N.nabla_cross_attn_fwd_lse(q, k, v, n, lse=lse[:1].clone())),
        ("lse must be torch.float32", lambda: N.nabla_cross_attn_bwd(q, k, v, q, lse.double(), q)),
        ("dout must be", lambda: N.nabla_cross_attn_bwd(q, k, v, q, lse, k)),
        ("o must be torch.bfloat16", lambda: N.nabla_cross_attn_bwd(q, k, v, q.float(), lse, q)),
        ("dk holds", lambda: N.nabla_cross_attn_bwd(q, k, v, q, lse, q, dk=k[:1].clone())),
        ("dq must be contiguous", lambda: N.nabla_cross_attn_bwd(
            q, k, v, q, lse, q, dq=q.transpose(1, 2).contiguous().transpose(1, 2))),
        ("workspace is on meta", lambda: N.nabla_cross_attn_bwd(
            q, k, v, q, lse, q, workspace=torch.empty(1 << 22, dtype=torch.uint8,
                                                      device="meta"))),
    ]:
        with pytest.raises((ValueError, TypeError), match=match):
            call()


@pytest.mark.parametrize("Sq,Sk,heads,D,runs", [
    (8, 8192, 8, 128, 32),     # eight rows a key head: two blocks on an SM, runs of four tiles
    (9, 8192, 8, 128, 19),     # more rows: one block on an SM, one wave of them
    (16, 2048, 24, 128, 6),
    (16, 8192, 60, 64, 5),     # two waves where one leaves a fifth of the SMs idle
    (10, 8192, 100, 64, 3),
    (16, 8192, 160, 64, 0),    # units enough without runs
], ids=lambda x: str(x))
def test_runs_of_few_fp32_rows_follow_the_blocks_an_sm_holds(lib, Sq, Sk, heads, D, runs):
    """Sums and log-sum-exps of that many runs, in fp32."""
    need = lib.nabla_cross_attn_fwd_workspace_bytes(0, 1, Sq, Sk, heads, heads, D)
    assert need == runs * heads * Sq * (D + 1) * 4


def test_lse_form_names_what_is_wrong_with_q():
    """As the form without lse does, before anything is allocated by q's sizes."""
    q, k, v, n = tensors()
    for call in (N.nabla_cross_attn_fwd, N.nabla_cross_attn_fwd_lse):
        for bad in (q[0, 0], q[0], q[None]):
            with pytest.raises(ValueError, match="q must be"):
                call(bad, k, v, n)
