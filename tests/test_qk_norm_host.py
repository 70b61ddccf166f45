"""Refusals of the query/key norm with rotation, on the host (no GPU): the C ABI's
checks of addresses, strides and sizes (nothing is launched), and the binding's
checks of tensors."""
import ctypes

import pytest
import torch

from block_sparse_attention_nablat_gb300 import nabla as N

INVALID = 1
M = 1 << 20  # 16-byte aligned addresses far apart; never dereferenced


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
    a = dict(q=M, q_st=None, k=2 * M, k_st=None, dt=1, B=2, S=8, hq=4, hk=2, D=64, wq=3 * M,
             wk=3 * M + 512, wdt=1, cos=4 * M, sin=5 * M, rows=8, R=64, il=1, pos=None, eps=1e-6,
             qo=6 * M, qo_st=None, ko=7 * M, ko_st=None, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.nabla_qk_norm_rope(*a.values())


def bwd(lib, **kw):
    a = dict(q=M, q_st=None, k=2 * M, k_st=None, dt=1, B=2, S=8, hq=4, hk=2, D=64, wq=3 * M,
             wk=3 * M + 512, wdt=1, cos=4 * M, sin=5 * M, rows=8, R=64, il=1, pos=None, eps=1e-6,
             dqo=8 * M, dqo_st=None, dko=9 * M, dko_st=None, dq=6 * M, dq_st=None, dk=7 * M,
             dk_st=None, dwq=10 * M, dwk=10 * M + 512, ws=11 * M, ws_bytes=1 << 22, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.nabla_qk_norm_rope_bwd(*a.values())


BAD = [dict(q=None), dict(q=M + 8), dict(k=2 * M + 2), dict(dt=2), dict(wdt=5), dict(B=0),
       dict(S=0), dict(hq=0), dict(hk=-1), dict(hk=0), dict(k=None), dict(D=96), dict(D=32),
       dict(R=-16), dict(R=8), dict(R=72), dict(R=128), dict(cos=None), dict(sin=5 * M + 4),
       dict(rows=7), dict(rows=0, pos=13 * M), dict(pos=13 * M + 2), dict(eps=-1.0),
       dict(eps=float("nan")), dict(eps=float("inf")), dict(wq=3 * M + 8),
       dict(q_st=st(8 * 256, 255)), dict(q_st=st(8 * 256, 260 * 1)), dict(q_st=st(2047, 256)),
       dict(q_st=st(7 * 256, 256)), dict(k_st=st(-8 * 128, 128)),
       dict(q_st=st(8 * 256, 256, 60)), dict(q_st=st(8 * 256, 256, 72)),
       dict(q_st=st(8 * 256, 64, 7 * 64)), dict(q_st=st(8 * 256, 256, 0)),
       dict(B=2 ** 31 - 1, S=2 ** 31 - 1)]


@pytest.mark.parametrize("kw", BAD, ids=lambda kw: "-".join(kw))
def test_bad_arguments(lib, kw):
    assert fwd(lib, **kw) == INVALID
    assert bwd(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(qo=None), dict(ko=None), dict(qo=6 * M + 4),
                                dict(qo_st=st(1024, 256)), dict(qo=M), dict(qo=M + 2 * 8 * 256),
                                dict(ko=2 * M + 16), dict(qo=3 * M), dict(ko=6 * M),
                                dict(qo=6 * M, ko=6 * M + 512, qo_st=st(8 * 320, 320),
                                     ko_st=st(8 * 320, 320))], ids=lambda kw: "-".join(kw))
def test_bad_outputs(lib, kw):
    assert fwd(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(dqo=None), dict(dko=None), dict(dqo=8 * M + 2), dict(dq=None),
                                dict(dq=8 * M), dict(dk=9 * M), dict(dq=7 * M), dict(ws=None),
                                dict(ws=11 * M + 16), dict(ws_bytes=1 << 10), dict(dwq=10 * M + 1),
                                dict(dwq=10 * M + 512), dict(dwq=3 * M), dict(dwq=6 * M),
                                dict(dko_st=st(8 * 64, 64))], ids=lambda kw: "-".join(kw))
def test_bad_gradient_arguments(lib, kw):
    assert bwd(lib, **kw) == INVALID


def test_workspace_bytes(lib):
    assert lib.nabla_qk_norm_rope_bwd_workspace_bytes(96) == 0
    assert lib.nabla_qk_norm_rope_bwd_workspace_bytes(128) > 0


def tensors(dtype=torch.bfloat16):
    q, k = torch.zeros(2, 8, 4, 64, dtype=dtype), torch.zeros(2, 8, 2, 64, dtype=dtype)
    w = torch.ones(64, dtype=dtype)
    return q, k, w, torch.ones(8, 32), torch.zeros(8, 32)


def test_binding_passes_good_tensors_up_to_the_device_check():
    q, k, w, c, s = tensors()
    pack = torch.zeros(2, 8, 8 * 64, dtype=torch.bfloat16)
    pq, pk = pack[..., :256].view(2, 8, 4, 64), pack[..., 256:384].view(2, 8, 2, 64)
    for call in (lambda: N.nabla_qk_norm_rope(q, k, w, w, c, s),
                 lambda: N.nabla_qk_norm_rope(pq, pk, w, None, c, s, interleaved=False),
                 lambda: N.nabla_qk_norm_rope(q),
                 lambda: N.nabla_qk_norm_rope(q.transpose(1, 2).contiguous().transpose(1, 2)),
                 lambda: N.nabla_qk_norm_rope(q, k, w, w, c, s, q_out=pq, k_out=pk),
                 lambda: N.nabla_qk_norm_rope(
                     q, k, w, w, c, s, pos=torch.zeros(2, 8, dtype=torch.int32)),
                 lambda: N.nabla_qk_norm_rope_bwd(q, k, w, w, q.clone(), k.clone(), c, s),
                 lambda: N.nabla_qk_norm_rope_bwd(q, None, None, None, q.clone())):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


def test_binding_refuses():
    q, k, w, c, s = tensors()
    for match, call in [
        ("q must be", lambda: N.nabla_qk_norm_rope(q[0])),
        ("k must be", lambda: N.nabla_qk_norm_rope(q, k[:, :4], w, w, c, s)),
        ("k must be torch.bfloat16", lambda: N.nabla_qk_norm_rope(q, k.float(), w, w, c, s)),
        ("k is on meta", lambda: N.nabla_qk_norm_rope(q, k.to("meta"), w, w, c, s)),
        ("lie together", lambda: N.nabla_qk_norm_rope(q.transpose(2, 3).contiguous()
                                                      .transpose(2, 3))),
        ("must not overlap", lambda: N.nabla_qk_norm_rope(q[:1].expand(2, 8, 4, 64))),
        ("wk must be torch.bfloat16", lambda: N.nabla_qk_norm_rope(q, k, w, w.float(), c, s)),
        ("wq holds", lambda: N.nabla_qk_norm_rope(q, k, w[:32], w)),
        ("wq must be", lambda: N.nabla_qk_norm_rope(q, k, torch.ones(128, dtype=q.dtype), w)),
        ("unsupported dtype", lambda: N.nabla_qk_norm_rope(q, None, w.half())),
        ("come together", lambda: N.nabla_qk_norm_rope(q, k, w, w, c)),
        ("same shape", lambda: N.nabla_qk_norm_rope(q, k, w, w, c, s[:4])),
        ("cos must be torch.float32", lambda: N.nabla_qk_norm_rope(q, k, w, w, c.double(),
                                                                   s.double())),
        ("sin must be contiguous", lambda: N.nabla_qk_norm_rope(q, k, w, w, c[:, :8].contiguous(),
                                                                s[:, :8])),
        ("pos must be", lambda: N.nabla_qk_norm_rope(q, k, w, w, c, s,
                                                     pos=torch.zeros(8, dtype=torch.int32))),
        ("pos must be torch.int32", lambda: N.nabla_qk_norm_rope(
            q, k, w, w, c, s, pos=torch.zeros(2, 8, dtype=torch.int64))),
        ("q_out must be", lambda: N.nabla_qk_norm_rope(q, k, w, w, c, s, q_out=k.clone())),
        ("k_out without k", lambda: N.nabla_qk_norm_rope(q, None, w, k_out=k)),
        ("are needed", lambda: N.nabla_qk_norm_rope_bwd(q, k, w, w, q.clone(), None, c, s)),
        ("dwk without", lambda: N.nabla_qk_norm_rope_bwd(q, k, w, None, q, k, c, s, dwk=w)),
        ("dwq must be", lambda: N.nabla_qk_norm_rope_bwd(q, k, w, w, q, k, c, s, dwq=w.float())),
        ("workspace is on meta", lambda: N.nabla_qk_norm_rope_bwd(
            q, k, w, w, q, k, c, s, workspace=torch.empty(1 << 22, dtype=torch.uint8,
                                                          device="meta"))),
    ]:
        with pytest.raises((ValueError, TypeError), match=match):
            call()


HM = 8 * 64  # a head of eight tokens, heads before tokens: [2, 6, 8, 64]


@pytest.mark.parametrize("kw", [
    dict(qo=6 * M, qo_st=st(6 * HM, 64, HM), ko=6 * M + 2 * 3 * HM, ko_st=st(6 * HM, 64, HM)),
    dict(qo=6 * M + 2 * 3 * HM, qo_st=st(6 * HM, 64, HM), ko=6 * M, ko_st=st(6 * HM, 64, HM)),
    dict(qo=6 * M, qo_st=st(6 * HM, 64, HM), ko=6 * M + 2 * 4 * HM - 16,
         ko_st=st(6 * HM, 64, HM)),
    dict(qo=6 * M, qo_st=st(9 * 384, 384), ko=6 * M + 2 * 9 * 384 + 2 * 192,
         ko_st=st(9 * 384, 384)),
    dict(q=M, q_st=st(8 * 640, 640), qo=M + 2 * 192, qo_st=st(8 * 640, 640)),
    dict(q=M, q_st=st(8 * 640, 640), qo=M + 2 * 7 * 640, qo_st=st(8 * 640, 640)),
], ids=["last head", "first head", "a piece", "next batch's head", "beside q", "q's last token"])
def test_views_that_share_elements(lib, kw):
    """Two outputs, or an output and q, as views of one tensor whose strides agree and which
    meet in some rows only."""
    assert fwd(lib, **kw) == INVALID
    names = dict(qo="dq", ko="dk", qo_st="dq_st", ko_st="dk_st")
    assert bwd(lib, **{names.get(a, a): v for a, v in kw.items()}) == INVALID
