"""fp32 cross attention by norm against the definition in 64 bits: every output is within
the bound that fp32_model derives from the kernels' own sums (the elementwise bounds of the
other tests leave room for worst cases hundreds of times as large).  Some cases have
thousands of states, or of rows to a key head, in one run, where a sum that is not folded
would be off by more (test_fp32_model.py)."""
import math

import pytest
import torch

import fp32_model as M

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def nabla():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    from block_sparse_attention_nablat_gb300 import nabla as N

    try:
        N.load()
    except RuntimeError:
        __graft_entry__.build()
        N.load()
    return N


def inputs(B, Sq, Sk, h, hk, D, spread):
    g = torch.Generator().manual_seed(Sk + D)

    def draw(s, *shape):
        return (torch.randn(*shape, generator=g) * s).to(DEV)

    return (draw(spread, B, Sq, h, D), draw(spread, B, Sk, hk, D), draw(1.0, B, Sk, hk, D),
            draw(0.5, B, Sq, h, D))


def heads(x, b, j, G):
    """The rows of key head j's group in batch b, [G Sq, D] in 64 bits."""
    return x[b, :, j * G:(j + 1) * G].double().reshape(-1, x.shape[-1])


def exact(q, k, v, dout=None):
    """o, or dq, dk and dv, in 64 bits."""
    G, D = q.shape[2] // k.shape[2], q.shape[3]
    o, dk, dv = (torch.zeros(t.shape, dtype=torch.float64, device=DEV) for t in (q, k, v))
    for b in range(q.shape[0]):
        for j in range(k.shape[2]):
            Q, K, V = heads(q, b, j, G), k[b, :, j].double(), v[b, :, j].double()
            P = torch.softmax(Q @ K.T / math.sqrt(D), -1)
            rows = P @ V
            if dout is not None:
                g = heads(dout, b, j, G)
                dP = g @ V.T
                dz = P * (dP - (P * dP).sum(-1, keepdim=True)) / math.sqrt(D)
                rows = dz @ K
                dk[b, :, j], dv[b, :, j] = dz.T @ Q, P.T @ g
            o[b, :, j * G:(j + 1) * G] = rows.view(-1, G, D)
    return o if dout is None else (o, dk, dv)


def off(x, want):
    return float((x.double() - want).norm() / want.norm())


ORDINARY = [(2, 300, 77, 3, 3, 128, 1.0), (3, 70, 500, 4, 2, 64, 1.0), (2, 16, 640, 2, 2, 128, 1.0),
            (2, 500, 130, 6, 2, 128, 0.7), (5, 1, 900, 24, 8, 64, 1.0)]


@pytest.mark.parametrize("B,Sq,Sk,h,hk,D,spread", ORDINARY + [
    (1, 2048, 7200, 8, 8, 64, 0.5),   # thousands of states in one run
    (2, 2432, 7200, 4, 4, 128, 0.5),
    (160, 2, 7200, 1, 1, 64, 0.5),    # the form for few rows
    (40, 3, 7200, 8, 4, 128, 0.5),
    (80, 16, 7200, 2, 2, 64, 0.5),
    (1, 300, 7200, 2, 2, 64, 0.5),    # runs, joined
])
def test_forward(nabla, B, Sq, Sk, h, hk, D, spread):
    q, k, v, _ = inputs(B, Sq, Sk, h, hk, D, spread)
    o = nabla.nabla_cross_attn_fwd(q, k, v)
    z = spread * spread / M.LN2
    assert off(o, exact(q, k, v)) <= M.forward(Sk, D, z)


@pytest.mark.parametrize("B,Sq,Sk,h,hk,D,spread", ORDINARY + [
    (1, 600, 7200, 2, 2, 64, 0.5),    # thousands of states
    (2, 333, 7200, 4, 2, 128, 0.5),
    (40, 3, 7200, 8, 4, 128, 0.5),    # the form for few rows
    (1, 7200, 100, 2, 2, 64, 0.5),    # thousands of rows a key head
    (30, 3600, 64, 4, 2, 128, 0.5),
])
def test_backward(nabla, B, Sq, Sk, h, hk, D, spread):
    q, k, v, dout = inputs(B, Sq, Sk, h, hk, D, spread)
    o, lse = nabla.nabla_cross_attn_fwd_lse(q, k, v)
    got = nabla.nabla_cross_attn_bwd(q, k, v, o, lse, dout)
    z, top = spread * spread / M.LN2, float(lse.abs().max())
    for name, x, want, n in zip(("dq", "dk", "dv"), got, exact(q, k, v, dout),
                                (Sk, Sq * (h // hk), Sq * (h // hk))):
        assert off(x, want) <= M.gradient(n, D, z, top), name
