"""The operators of a transformer block run together, forward and backward:

  packed projection -> norm and rotation of q, k -> mask -> block-sparse attention
  -> cross attention of its rows to packed encoder states, and all the way back.

Values, fp32: the forward's o and every gradient of <g, o> against the fp64 oracle run
through the same chain with the mask the device chose, by norm.  Tolerance 2^-9: a base-2
score here is at most 30, so it is off by at most 2^-17 of that (the operators' own tests
derive this), which moves P, and with it a stage's result, by at most 3 * 30 * 2^-17 <
2^-10.5 of its norm where every error had the same sign; over some 10^5 elements they have
not, and the sum over the chain's two softmaxes and their backwards stays below 4 times
the root mean square of one stage's, 2^-13, times 4 stages.  A wrong term is off by O(1).

Order, bf16 and fp32: the chain without a synchronisation, on another stream, and captured
into a graph whose inputs change between replays gives the bits of the chain run with a
synchronisation after every call.
"""
import math

import numpy as np
import pytest
import torch

from oracle import nabla_oracle as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
B, S, H, HK, SK = 2, 256, 3, 1, 77
LENS = [77, 30]
TOL = 2.0 ** -9


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


class Inputs:
    def __init__(self, D, dtype, seed):
        g = torch.Generator().manual_seed(seed)
        dt = TYPES[dtype]

        def draw(*shape, s=1.0):
            return (torch.randn(*shape, generator=g) * s).to(dt).to(DEV)

        self.qkv = draw(B, S, 3, H, D)
        self.wq, self.wk = 1 + draw(D, s=0.2), 1 + draw(D, s=0.2)
        self.enc = draw(B, SK, 2, HK, D)
        self.g = draw(B, S, H, D)
        a = np.random.default_rng(seed).uniform(-300.0, 300.0, (S, D // 2))
        self.cos = torch.from_numpy(np.cos(a)).float().to(DEV)
        self.sin = torch.from_numpy(np.sin(a)).float().to(DEV)
        self.lens = torch.tensor(LENS, dtype=torch.int32, device=DEV)
        self.sta = torch.from_numpy(O.sta_mask(4, 1, 1, 1, 1, 1).astype(np.uint8)).to(DEV)

    def tensors(self):
        return [self.qkv, self.wq, self.wk, self.enc, self.g]


def chain(N, x, done=lambda: None):
    """o, the mask and the gradients of <g, o> for qkv, wq, wk and enc's k and v."""
    q, k = x.qkv[:, :, 0], x.qkv[:, :, 1]
    v = x.qkv[:, :, 2].contiguous()
    ek, ev = x.enc[:, :, 0], x.enc[:, :, 1]
    qn, kn = N.nabla_qk_norm_rope(q, k, x.wq, x.wk, x.cos, x.sin)
    done()
    nb, inds = N.nabla_build_mask(qn, kn, x.sta, 0.3)
    done()
    o1, lse1 = N.nabla_attn_fwd_lse(qn, kn, v, nb, inds)
    done()
    o, lse = N.nabla_cross_attn_fwd_lse(o1, ek, ev, x.lens)
    done()
    do1, dek, dev = N.nabla_cross_attn_bwd(o1, ek, ev, o, lse, x.g, kv_len=x.lens)
    done()
    dqn, dkn, dv = N.nabla_attn_bwd(qn, kn, v, o1, do1, nb, inds, lse=lse1)
    done()
    dqkv = torch.empty_like(x.qkv)
    _, _, dwq, dwk = N.nabla_qk_norm_rope_bwd(q, k, x.wq, x.wk, dqn, dkn, x.cos, x.sin,
                                              dq=dqkv[:, :, 0], dk=dqkv[:, :, 1])
    dqkv[:, :, 2].copy_(dv)
    done()
    return [o, dqkv, dwq, dwk, dek, dev], (nb, inds)


def expected(x, mask):
    qkv, enc, g = (t.double().cpu().numpy() for t in (x.qkv, x.enc, x.g))
    wq, wk, c, s = (t.double().cpu().numpy() for t in (x.wq, x.wk, x.cos, x.sin))
    c, s, scale = c[None], s[None], 1.0 / math.sqrt(qkv.shape[-1])
    nb, inds = (t.cpu().numpy() for t in mask)
    q, k, v = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
    qn, kn = (O.qk_norm_rope(t, w, c, s, True, 1e-6) for t, w in ((q, wq), (k, wk)))
    o1 = O.block_sparse_attention(qn, kn, v, nb, inds, scale)
    ek, ev = enc[:, :, 0], enc[:, :, 1]
    o, _ = O.cross_attention(o1, ek, ev, LENS, scale)
    do1, dek, dev = O.cross_attention_bwd(o1, ek, ev, g, LENS, scale)
    dqn, dkn, dv = O.block_sparse_attention_bwd(qn, kn, v, do1, nb, inds, scale)
    dq, dwq = O.qk_norm_rope_bwd(q, wq, dqn, c, s, True, 1e-6)
    dk, dwk = O.qk_norm_rope_bwd(k, wk, dkn, c, s, True, 1e-6)
    return [o, np.stack([dq, dk, dv], axis=2), dwq, dwk, dek, dev]


@pytest.mark.parametrize("D", [64, 128])
def test_values(nabla, D):
    x = Inputs(D, "f32", 1)
    got, mask = chain(nabla, x)
    assert nabla.nabla_get_last_device_status() == 0
    nb = mask[0].cpu().numpy()
    assert nb.min() >= 1 and nb.min() < S // 64  # the mask leaves blocks out
    for a, want in zip(got, expected(x, mask)):
        a = a.double().cpu().numpy()
        assert np.linalg.norm(a - want) <= TOL * np.linalg.norm(want)


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("f32", 64)])
def test_order(nabla, dtype, D):
    x, y = Inputs(D, dtype, 2), Inputs(D, dtype, 3)
    y.cos, y.sin = x.cos, x.sin
    want = [chain(nabla, t, torch.cuda.synchronize)[0] for t in (x, y)]
    torch.cuda.synchronize()
    got, _ = chain(nabla, x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other, _ = chain(nabla, y)
    torch.cuda.synchronize()
    for a, b in zip(want[0] + want[1], got + other):
        assert torch.equal(a, b)
    live = Inputs(D, dtype, 2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs, _ = chain(nabla, live)
    for new, ref in ((x, want[0]), (y, want[1]), (x, want[0])):
        for t, n in zip(live.tensors(), new.tensors()):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(ref, outs):
            assert torch.equal(a, b)
    assert nabla.nabla_get_last_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_past_32_bits(nabla, dtype):
    """Rows more than 2^31 elements apart give the bits of the dense call."""
    n, h, D = 260, 2, 64
    pitch = 2 ** 31 // (n - 1) // 8 * 8 + 64  # of a token, elements
    assert (n - 2) * pitch <= 2 ** 31 < (n - 1) * pitch
    g = torch.Generator().manual_seed(5)
    dense = [torch.randn(1, n, h, D, generator=g).to(TYPES[dtype]).to(DEV) for _ in range(4)]

    def far(t=None):
        room = torch.empty((n - 1) * pitch + h * D, dtype=TYPES[dtype], device=DEV)
        view = room.as_strided((1, n, h, D), (room.numel(), pitch, D, 1))
        if t is not None:
            view.copy_(t)
        return view

    q, k, v, go = dense
    fq, fk, fv, fg = [far(t) for t in dense]
    w = torch.rand(D, generator=g).to(TYPES[dtype]).to(DEV)
    zq, zk = nabla.nabla_qk_norm_rope(q, k, w, w)
    yq, yk = nabla.nabla_qk_norm_rope(fq, fk, w, w, q_out=far(), k_out=far())
    assert torch.equal(zq, yq) and torch.equal(zk, yk)
    want = nabla.nabla_qk_norm_rope_bwd(q, k, w, w, go, v)
    got = nabla.nabla_qk_norm_rope_bwd(fq, fk, w, w, fg, fv, dq=yq, dk=yk)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    o, lse = nabla.nabla_cross_attn_fwd_lse(q, k, v)
    p, pse = nabla.nabla_cross_attn_fwd_lse(fq, fk, fv)
    assert torch.equal(o, p) and torch.equal(lse, pse)
    yq.copy_(o)
    want = nabla.nabla_cross_attn_bwd(q, k, v, o, lse, go)
    got = nabla.nabla_cross_attn_bwd(fq, fk, fv, yq, lse, fg)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert nabla.nabla_get_last_device_status() == 0
