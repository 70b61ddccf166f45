"""A block of differential attention run whole, forward and backward, as a user's program does:

  adaptive norm -> projection -> norm and rotation of q, k -> differential attention of the
  tokens to themselves -> norm of every head's row -> projection -> gated, normed sum with the
  residual and the next adaptive norm, and all the way back, projections by matrix products.

Values, fp32: the outputs and every gradient against the fp64 oracle through the same chain,
by norm.  Tolerance 2^-9: a base-2 score here is at most 30, so it is off by at most 2^-17 of
that, which moves P, and with it a stage's result, by at most 3 * 30 * 2^-17 < 2^-10.5 of its
norm where every error had the same sign; over some 10^4 elements they have not, and the sum
over the chain's softmaxes, norms and their backwards stays below 4 times the root mean
square of one stage's, 2^-13, times 4 stages.  A wrong term is off by O(1).

Order, bf16 and fp32: the chain without a synchronisation, on another stream, and captured
into a graph whose inputs change between replays gives the bits of the chain run with a
synchronisation after every call.
"""
import numpy as np
import pytest
import torch

from oracle import nabla_oracle as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
B, S, H, EPS = 2, 150, 3, 1e-6
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
        dt, C = TYPES[dtype], H * D

        def draw(*shape, s=1.0, m=0.0, kind=dt):
            return (torch.randn(*shape, generator=g) * s + m).to(kind).to(DEV)

        self.x, self.ds, self.dy = draw(B, S, C), draw(B, S, C), draw(B, S, C)
        self.mod = draw(B, 5, C, s=0.3, kind=torch.float32)  # of the two norms, and the gate
        self.w_in, self.w_out = draw(C, 3 * C, s=C ** -0.5), draw(C, C, s=C ** -0.5)
        self.wq, self.wk, self.wo, self.pw = (draw(n, s=0.2, m=1.0) for n in (D, D, D, C))
        self.lam = draw(H, s=0.2, m=0.6, kind=torch.float32)
        a = np.random.default_rng(seed).uniform(-300.0, 300.0, (S, D // 4))
        self.cos = torch.from_numpy(np.cos(a)).float().to(DEV)
        self.sin = torch.from_numpy(np.sin(a)).float().to(DEV)

    def tensors(self):
        return [self.x, self.ds, self.dy, self.mod, self.lam]


def chain(N, t, done=lambda: None):
    """s, y and the gradients of <ds, s> + <dy, y>."""
    D, C = t.wq.numel(), t.x.shape[-1]
    m = [t.mod[:, i] for i in range(5)]
    _, a = N.nabla_block_norm(t.x, scale=m[0], shift=m[1], norm="layer", eps=EPS)
    done()
    qkv = (a.view(B * S, C) @ t.w_in).view(B, S, 3, H, D)
    q, k, v = (qkv[:, :, i] for i in range(3))
    wq, wk = t.wq, t.wk
    qn, kn = N.nabla_qk_norm_rope(q, k, wq, wk, t.cos, t.sin, eps=EPS)
    done()
    o, o2, lse = N.nabla_diff_attn_fwd_lse(qn, kn, v, t.lam)
    done()
    on, _ = N.nabla_qk_norm_rope(o, None, t.wo, eps=EPS)
    done()
    u = (on.view(B * S, C) @ t.w_out).view(B, S, C)
    args = dict(gate=m[2], scale=m[3], shift=m[4], post_weight=t.pw, norm="layer",
                post_norm="rms", residual_scale=0.8, eps=EPS)
    s, y = N.nabla_block_norm(t.x, u, **args)
    done()
    dx, du, dgate, dscale, dshift, _, dpw = N.nabla_block_norm_bwd(s, u, t.ds, t.dy, **args)
    done()
    d_out = on.view(B * S, C).t() @ du.view(B * S, C)
    don = (du.view(B * S, C) @ t.w_out.t()).view(B, S, H, D)
    do, _, dwo, _ = N.nabla_qk_norm_rope_bwd(o, None, t.wo, None, don, eps=EPS)
    done()
    dqn, dkn, dv, dlam = N.nabla_diff_attn_bwd(qn, kn, v, t.lam, o, o2, lse, do)
    done()
    dqkv = torch.empty(B, S, 3, H, D, dtype=t.x.dtype, device=DEV)
    _, _, dwq, dwk = N.nabla_qk_norm_rope_bwd(q, k, wq, wk, dqn, dkn, t.cos, t.sin, eps=EPS,
                                              dq=dqkv[:, :, 0], dk=dqkv[:, :, 1])
    dqkv[:, :, 2].copy_(dv)
    done()
    d_in = a.view(B * S, C).t() @ dqkv.view(B * S, 3 * C)
    da = (dqkv.view(B * S, 3 * C) @ t.w_in.t()).view(B, S, C)
    dx, _, _, dscale0, dshift0, _, _ = N.nabla_block_norm_bwd(t.x, None, dx, da, scale=m[0],
                                                              shift=m[1], norm="layer", eps=EPS)
    done()
    return [s, y, dx, dgate, dscale, dshift, dpw, dwo, dwq, dwk, dlam, d_in, d_out, dscale0,
            dshift0]


def expected(t):
    x, ds, dy, mod, w_in, w_out, wq, wk, wo, pw, lam, c, s = (
        v.double().cpu().numpy() for v in (t.x, t.ds, t.dy, t.mod, t.w_in, t.w_out, t.wq, t.wk,
                                           t.wo, t.pw, t.lam, t.cos, t.sin))
    D, C = wq.size, x.shape[-1]
    m = [mod[:, i] for i in range(5)]
    c, s, none = c[None], s[None], np.zeros((1, S, 0))
    _, a = O.block_norm(x, None, None, m[0], m[1], None, None, "layer", None, 1.0, EPS)
    qkv = (a @ w_in).reshape(B, S, 3, H, D)
    q, k, v = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
    qn, kn = (O.qk_norm_rope(z, w, c, s, True, EPS) for z, w in ((q, wq), (k, wk)))
    scale, lens = np.sqrt(2.0 / D), [S] * B
    o, o2, _ = O.diff_attention(qn, kn, v, lam, lens, scale)
    on = O.qk_norm_rope(o, wo, none, none, True, EPS)
    u = on.reshape(B, S, C) @ w_out
    rest = (None, pw, "layer", "rms", 0.8, EPS)
    sm, y = O.block_norm(x, u, m[2], m[3], m[4], *rest)
    dx, du, dgate, dscale, dshift, _, dpw = O.block_norm_bwd(sm, u, ds, dy, m[2], m[3], m[4],
                                                             *rest)
    d_out = on.reshape(B * S, C).T @ du.reshape(B * S, C)
    do, dwo = O.qk_norm_rope_bwd(o, wo, (du @ w_out.T).reshape(B, S, H, D), none, none, True, EPS)
    dqn, dkn, dv, dlam = O.diff_attention_bwd(qn, kn, v, lam, do, lens, scale, o=o, o2=o2)
    dq, dwq = O.qk_norm_rope_bwd(q, wq, dqn, c, s, True, EPS)
    dk, dwk = O.qk_norm_rope_bwd(k, wk, dkn, c, s, True, EPS)
    dqkv = np.stack([dq, dk, dv], axis=2).reshape(B * S, 3 * C)
    d_in = a.reshape(B * S, C).T @ dqkv
    dx, _, _, dscale0, dshift0, _, _ = O.block_norm_bwd(
        x, None, dx, (dqkv @ w_in.T).reshape(B, S, C), None, m[0], m[1], None, None, "layer",
        None, 1.0, EPS)
    return [sm, y, dx, dgate, dscale, dshift, dpw, dwo, dwq, dwk, dlam, d_in, d_out, dscale0,
            dshift0]


@pytest.fixture
def exact_products():
    before = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    yield
    torch.backends.cuda.matmul.allow_tf32 = before


@pytest.mark.parametrize("D", [64, 128])
def test_values(nabla, D, exact_products):
    t = Inputs(D, "f32", 1)
    got = chain(nabla, t)
    assert nabla.nabla_get_last_device_status() == 0
    for i, (a, want) in enumerate(zip(got, expected(t))):
        a = a.double().cpu().numpy()
        assert a.shape == want.shape
        assert np.linalg.norm(a - want) <= TOL * np.linalg.norm(want), i


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("f32", 64)])
def test_order(nabla, dtype, D):
    x, y = Inputs(D, dtype, 2), Inputs(D, dtype, 3)
    for n in ("w_in", "w_out", "wq", "wk", "wo", "pw", "cos", "sin"):
        setattr(y, n, getattr(x, n))
    want = [chain(nabla, t, torch.cuda.synchronize) for t in (x, y)]
    torch.cuda.synchronize()
    got = chain(nabla, x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = chain(nabla, y)
    torch.cuda.synchronize()
    for a, b in zip(want[0] + want[1], got + other):
        assert torch.equal(a, b)
    live = Inputs(D, dtype, 2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = chain(nabla, live)
    for new, ref in ((x, want[0]), (y, want[1]), (x, want[0])):
        for t, n in zip(live.tensors(), new.tensors()):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(ref, outs):
            assert torch.equal(a, b)
    assert nabla.nabla_get_last_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("handles", [False, True], ids=["objects", "handles"])
def test_overlapping_calls_keep_their_memory(nabla, dtype, handles):
    """Calls on three streams that allocate their own scratch and outputs, while the current
    stream writes memory of the same sizes, give the bits of the same calls in order."""
    def operators(seed):
        g = torch.Generator().manual_seed(seed)

        def draw(*shape, kind=dtype):
            return torch.randn(*shape, generator=g).to(kind).to(DEV)

        x, u, ds, dy = (draw(2, 700, 512) for _ in range(4))
        p, w = draw(2, 3, 512, kind=torch.float32), draw(512)
        args = dict(gate=p[:, 0], scale=p[:, 1], shift=p[:, 2], weight=w, post_weight=w,
                    norm="layer", post_norm="rms")
        q, k, v, do = (draw(1, 900, 4, 64) for _ in range(4))
        sq, sk, sv = draw(2, 2, 6, 128), draw(2, 3000, 2, 128), draw(2, 3000, 2, 128)
        lam = torch.rand(4, generator=g).to(DEV)
        f = nabla.nabla_diff_attn_fwd_lse(q, k, v, lam)
        torch.cuda.synchronize()
        return [
            lambda s: nabla.nabla_block_norm(x, u, stream=s, **args),
            lambda s: nabla.nabla_block_norm_bwd(x, u, ds, dy, stream=s, **args),
            lambda s: nabla.nabla_diff_attn_fwd_lse(sq, sk, sv, lam[:1], stream=s),
            lambda s: nabla.nabla_diff_attn_bwd(q, k, v, lam, *f, do, stream=s),
        ]

    ops = [operators(i) for i in range(3)]
    want = [[[t.clone() for t in op(None)] for op in row] for row in ops]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(3)]
    got = [[None] * len(row) for row in ops]
    for j in range(len(ops[0])):
        for i, side in enumerate(sides):
            outs = ops[i][j](side.cuda_stream if handles else side)
            noise = [torch.full((1 << 20,), 3.0, device=DEV) for _ in range(4)]
            with torch.cuda.stream(side):
                got[i][j] = [t.clone() for t in outs]
            del outs, noise
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert all(torch.equal(s, t) for s, t in zip(x, y))
