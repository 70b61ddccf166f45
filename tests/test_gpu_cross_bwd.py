"""Cross attention backward on the GPU vs the fp64 oracle, through the binding.

The forward's o and lse (as stored) go to both sides.  Tolerances, from the arithmetic,
per element (half = half a step of the stored type: 2^-8 for bf16, 2^-24 for fp32; the
operands' rounding on the tensor cores is the stored type's too):
  scores    e_z = 2^-17 scale log2(e) sum_d |q_d k_d| in base 2 (D <= 128 products and
            sums of 2^-24, or the tensor cores' truncations of 2^-23 per 16 of them);
  P         relative e_P = 3 e_z + 2^-17 + 2^-22 |lse|: the score's error, the lse's (the
            forward's own bound, e_z + 2^-18 + 2^-23 |lse|), ex2's;
  dP, delta e_d = 2^-17 (sum_d |dout_d v_d| + sum_d |dout_d o_d|);
  dz        E = (half + e_P) |dz| + P e_d;
  dv        (half + e_P + sums) sum_s P |dout| + half |dv|,
  dq        scale (sum_u E |k| + sums sum_u |dz| |k|) + half |dq|, dk likewise over s,
with sums = 2^-14: fp32 additions of up to a thousand terms or steps (2^-24 each).
"""
import math

import numpy as np
import pytest
import torch

from oracle import nabla_oracle as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SUMS = 2.0 ** -14


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


def f64(t):
    return t.double().cpu().numpy()


def inputs(B, Sq, Sk, h, hk, D, dtype, seed=0, packed=False, spread=1.2):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[dtype]

    def draw(*shape, s=spread):
        return (torch.randn(*shape, generator=g) * s).to(dt).to(DEV)

    if packed == "heads":  # everything heads before tokens
        q, k, v, g_ = [draw(*s).transpose(1, 2) for s in
                       ((B, h, Sq, D), (B, hk, Sk, D), (B, hk, Sk, D), (B, h, Sq, D))]
        return q, k, v, g_ * 0.5
    if packed:
        q = draw(B, Sq, (h + 1) * D)[..., D:].unflatten(-1, (h, D))
        kv = draw(B, Sk, 2, hk, D)
        k, v = kv[:, :, 0], kv[:, :, 1]
    else:
        q, k, v = draw(B, Sq, h, D), draw(B, Sk, hk, D), draw(B, Sk, hk, D)
    return q, k, v, draw(B, Sq, h, D, s=0.5)


def bounds(q, k, v, o, dout, lens, scale, half):
    """The tolerances of dq, dk, dv without their own rounding, in float64."""
    B, Sq, h, D = q.shape
    G = h // k.shape[2]
    tq, tk, tv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(k.shape)
    for b in range(B):
        n = int(lens[b])
        for i in range(h if n else 0):
            j = i // G
            Q, K, V, g, Oi = q[b, :, i], k[b, :n, j], v[b, :n, j], dout[b, :, i], o[b, :, i]
            z = scale * (Q @ K.T)
            m = z.max(1, keepdims=True)
            P = np.exp(z - m)
            lse = np.abs((m + np.log(P.sum(1, keepdims=True))) / math.log(2.0))
            P /= P.sum(1, keepdims=True)
            ez = 2.0 ** -17 * abs(scale) * 1.4427 * (np.abs(Q) @ np.abs(K).T)
            eP = 3 * ez + 2.0 ** -17 + 2.0 ** -22 * lse
            ed = 2.0 ** -17 * (np.abs(g) @ np.abs(V).T + (np.abs(g * Oi)).sum(1, keepdims=True))
            dz = np.abs(P * (g @ V.T - (g * Oi).sum(1, keepdims=True)))
            E = (half + eP + SUMS) * dz + P * ed
            tq[b, :, i] = abs(scale) * (E @ np.abs(K))
            tk[b, :n, j] += abs(scale) * (E.T @ np.abs(Q))
            tv[b, :n, j] += ((half + eP + SUMS) * P).T @ np.abs(g)
    return tq, tk, tv


def check(got, q, k, v, o, dout, lens, scale):
    half = torch.finfo(q.dtype).eps / 2
    Q, K, V, Oo, G = (f64(t) for t in (q, k, v, o, dout))
    for b, n in enumerate(lens):  # what lies behind the lengths is not part of the problem
        K[b, n:] = V[b, n:] = 0.0
    ref = O.cross_attention_bwd(Q, K, V, G, lens, scale, o=Oo)
    tol = bounds(Q, K, V, Oo, G, lens, scale, half)
    for name, x, r, t in zip(("dq", "dk", "dv"), got, ref, tol):
        err = np.abs(f64(x) - r)
        worst = (err - t - half * np.abs(r)).max()
        assert worst <= 1e-37, (name, err.max(), worst)
    for b, n in enumerate(lens):
        assert (got[1][b, n:] == 0).all() and (got[2][b, n:] == 0).all()


def lengths(lens):
    return torch.tensor(lens, dtype=torch.int32, device=DEV)


CASES = [  # B, Sq, Sk, h, hk, D, lens, packed
    (1, 1, 2, 1, 1, 64, None, False),
    (1, 1, 1, 4, 1, 128, None, False),              # one state: P = 1
    (2, 300, 77, 3, 3, 128, [77, 16], False),
    (3, 129, 128, 2, 2, 64, [128, 0, 1], True),     # a full tile, an empty batch, one state
    (2, 40, 300, 6, 2, 128, [257, 128], True),      # three heads a group
    (2, 23, 130, 10, 2, 64, [129, 127], False),     # five heads a group
    (1, 700, 513, 2, 1, 128, None, True),
    (1, 5, 700, 64, 1, 64, [641], False),           # 64 heads on one key head
    (2, 900, 64, 14, 2, 128, [64, 50], False),      # seven heads a group
    (1, 2000, 200, 4, 4, 64, [199], False),
    (2, 333, 150, 4, 2, 128, [150, 90], "heads"),
    (4, 1, 2000, 24, 8, 128, [2000, 1999, 130, 0], False),  # one token each
    (3, 5, 300, 6, 2, 64, [300, 0, 65], True),      # fifteen rows a key head
    (2, 16, 129, 2, 2, 128, [129, 1], "heads"),     # sixteen
    (1, 17, 129, 2, 2, 64, None, False),            # one more
    (3, 6, 2300, 4, 4, 128, [2300, 700, 0], True),  # few rows, runs of states
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,Sq,Sk,h,hk,D,lens,packed", CASES)
def test_backward(nabla, B, Sq, Sk, h, hk, D, lens, packed, dtype):
    q, k, v, dout = inputs(B, Sq, Sk, h, hk, D, dtype, seed=Sk, packed=packed)
    n = None if lens is None else lengths(lens)
    if lens is not None:
        for b, m in enumerate(lens):
            k[b, m:] = float("nan")
            v[b, m:] = float("inf") if b % 2 else float("nan")
    o, lse = nabla.nabla_cross_attn_fwd_lse(q, k, v, kv_len=n)
    if packed == "heads":
        o = o.transpose(1, 2).contiguous().transpose(1, 2)
    got = nabla.nabla_cross_attn_bwd(q, k, v, o, lse, dout, kv_len=n)
    assert nabla.nabla_get_last_device_status() == 0
    check(got, q, k, v, o, dout, lens or [Sk] * B, 1 / math.sqrt(D))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.1])
def test_scales(nabla, dtype, scale):
    q, k, v, dout = inputs(2, 70, 200, 2, 2, 64, dtype, seed=7, spread=0.8)
    n = lengths([200, 73])
    o, lse = nabla.nabla_cross_attn_fwd_lse(q, k, v, kv_len=n, scale=scale)
    got = nabla.nabla_cross_attn_bwd(q, k, v, o, lse, dout, kv_len=n, scale=scale)
    check(got, q, k, v, o, dout, [200, 73], scale)


def test_bad_lengths_are_clamped_and_reported(nabla):
    q, k, v, dout = inputs(3, 20, 50, 2, 2, 64, "bf16", seed=9)
    good = lengths([50, 0, 50])
    o, lse = nabla.nabla_cross_attn_fwd_lse(q, k, v, kv_len=good)
    want = nabla.nabla_cross_attn_bwd(q, k, v, o, lse, dout, kv_len=good)
    assert nabla.nabla_get_last_device_status() == 0
    got = nabla.nabla_cross_attn_bwd(q, k, v, o, lse, dout, kv_len=lengths([51, -1, 50]))
    assert nabla.nabla_get_last_device_status() == 5  # NABLA_ERR_BAD_INDEX
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_repeats_streams_and_graphs(nabla, dtype):
    """Same bits from call to call, on another stream, and from two graphs with a
    workspace each; a replay reads the lengths anew."""
    B, Sq, Sk, h, hk, D = 2, 1500, 130, 6, 2, 128
    q, k, v, dout = inputs(B, Sq, Sk, h, hk, D, dtype, seed=10)
    n = lengths([130, 67])
    o, lse = nabla.nabla_cross_attn_fwd_lse(q, k, v, kv_len=n)
    want = nabla.nabla_cross_attn_bwd(q, k, v, o, lse, dout, kv_len=n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = nabla.nabla_cross_attn_bwd(q, k, v, o, lse, dout, kv_len=n, stream=side)
    side.synchronize()
    need = nabla.nabla_cross_attn_bwd_workspace_bytes(q.dtype, B, Sq, Sk, h, hk, D)
    runs = []
    for _ in range(2):
        outs = [torch.zeros_like(t) for t in want]
        ws = torch.empty(need, dtype=torch.uint8, device=DEV)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            nabla.nabla_cross_attn_bwd(q, k, v, o, lse, dout, kv_len=n, dq=outs[0], dk=outs[1],
                                       dv=outs[2], workspace=ws)
        runs.append((graph, outs, ws))
    with torch.cuda.stream(side):
        runs[0][0].replay()
    runs[1][0].replay()
    torch.cuda.synchronize()
    for a, b, c, d in zip(want, other, runs[0][1], runs[1][1]):
        assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, d)
    n.copy_(lengths([12, 130]))
    fresh = nabla.nabla_cross_attn_bwd(q, k, v, o, lse, dout, kv_len=n)
    runs[0][0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(fresh, runs[0][1]))


def test_gradient_against_differences(nabla):
    """Central differences of sum(dout * o) with the fp32 forward itself, whose rows are
    off by at most (2 e_z + 2^-17) A <= 2^-13 here (see the forward's test), so the
    quotient is off by sum |dout| 2^-13 / step; the third-order term is below 1e-3."""
    B, Sq, Sk, h, hk, D = 1, 3, 9, 2, 1, 64
    q, k, v, dout = inputs(B, Sq, Sk, h, hk, D, "f32", seed=3, spread=0.5)
    dout = dout * 0.05
    n = lengths([8])
    o, lse = nabla.nabla_cross_attn_fwd_lse(q, k, v, kv_len=n)
    grads = nabla.nabla_cross_attn_bwd(q, k, v, o, lse, dout, kv_len=n)

    def loss(q, k, v):
        return float((nabla.nabla_cross_attn_fwd(q, k, v, kv_len=n).double() *
                      dout.double()).sum())

    step = 0.25
    tol = float(dout.abs().sum()) * 2.0 ** -13 / step + 1e-3
    for which, at in [(0, (0, 1, 1, 5)), (0, (0, 2, 0, 63)), (1, (0, 3, 0, 7)), (1, (0, 8, 0, 0)),
                      (2, (0, 0, 0, 31)), (2, (0, 7, 0, 9))]:
        hi, lo = [q, k, v], [q, k, v]
        e = torch.zeros_like(hi[which])
        e[at] = step
        hi[which], lo[which] = hi[which] + e, lo[which] - e
        got = (loss(*hi) - loss(*lo)) / (2 * step)
        assert abs(got - float(grads[which][at])) <= tol


def loss64(q, k, v, dout, lens, scale):
    """<dout, o> by the definition, in 64 bits (none of the oracle)."""
    total = 0.0
    for b, n in enumerate(lens):
        if n:
            rep = q.shape[2] // k.shape[2]
            z = torch.einsum("shd,uhd->hsu", q[b], k[b, :n].repeat_interleave(rep, 1)) * scale
            o = torch.einsum("hsu,uhd->shd", z.softmax(-1), v[b, :n].repeat_interleave(rep, 1))
            total += float((dout[b] * o).sum())
    return total


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,Sq,Sk,h,hk,D,lens,scale", [
    (2, 3, 9, 4, 2, 64, [8, 5], None),      # few rows
    (3, 70, 150, 4, 2, 64, [150, 0, 33], None),
    (1, 200, 77, 3, 1, 128, [60], -0.07),
    (2, 5, 1100, 2, 2, 128, [1100, 700], 0.2),
])
def test_gradient_along_directions(nabla, B, Sq, Sk, h, hk, D, lens, scale, dtype):
    """<gradient, d> of q, k and v, one at a time, against central differences of the
    definition in 64 bits, along the gradient itself and along the halves of it that a
    random choice of elements gives, d of length 1.  So the probe reads |d g|^2 / |d g|, a
    half of the gradient's length or more, and a gradient that is 0, turned round, or off by
    a factor in any large part of its elements is off by as much.

    Tolerance, of the gradient's length: a gradient off by e elementwise moves the probe by
    at most |e|.  fp32, by norm: scores and dP carry the roundings of 64 products a lane
    (2^-21 of their size), lse 2^-21 at sizes to 16, ex2 2^-22, the sums over tens of tiles
    less than 2^-20: below 2^-18 together, where scores spread over a few units; twice that
    for o's and lse's own.  bf16: P, dz and the result are rounded by at most 2^-8 each, and
    delta, from a rounded o, by 2^-8 of |dout| |o|, which is of dz's size: 2^-6.
    The differences: step^2 / 6 of a third derivative of the first one's size, below 2^-22."""
    scale = 1 / math.sqrt(D) if scale is None else scale
    q, k, v, dout = inputs(B, Sq, Sk, h, hk, D, dtype, seed=Sk, spread=0.9)
    n = lengths(lens)
    o, lse = nabla.nabla_cross_attn_fwd_lse(q, k, v, kv_len=n, scale=scale)
    grads = nabla.nabla_cross_attn_bwd(q, k, v, o, lse, dout, kv_len=n, scale=scale)
    step, tol = 2.0 ** -11, 2.0 ** -6 if dtype == "bf16" else 2.0 ** -17
    x = [t.double() for t in (q, k, v)]
    gen = torch.Generator().manual_seed(Sq)
    for which, grad in enumerate(grads):
        g = grad.double()
        pick = (torch.rand(g.shape, generator=gen) < 0.5).to(DEV)
        for part in (torch.ones_like(pick), pick, ~pick):
            d = torch.where(part, g, torch.zeros_like(g))
            length = float(d.norm())
            assert length >= 0.5 * float(g.norm()) > 0 and 10 * tol * float(g.norm()) <= length
            d /= length
            hi, lo = list(x), list(x)
            hi[which], lo[which] = x[which] + step * d, x[which] - step * d
            got = (loss64(*hi, dout.double(), lens, scale) -
                   loss64(*lo, dout.double(), lens, scale)) / (2 * step)
            assert abs(got - float((g * d).sum())) <= tol * float(g.norm()), (which, got, length)
    for b, m in enumerate(lens):
        assert (grads[1][b, m:] == 0).all() and (grads[2][b, m:] == 0).all()
        assert m or (grads[0][b] == 0).all()
