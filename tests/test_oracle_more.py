"""Pins of the oracle's gated sum with adaptive norm and of its differential attention
(CPU, no GPU), by means that share none of its formulas: torch's own norms and softmax
attention in 64 bits, automatic differentiation, hand-worked rows and central differences.
"""
import numpy as np
import pytest
import torch

from oracle import nabla_oracle as O


def norm_of(t, kind, eps):
    if kind is None:
        return t
    if kind == "layer":
        return torch.nn.functional.layer_norm(t, t.shape[-1:], eps=eps)
    return torch.nn.functional.rms_norm(t, t.shape[-1:], eps=eps)


CASES = [  # norm, post, modulations, weights, branch
    ("layer", None, "batch", False, True), ("rms", "rms", "frames", True, True),
    ("layer", "layer", "one", True, True), ("rms", "layer", None, True, True),
    (None, "rms", "tokens", True, True), (None, None, "batch", False, True),
    ("layer", None, "frames", True, False), ("rms", None, None, False, False),
]


@pytest.mark.parametrize("norm,post,mod,weights,branch", CASES)
def test_block_norm_and_its_gradients(norm, post, mod, weights, branch):
    B, S, C, eps, rs = 2, 6, 8, 1e-3, 0.7
    g = torch.Generator().manual_seed(1)

    def draw(*shape):
        return torch.randn(*shape, generator=g, dtype=torch.float64).requires_grad_()

    shape = {"one": (C,), "batch": (B, C), "frames": (B, 3, C), "tokens": (B, S, C)}.get(mod)
    x, u = draw(B, S, C), draw(B, S, C) if branch else None
    gate = draw(*shape) if shape and branch else None
    scale, shift = (draw(*shape), draw(*shape)) if shape and norm else (None, None)
    w = draw(C) if weights and norm else None
    pw = draw(C) if weights and post else None

    def spread(m):
        if m.dim() == 3:
            return m.repeat_interleave(S // m.shape[1], 1)
        return m[:, None] if m.dim() == 2 else m

    s = x
    if branch:
        b = norm_of(u, post, eps)
        b = b if pw is None else b * pw
        s = x + rs * (b if gate is None else b * spread(gate))
    y = None
    if norm:
        y = norm_of(s, norm, eps)
        y = y if w is None else y * w
        y = y if scale is None else y * (1 + spread(scale)) + spread(shift)
    n = [None if t is None else t.detach().numpy() for t in (x, u, gate, scale, shift, w, pw)]
    gs, gy = O.block_norm(*n, norm, post, rs, eps)
    assert np.allclose(gs, s.detach().numpy(), atol=1e-12)
    assert norm is None or np.allclose(gy, y.detach().numpy(), atol=1e-12)
    dsum, dy = (torch.randn(B, S, C, generator=g, dtype=torch.float64) for _ in range(2))
    ((s * dsum).sum() + (0 if y is None else (y * dy).sum())).backward()
    got = O.block_norm_bwd(gs, n[1], dsum.numpy(), None if norm is None else dy.numpy(), *n[2:],
                           norm, post, rs, eps)
    for a, t in zip(got, (x, u, gate, scale, shift, w, pw)):
        assert (a is None) == (t is None)
        if t is not None:
            assert a.shape == tuple(t.shape) and np.allclose(a, t.grad.numpy(), atol=1e-11)


def test_norm_of_hand_worked_rows():
    x = np.array([1.0, 3.0, 5.0, 7.0]).reshape(1, 1, 4)      # mean 4, variance 5
    _, y = O.block_norm(x, None, None, None, None, None, None, "layer", None, 1.0, 0.0)
    assert np.allclose(y.ravel() * np.sqrt(5.0), [-3, -1, 1, 3], atol=1e-14)
    s, y = O.block_norm(x, x, np.array([2.0, 0, 1, -1]), np.full(4, 1.0), np.full(4, 0.5), None,
                        None, "rms", None, 0.5, 0.0)
    assert np.allclose(s.ravel(), [2.0, 3.0, 7.5, 3.5], atol=1e-14)
    r = np.sqrt((4 + 9 + 56.25 + 12.25) / 4)
    assert np.allclose(y.ravel(), s.ravel() / r * 2 + 0.5, atol=1e-14)


def diff_inputs(seed, B=3, Sq=4, Sk=7, h=6, hk=2, D=6, lens=(7, 3, 0), one=False):
    rng = np.random.default_rng(seed)
    q, dout = rng.standard_normal((2, B, Sq, h, D))
    k, v = rng.standard_normal((2, B, Sk, hk, D))
    return q, k, v, rng.uniform(0.2, 0.9, 1 if one else h), dout, np.array(lens)


def torch_diff(q, k, v, lam, lens, scale):
    """The library's own attention for each map, one batch at a time, key heads repeated."""
    outs, d = [], q.shape[-1] // 2
    for b, n in enumerate(lens):
        if n == 0:
            outs.append(torch.zeros_like(q[b]))
            continue
        rep = q.shape[2] // k.shape[2]
        kk, vv = (t[b, :n].repeat_interleave(rep, 1).transpose(0, 1) for t in (k, v))
        qq = q[b].transpose(0, 1)
        a, c = (torch.nn.functional.scaled_dot_product_attention(
            qq[..., at], kk[..., at], vv, scale=scale) for at in (slice(0, d), slice(d, None)))
        outs.append((a - lam[:, None, None] * c).transpose(0, 1))
    return torch.stack(outs)


@pytest.mark.parametrize("one", [False, True])
def test_diff_attention_matches_torch_and_its_gradients(one):
    q, k, v, lam, dout, lens = diff_inputs(3, one=one)
    t = [torch.from_numpy(x).requires_grad_() for x in (q, k, v, lam)]
    ref = torch_diff(*t, lens, 0.7)
    o, o2, lse = O.diff_attention(q, k, v, lam, lens, 0.7)
    assert np.allclose(o, ref.detach().numpy(), atol=1e-13)
    assert np.all(o[2] == 0) and np.all(o2[2] == 0) and np.all(np.isneginf(lse[2]))
    ref.backward(torch.from_numpy(dout))
    for given in (dict(), dict(o=o, o2=o2)):
        for got, x in zip(O.diff_attention_bwd(q, k, v, lam, dout, lens, 0.7, **given), t):
            assert got.shape == tuple(x.shape) and np.allclose(got, x.grad.numpy(), atol=1e-12)


def test_diff_lse_rebuilds_the_weights():
    q, k, _, _, _, lens = diff_inputs(4)
    v = np.random.default_rng(5).standard_normal(k.shape)
    _, _, lse = O.diff_attention(q, k, v, np.full(6, 0.5), lens, 0.5)
    for b, i, m, s in [(0, 0, 0, 0), (0, 5, 1, 3), (1, 2, 1, 1)]:
        z = 0.5 * (k[b, :lens[b], i // 3, m * 3:m * 3 + 3] @ q[b, s, i, m * 3:m * 3 + 3])
        assert abs((2.0 ** (z / np.log(2.0) - lse[b, i, m, s])).sum() - 1.0) < 1e-12


def test_diff_backward_matches_differences():
    x = list(diff_inputs(5))
    dout, lens = x[4], x[5]

    def loss(q, k, v, lam):
        return (O.diff_attention(q, k, v, lam, lens, 0.6)[0] * dout).sum()

    grads = O.diff_attention_bwd(*x[:4], dout, lens, 0.6)
    step = 1e-6
    for which, at in [(0, (0, 1, 4, 2)), (0, (1, 3, 0, 5)), (1, (0, 6, 1, 3)), (1, (1, 2, 0, 1)),
                      (2, (0, 0, 0, 4)), (2, (1, 1, 1, 0)), (1, (1, 3, 0, 0)), (3, (0,)), (3, (5,))]:
        hi, lo = x[:4], x[:4]
        e = np.zeros_like(hi[which])
        e[at] = step
        hi[which], lo[which] = hi[which] + e, lo[which] - e
        assert abs((loss(*hi) - loss(*lo)) / (2 * step) - grads[which][at]) < 1e-7
