"""Pins of the oracle's operators around the self-attention (CPU, no GPU): the
per-head norm with rotation and the cross attention.  None reuses the oracle's
formulas: complex multiplication, hand-worked rows, torch's own softmax attention
in 64 bits, autograd and central differences.
"""
import numpy as np
import pytest
import torch

from oracle import nabla_oracle as O


def angles(rng, B, S, n):
    a = rng.uniform(-40.0, 40.0, (B, S, n))
    return a, np.cos(a), np.sin(a)


def test_norm_of_a_hand_worked_row():
    x = np.array([3.0, 4.0, 0.0, 0.0]).reshape(1, 1, 1, 4)  # mean square 6.25
    none = np.zeros((1, 1, 0))
    z = O.qk_norm_rope(x, np.array([1.0, 2.0, 5.0, 7.0]), none, none, True, 0.0)
    assert np.allclose(z.ravel(), [1.2, 3.2, 0.0, 0.0], atol=1e-15)
    z = O.qk_norm_rope(x, None, none, none, True, 2.75)     # sqrt(6.25 + 2.75) = 3
    assert np.allclose(z.ravel(), [1.0, 4.0 / 3.0, 0.0, 0.0], atol=1e-15)


def test_quarter_turns():
    """cos = 0, sin = 1: (a, b) -> (-b, a) in the columns of each convention."""
    y = np.arange(1.0, 9.0).reshape(1, 1, 1, 8)
    c, s = np.zeros((1, 1, 2)), np.ones((1, 1, 2))
    assert O.rotate(y, c, s, True).ravel().tolist() == [-2, 1, -4, 3, 5, 6, 7, 8]
    assert O.rotate(y, c, s, False).ravel().tolist() == [-3, -4, 1, 2, 5, 6, 7, 8]


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    y = rng.standard_normal((2, 5, 3, 12))
    a, c, s = angles(rng, 2, 5, 4)
    got = O.rotate(y, c, s, interleaved)
    z = (y[..., 0:8:2] + 1j * y[..., 1:8:2]) if interleaved else (y[..., :4] + 1j * y[..., 4:8])
    z = z * np.exp(1j * a)[:, :, None]
    re, im = (got[..., 0:8:2], got[..., 1:8:2]) if interleaved else (got[..., :4], got[..., 4:8])
    assert np.allclose(re, z.real, atol=1e-13) and np.allclose(im, z.imag, atol=1e-13)
    assert np.array_equal(got[..., 8:], y[..., 8:])


@pytest.mark.parametrize("interleaved", [True, False])
def test_norm_backward_matches_differences(interleaved):
    rng = np.random.default_rng(2)
    x, dz = rng.standard_normal((2, 3, 2, 8)), rng.standard_normal((2, 3, 2, 8))
    w = rng.uniform(0.5, 1.5, 8)
    _, c, s = angles(rng, 2, 3, 3)

    def loss(x, w):
        return (O.qk_norm_rope(x, w, c, s, interleaved, 1e-3) * dz).sum()

    dx, dw = O.qk_norm_rope_bwd(x, w, dz, c, s, interleaved, 1e-3)
    step = 1e-6
    for at in [(0, 0, 0, 0), (1, 2, 1, 7), (0, 1, 1, 3), (1, 0, 0, 5)]:
        e = np.zeros_like(x)
        e[at] = step
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * step) - dx[at]) < 1e-8
    for j in range(8):
        e = np.zeros(8)
        e[j] = step
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * step) - dw[j]) < 1e-7


def cross_inputs(seed, B=3, Sq=4, Sk=7, h=6, hk=2, D=5, lens=(7, 3, 0)):
    rng = np.random.default_rng(seed)
    q, dout = rng.standard_normal((2, B, Sq, h, D))
    k, v = rng.standard_normal((2, B, Sk, hk, D))
    return q, k, v, dout, np.array(lens)


def torch_cross(q, k, v, lens, scale):
    """The library's own attention, one batch at a time, key heads repeated."""
    outs = []
    for b, n in enumerate(lens):
        if n == 0:
            outs.append(torch.zeros_like(q[b]))
            continue
        rep = q.shape[2] // k.shape[2]
        kk, vv = (t[b, :n].repeat_interleave(rep, 1).transpose(0, 1) for t in (k, v))
        outs.append(torch.nn.functional.scaled_dot_product_attention(
            q[b].transpose(0, 1), kk, vv, scale=scale).transpose(0, 1))
    return torch.stack(outs)


def test_cross_attention_matches_torch_and_its_gradients():
    q, k, v, dout, lens = cross_inputs(3)
    t = [torch.from_numpy(x).requires_grad_() for x in (q, k, v)]
    ref = torch_cross(*t, lens, 0.7)
    o, lse = O.cross_attention(q, k, v, lens, 0.7)
    assert np.allclose(o, ref.detach().numpy(), atol=1e-13)
    assert np.all(o[2] == 0) and np.all(np.isneginf(lse[2]))
    ref.backward(torch.from_numpy(dout))
    for got, x in zip(O.cross_attention_bwd(q, k, v, dout, lens, 0.7), t):
        assert np.allclose(got, x.grad.numpy(), atol=1e-12)


def test_cross_lse_rebuilds_the_weights():
    q, k, v, _, lens = cross_inputs(4)
    _, lse = O.cross_attention(q, k, v, lens, 0.5)
    for b, i, s in [(0, 0, 0), (0, 5, 3), (1, 2, 1)]:
        z = 0.5 * (k[b, :lens[b], i // 3] @ q[b, s, i])
        assert abs((2.0 ** (z / np.log(2.0) - lse[b, i, s])).sum() - 1.0) < 1e-12


def test_cross_backward_matches_differences():
    q, k, v, dout, lens = cross_inputs(5)

    def loss(q, k, v):
        return (O.cross_attention(q, k, v, lens, 0.6)[0] * dout).sum()

    grads = O.cross_attention_bwd(q, k, v, dout, lens, 0.6)
    step = 1e-6
    for which, at in [(0, (0, 1, 4, 2)), (0, (1, 3, 0, 0)), (1, (0, 6, 1, 3)), (1, (1, 2, 0, 1)),
                      (2, (0, 0, 0, 4)), (2, (1, 1, 1, 0)), (1, (1, 3, 0, 0)), (2, (2, 0, 0, 0))]:
        hi, lo = [q, k, v], [q, k, v]
        e = np.zeros_like(hi[which])
        e[at] = step
        hi[which], lo[which] = hi[which] + e, lo[which] - e
        assert abs((loss(*hi) - loss(*lo)) / (2 * step) - grads[which][at]) < 1e-8


def test_cross_backward_invariants():
    """dz of a row sums to 0, so dk sums to 0 over the states; the weights of a row sum
    to 1, so dv sums to dout over the rows of the heads that share the key head."""
    q, k, v, dout, lens = cross_inputs(6)
    _, dk, dv = O.cross_attention_bwd(q, k, v, dout, lens, 0.6)
    assert np.abs(dk.sum(1)).max() < 1e-12
    want = dout.sum(1).reshape(3, 2, 3, 5).sum(2)
    want[2] = 0
    assert np.allclose(dv.sum(1), want, atol=1e-12)
