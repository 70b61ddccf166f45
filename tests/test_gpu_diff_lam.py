"""The gradient of differential attention's lam in fp32, a sum over all rows whose terms cancel,
against 64 bits: over many heads and inputs it is off by no more than elementary fp32 operations
with a 64-bit sum over the rows are, measured by the terms' norm (an error of a row's sum shows
in the gradient whole, however much the rows cancel)."""
import math

import numpy as np
import pytest
import torch

from oracle import nabla_oracle as O
from test_gpu_diff import f64, inputs, lengths, nabla  # noqa: F401

pytestmark = pytest.mark.gpu


def maps(q, k, which, scale):
    d, G = q.shape[-1] // 2, q.shape[2] // k.shape[2]
    at = slice(which * d, which * d + d)
    z = q[..., at].transpose(1, 2) @ k[..., at].transpose(1, 2).repeat_interleave(
        G, 1).transpose(-1, -2)
    return torch.softmax(z * scale, -1)


def rows(q, k, v, dout, lens, scale):
    """[B, h, Sq]: the rows' sums of P_2 <dout, v>, in the type of the inputs."""
    out = torch.zeros(q.shape[0], q.shape[2], q.shape[1], dtype=q.dtype, device=q.device)
    for b, n in enumerate(lens):
        one = slice(b, b + 1)
        p = maps(q[one], k[one, :n], 1, scale)
        y = dout[one].transpose(1, 2) @ v[one, :n].transpose(1, 2).repeat_interleave(
            q.shape[2] // k.shape[2], 1).transpose(-1, -2)
        out[one] = (p * y).sum(-1)
    return out


@pytest.mark.parametrize("B,Sq,Sk,h,hk,D,lens", [(2, 300, 77, 6, 2, 128, [77, 40]),
                                                 (1, 400, 500, 8, 8, 64, [500]),
                                                 (3, 2, 900, 4, 4, 128, [900, 70, 333])])
def test_error_of_the_gradient(nabla, B, Sq, Sk, h, hk, D, lens):  # noqa: F811
    assert not torch.backends.cuda.matmul.allow_tf32
    scale, mine, plain = math.sqrt(2 / D), [], []
    for seed in range(16):
        q, k, v, lam, dout = inputs(B, Sq, Sk, h, hk, D, "f32", seed=seed)
        n = lengths(lens)
        o, o2, lse = nabla.nabla_diff_attn_fwd_lse(q, k, v, lam, kv_len=n)
        got = nabla.nabla_diff_attn_bwd(q, k, v, lam, o, o2, lse, dout, kv_len=n)[3]
        t = rows(*(x.double() for x in (q, k, v, dout)), lens, scale)
        want, size = -t.sum((0, 2)), t.square().sum((0, 2)).sqrt()
        elementary = -rows(q, k, v, dout, lens, scale).double().sum((0, 2)).float()
        mine.append((got.double() - want) / size)
        plain.append((elementary.double() - want) / size)
        if seed == 0:
            K, V = f64(k), f64(v)
            ref = O.diff_attention_bwd(f64(q), K, V, f64(lam), f64(dout), lens, scale)[3]
            np.testing.assert_allclose(want.cpu().numpy(), ref, rtol=1e-9, atol=1e-9)
    rms = [float(torch.stack(x).square().mean().sqrt()) for x in (mine, plain)]
    assert rms[0] <= rms[1], rms
    # one weight for all heads is their sum
    one = torch.full((1,), 0.5, device=q.device)
    o, o2, lse = nabla.nabla_diff_attn_fwd_lse(q, k, v, one, kv_len=n)
    got = nabla.nabla_diff_attn_bwd(q, k, v, one, o, o2, lse, dout, kv_len=n)[3]
    assert abs(float(got.double() - want.sum())) <= 8 * rms[1] * float(size.square().sum().sqrt())
