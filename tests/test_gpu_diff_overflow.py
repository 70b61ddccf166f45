"""Differential attention where the first states' scores are too far below zero for fp32: they
weigh nothing, and the rows are those of the other states; a map whose scores all are gives 0
and a log-sum-exp of -infinity, as one without states does.  Every form of the kernels.

A query and a key of 2^70 and -2^70 in one column make a score of -2^140, -infinity in fp32;
that column of the other states is 0, so it adds nothing to theirs.  Tolerances: those of
test_gpu_diff, of the states that count."""
import math

import pytest
import torch

from test_gpu_diff import check_backward, check_forward, inputs, lengths, nabla  # noqa: F401

pytestmark = pytest.mark.gpu

FAR = 2.0 ** 70


def overflow(q, k, maps, first):
    """Scores of -infinity in `maps` for the first states."""
    d = q.shape[-1] // 2
    for m in maps:
        q[..., m * d] = FAR
        k[..., m * d] = 0.0
        k[:, :first, :, m * d] = -FAR


SHAPES = [  # B, Sq, Sk, h, hk, D, lens, states that weigh nothing
    (1, 200, 200, 2, 2, 64, None, 64),            # a step of the tensor cores' form
    (2, 130, 300, 4, 2, 128, [300, 201], 130),    # two and a part of the third
    (3, 40, 5000, 4, 2, 64, [5000, 1800, 4321], 1300),  # whole parts of the cut units
    (2, 9800, 1030, 1, 1, 128, None, 70),
    (2, 1, 1500, 6, 2, 128, [1500, 700], 600),    # few rows, whole runs of them
    (1, 1, 90, 1, 1, 64, None, 33),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,Sq,Sk,h,hk,D,lens,first", SHAPES)
def test_first_states_weigh_nothing(nabla, B, Sq, Sk, h, hk, D, lens, first, dtype):  # noqa: F811
    q, k, v, lam, dout = inputs(B, Sq, Sk, h, hk, D, dtype, seed=Sk)
    overflow(q, k, (0, 1), first)
    n = None if lens is None else lengths(lens)
    o, o2, lse = nabla.nabla_diff_attn_fwd_lse(q, k, v, lam, kv_len=n)
    rest = [m - first for m in (lens or [Sk] * B)]
    scale = math.sqrt(2 / D)
    check_forward(o, o2, lse, q, k[:, first:], v[:, first:], lam, rest, scale)
    dq, dk, dv, dlam = nabla.nabla_diff_attn_bwd(q, k, v, lam, o, o2, lse, dout, kv_len=n)
    assert (dk[:, :first] == 0).all() and (dv[:, :first] == 0).all()
    check_backward((dq, dk[:, first:], dv[:, first:], dlam), q, k[:, first:], v[:, first:], lam,
                   o, o2, dout, rest, scale)
    assert nabla.nabla_get_last_device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("B,Sq,Sk,h,hk,D,lens,first", SHAPES[:1] + SHAPES[2:3] + SHAPES[4:])
def test_a_map_of_nothing(nabla, B, Sq, Sk, h, hk, D, lens, first, which, dtype):  # noqa: F811
    q, k, v, lam, dout = inputs(B, Sq, Sk, h, hk, D, dtype, seed=Sk)
    overflow(q, k, (which,), Sk)
    n = None if lens is None else lengths(lens)
    o, o2, lse = nabla.nabla_diff_attn_fwd_lse(q, k, v, lam, kv_len=n)
    assert torch.isneginf(lse[:, :, which]).all() and torch.isfinite(lse[:, :, 1 - which]).all()
    lens, scale = lens or [Sk] * B, math.sqrt(2 / D)
    if which:  # o is the first map's rows alone
        assert (o2 == 0).all()
        check_forward(o, None, None, *only(q, k, 0), v, 0.0 * lam, lens, scale)
    else:  # o = -lam o2
        check_forward(o2, None, None, *only(q, k, 1), v, 0.0 * lam, lens, scale)
        got, ref = o.double(), -lam.double()[:, None] * o2.double()
        # from the same sums: each rounded once, and three fp32 products
        room = torch.finfo(o.dtype).eps + 2.0 ** -22
        assert bool(((got - ref).abs() <= room * ref.abs()).all())
    grads = nabla.nabla_diff_attn_bwd(q, k, v, lam, o, o2, lse, dout, kv_len=n)
    d = D // 2
    none = slice(which * d, which * d + d)
    assert all(bool(torch.isfinite(t).all()) for t in grads)
    assert (grads[0][..., none] == 0).all() and (grads[1][..., none] == 0).all()
    assert not which or (grads[3] == 0).all()


def only(q, k, m):
    """Both maps as the one of them."""
    d = q.shape[-1] // 2
    at = slice(m * d, m * d + d)
    return torch.cat([q[..., at]] * 2, -1), torch.cat([k[..., at]] * 2, -1)
