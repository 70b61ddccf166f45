"""Differential attention of few rows, as a serving step asks for it: one to nine packed rows a
key head, lengths around a tile's 16 states and a run's 512, ragged batches, views; against
the 64-bit oracle with test_gpu_diff's tolerances.
"""
import pytest
import torch

from test_gpu_diff import (DEV, TYPES, check_forward, fill_behind, inputs, lengths,  # noqa: F401
                           nabla)

pytestmark = pytest.mark.gpu

CASES = [
    # B, Sq, Sk, h, hk, D, lens (None: all), packed
    (1, 1, 1, 2, 1, 64, None, False),
    (2, 2, 15, 2, 2, 128, None, False),
    (1, 1, 16, 3, 1, 64, None, True),
    (3, 1, 17, 8, 2, 128, [17, 0, 16], True),
    (2, 1, 63, 5, 1, 64, [1, 63], False),
    (1, 3, 64, 4, 2, 128, None, "heads"),
    (1, 7, 65, 1, 1, 128, None, False),
    (4, 1, 511, 16, 2, 64, [511, 510, 497, 2], True),
    (2, 4, 513, 2, 1, 128, None, False),
    (1, 8, 1500, 3, 3, 128, None, False),
    (16, 1, 1200, 24, 8, 128, [75 * i for i in range(1, 17)], False),
    (160, 1, 300, 2, 1, 64, [i * 7 % 301 for i in range(160)], False),
    (1, 1, 20000, 8, 1, 128, None, False),
    (2, 3, 700, 3, 1, 128, [700, 3], False),             # nine rows
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,Sq,Sk,h,hk,D,lens,packed", CASES)
def test_forward(nabla, B, Sq, Sk, h, hk, D, lens, packed, dtype):  # noqa: F811
    q, k, v, lam, _ = inputs(B, Sq, Sk, h, hk, D, dtype, seed=Sk, packed=packed, one=Sq == 1)
    kv_len = None if lens is None else lengths(lens)
    fill_behind(k, v, lens)
    need = nabla.nabla_diff_attn_fwd_workspace_bytes(TYPES[dtype], B, Sq, Sk, h, hk, D)
    ws = torch.full((max(need, 1),), 0xff, dtype=torch.uint8, device=DEV)
    o, o2, lse = nabla.nabla_diff_attn_fwd_lse(q, k, v, lam, kv_len, workspace=ws)
    assert nabla.nabla_get_last_device_status() == 0
    check_forward(o, o2, lse, q, k, v, lam, [Sk] * B if lens is None else lens, (2.0 / D) ** 0.5)
    assert torch.equal(nabla.nabla_diff_attn_fwd(q, k, v, lam, kv_len), o)


@pytest.mark.parametrize("scale", [0.0, -0.7, 3.0])
def test_scores_that_rise(nabla, scale):  # noqa: F811
    """Every tile's scores pass the last one's, so that the bias is raised again and again."""
    q, k, v, lam, _ = inputs(1, 2, 600, 6, 2, 128, "bf16", seed=5)
    k *= torch.linspace(0.1, 4.0, 600, device=DEV).to(k.dtype)[None, :, None, None]
    o, o2, lse = nabla.nabla_diff_attn_fwd_lse(q, k, v, lam, scale=scale)
    assert nabla.nabla_get_last_device_status() == 0
    check_forward(o, o2, lse, q, k, v, lam, [600], scale)


def test_not_a_number_stays_in_its_rows(nabla):  # noqa: F811
    """A NaN in one row of q reaches that head's output and no other's."""
    q, k, v, lam, _ = inputs(1, 1, 100, 4, 1, 64, "bf16", seed=6)
    clean = nabla.nabla_diff_attn_fwd(q, k, v, lam)
    q[0, 0, 2, 5] = float("nan")
    o = nabla.nabla_diff_attn_fwd(q, k, v, lam)
    assert torch.isnan(o[0, 0, 2]).all()
    for i in (0, 1, 3):
        assert torch.equal(o[0, 0, i], clean[0, 0, i])
