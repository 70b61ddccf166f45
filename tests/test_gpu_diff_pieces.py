"""Differential attention whose last units go to the SMs in pieces: few units of many states,
ragged batches, units that stay whole before them, few rows in a unit; against the 64-bit
oracle with test_gpu_diff's tolerances, the scratch filled with NaN before the call.
"""
import pytest
import torch

from test_gpu_diff import DEV, TYPES, check_backward, check_forward, inputs, nabla  # noqa: F401

pytestmark = pytest.mark.gpu

CASES = [
    # B, Sq, Sk, h, hk, D, lens (None: all)
    (1, 100, 2500, 2, 2, 128, None),                    # 76 parts a unit
    (1, 7, 4000, 6, 2, 64, None),                       # 21 rows a unit
    (2, 1, 3601, 33, 1, 128, [3601, 2]),                # 33 rows; 57 tiles
    (3, 130, 3700, 4, 2, 128, [3700, 0, 65]),
    (5, 40, 3600, 8, 2, 64, [1, 3600, 64, 63, 1000]),
    (2, 64, 3584, 1, 1, 64, [0, 0]),
    (4, 200, 5000, 3, 3, 128, [5000, 4999, 4993, 1]),
    (1, 3600, 2100, 11, 11, 64, None),                  # 319 units: one round of whole ones
    (160, 9, 3584, 2, 2, 128, [3584 if i % 40 == 7 else i % 5 for i in range(160)]),
]


@pytest.mark.parametrize("B,Sq,Sk,h,hk,D,lens", CASES)
def test_forward(nabla, B, Sq, Sk, h, hk, D, lens):  # noqa: F811
    q, k, v, lam, _ = inputs(B, Sq, Sk, h, hk, D, "bf16")
    kv_len = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    need = nabla.nabla_diff_attn_fwd_workspace_bytes(TYPES["bf16"], B, Sq, Sk, h, hk, D)
    assert need > 1 << 20  # there are parts
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    o, o2, lse = nabla.nabla_diff_attn_fwd_lse(q, k, v, lam, kv_len, workspace=ws)
    assert nabla.nabla_get_last_device_status() == 0
    check_forward(o, o2, lse, q, k, v, lam, [Sk] * B if lens is None else lens, (2.0 / D) ** 0.5)
    again = nabla.nabla_diff_attn_fwd(q, k, v, lam, kv_len)
    assert torch.equal(again, o)


@pytest.mark.parametrize("B,Sq,Sk,h,hk,D,lens", [
    (1, 40, 900, 2, 2, 64, None),
    (1, 200, 1000, 2, 1, 128, None),
    (3, 70, 700, 4, 2, 64, [700, 0, 65]),
    (2, 5, 2000, 24, 8, 128, [1, 2000]),
])
def test_backward_in_runs_of_states(nabla, B, Sq, Sk, h, hk, D, lens):  # noqa: F811
    """fp32: few units of rows, their states in runs; the scratch holds NaN."""
    q, k, v, lam, dout = inputs(B, Sq, Sk, h, hk, D, "f32")
    kv_len = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    o, o2, lse = nabla.nabla_diff_attn_fwd_lse(q, k, v, lam, kv_len)
    need = nabla.nabla_diff_attn_bwd_workspace_bytes(TYPES["f32"], B, Sq, Sk, h, hk, D)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    got = nabla.nabla_diff_attn_bwd(q, k, v, lam, o, o2, lse, dout, kv_len, workspace=ws)
    assert nabla.nabla_get_last_device_status() == 0
    check_backward(got, q, k, v, lam, o, o2, dout, [Sk] * B if lens is None else lens,
                   (2.0 / D) ** 0.5)
