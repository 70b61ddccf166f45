"""Cross attention on the GPU vs the fp64 oracle, through the binding.

Tolerances, from the arithmetic, per element, with A = sum_u p_u |v_u| (p the row's
softmax weights) and Z the largest |scale log2(e) <q, k_u>| of the row:
  scores    fp32 products and sums over D <= 128 (bf16 inputs multiply exactly; the
            tensor cores may truncate each of the D/16 accumulator steps by 2^-23):
            their base-2 error is at most e_z = 2^-17 scale log2(e) sum_d |q_d k_d| (more
            than 128 roundings of 2^-24); p is then off by at most 2 e_z ln 2 relative,
            plus 2^-20 for ex2 and the sum;
  bf16      P is rounded before the second product (half a step, 2^-8) and so is o:
            |err| <= (2^-8 + 2 e_z + 2^-18) A + 2^-8 |o|;
  f32       |err| <= (2 e_z + 2^-17) A + 2^-24 |o|.
  lse       the largest score error plus 2^-18 (fp32 sum, log2) plus 2^-23 |lse|.
"""
import math

import numpy as np
import pytest
import torch

from oracle import nabla_oracle as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BAD_INDEX = 5


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


def inputs(B, Sq, Sk, h, hk, D, dtype, seed=0, packed=False, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[dtype]

    def draw(*shape):
        return (torch.randn(*shape, generator=g) * spread).to(dt).to(DEV)

    if packed == "heads":  # heads before tokens
        return [draw(*s).transpose(1, 2) for s in
                ((B, h, Sq, D), (B, hk, Sk, D), (B, hk, Sk, D))]
    if packed:  # q between other columns, k and v in one projection
        q = draw(B, Sq, (h + 1) * D)[..., D:].unflatten(-1, (h, D))
        kv = draw(B, Sk, 2, hk, D)
        return q, kv[:, :, 0], kv[:, :, 1]
    return draw(B, Sq, h, D), draw(B, Sk, hk, D), draw(B, Sk, hk, D)


def bounds(q, k, v, lens, scale):
    """The tolerance's A, e_z (largest of the row) per row, in float64."""
    B, Sq, h, D = q.shape
    G = h // k.shape[2]
    A, ez = np.zeros(q.shape), np.zeros((B, h, Sq))
    for b in range(B):
        n = int(lens[b])
        for i in range(h if n else 0):
            Q, K, V = q[b, :, i], k[b, :n, i // G], v[b, :n, i // G]
            z = scale * (Q @ K.T)
            p = np.exp(z - z.max(1, keepdims=True))
            A[b, :, i] = (p @ np.abs(V)) / p.sum(1, keepdims=True)
            ez[b, i] = 2.0 ** -17 * abs(scale) * 1.4427 * (np.abs(Q) @ np.abs(K).T).max(1)
    return A, ez


def check(o, lse, q, k, v, lens, scale):
    Q, K, V = f64(q), f64(k), f64(v)
    ref, rl = O.cross_attention(Q, K, V, lens, scale)
    A, ez = bounds(Q, K, V, lens, scale)
    e = 2 * ez.transpose(0, 2, 1)[..., None]
    if o.dtype == torch.bfloat16:
        tol = (2.0 ** -8 + e + 2.0 ** -18) * A + 2.0 ** -8 * np.abs(ref)
    else:
        tol = (e + 2.0 ** -17) * A + 2.0 ** -24 * np.abs(ref)
    err = np.abs(f64(o) - ref)
    assert np.all(err <= tol + 1e-37), (err.max(), (err - tol).max())
    if lse is not None:
        got = f64(lse)
        dead = np.isneginf(rl)
        assert np.array_equal(dead, np.isneginf(got))
        live = ~dead
        assert np.all(np.abs(got[live] - rl[live]) <=
                      (ez + 2.0 ** -18)[live] + 2.0 ** -23 * np.abs(rl[live]))


def lengths(lens):
    return torch.tensor(lens, dtype=torch.int32, device=DEV)


CASES = [  # B, Sq, Sk, h, hk, D, lens, packed
    (1, 1, 1, 1, 1, 64, None, False),
    (1, 1, 1, 4, 1, 128, None, False),
    (2, 300, 77, 3, 3, 128, [77, 16], False),      # text of 77 states
    (3, 129, 128, 2, 2, 64, [128, 0, 1], True),    # a full tile, an empty batch, one state
    (2, 40, 300, 6, 2, 128, [257, 128], True),     # three heads a group (21 tokens a subtile)
    (2, 23, 130, 10, 2, 64, [129, 127], False),    # five heads a group
    (4, 1, 2000, 24, 8, 128, [2000, 1999, 130, 0], False),   # a serving step, runs of states
    (1, 1, 8192, 2, 2, 64, None, False),           # two rows in all
    (1, 5, 700, 64, 1, 64, [641], False),          # 64 heads on one key head
    (2, 1, 900, 14, 2, 128, [900, 385], True),     # seven heads a group, runs
    (1, 1537, 513, 2, 1, 128, None, True),
    (2, 333, 150, 4, 2, 128, [150, 90], "heads"),
    (3, 5, 300, 6, 2, 64, [300, 0, 65], True),      # fifteen rows a key head
    (2, 16, 129, 2, 2, 128, [129, 1], "heads"),     # sixteen
    (1, 17, 129, 2, 2, 64, None, False),            # one more
    (160, 2, 70, 2, 1, 64, None, False),            # four rows a key head, more than fill the GPU
    (3, 650, 1200, 9, 9, 64, [1200, 1100, 64], False),  # many tiles in one run
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,Sq,Sk,h,hk,D,lens,packed", CASES)
def test_forward(nabla, B, Sq, Sk, h, hk, D, lens, packed, dtype):
    q, k, v = inputs(B, Sq, Sk, h, hk, D, dtype, seed=Sk, packed=packed, spread=1.3)
    n = None if lens is None else lengths(lens)
    if lens is not None:  # what lies behind the lengths must not matter
        for b, m in enumerate(lens):
            k[b, m:] = float("nan")
            v[b, m:] = float("inf") if b % 2 else float("nan")
    o, lse = nabla.nabla_cross_attn_fwd_lse(q, k, v, kv_len=n)
    assert nabla.nabla_get_last_device_status() == 0
    check(o, lse, q, k, v, lens or [Sk] * B, 1 / math.sqrt(D))
    assert torch.equal(nabla.nabla_cross_attn_fwd(q, k, v, kv_len=n), o)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.5])
def test_scales(nabla, dtype, scale):
    q, k, v = inputs(2, 70, 200, 2, 2, 64, dtype, seed=7)
    o, lse = nabla.nabla_cross_attn_fwd_lse(q, k, v, kv_len=lengths([200, 73]), scale=scale)
    check(o, lse, q, k, v, [200, 73], scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_that_jump(nabla, dtype):
    """Scores that rise by hundreds of base-2 units from tile to tile, in rows apart:
    the running bias has to be raised and O rescaled."""
    q, k, v = inputs(1, 200, 640, 2, 2, 64, dtype, seed=8, spread=0.5)
    k[0, 130:140, 0] *= 12.0
    k[0, 300, 0] *= 60.0
    k[0, 520:600, 1] *= 40.0
    q[0, ::3] *= 8.0
    q[0, 5] = 0.0
    o, lse = nabla.nabla_cross_attn_fwd_lse(q, k, v)
    assert nabla.nabla_get_last_device_status() == 0
    check(o, lse, q, k, v, [640], 1 / 8)


def test_bad_lengths_are_clamped_and_reported(nabla):
    q, k, v = inputs(3, 20, 50, 2, 2, 64, "bf16", seed=9)
    o = nabla.nabla_cross_attn_fwd(q, k, v, kv_len=lengths([51, -1, 50]))
    assert nabla.nabla_get_last_device_status() == BAD_INDEX
    assert torch.equal(o, nabla.nabla_cross_attn_fwd(q, k, v, kv_len=lengths([50, 0, 50])))
    assert nabla.nabla_get_last_device_status() == 0


@pytest.mark.parametrize("Sq,Sk", [(1, 3000), (600, 300)])
def test_streams_and_graphs(nabla, Sq, Sk):
    """Same bits on another stream and from two graphs with a workspace each."""
    B, h, hk, D = 2, 6, 2, 128
    q, k, v = inputs(B, Sq, Sk, h, hk, D, "bf16", seed=10)
    n = lengths([Sk, Sk // 2 + 1])
    want = nabla.nabla_cross_attn_fwd(q, k, v, kv_len=n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = nabla.nabla_cross_attn_fwd(q, k, v, kv_len=n, stream=side)
    side.synchronize()
    assert torch.equal(want, other)
    need = nabla.nabla_cross_attn_fwd_workspace_bytes(q.dtype, B, Sq, Sk, h, hk, D)
    graphs, outs = [], []
    for _ in range(2):
        o = torch.zeros_like(want)
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=DEV)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            nabla.nabla_cross_attn_fwd(q, k, v, kv_len=n, o=o, workspace=ws)
        graphs.append((g, ws))
        outs.append(o)
    with torch.cuda.stream(side):
        graphs[0][0].replay()
    graphs[1][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    n.copy_(lengths([1, 3 * Sk // 4]))  # a replay reads the lengths anew
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], nabla.nabla_cross_attn_fwd(q, k, v, kv_len=n))
