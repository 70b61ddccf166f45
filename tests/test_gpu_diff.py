"""Differential attention on the GPU vs the fp64 oracle, through the binding, forward and
backward (the forward's o, o2 and lse, as stored, go to both sides of the backward).

Tolerances, from the arithmetic, per element and map m, half = half a step of the stored type
(2^-8 for bf16, 2^-24 for fp32), with p_m the row's softmax weights and A_m = sum_u p_m |v_u|:
  scores    fp32 products and sums over D / 2 <= 64 (bf16 inputs multiply exactly; the tensor
            cores may truncate each accumulator step by 2^-23): their base-2 error is at
            most e_m = 2^-17 scale log2(e) sum_d |q_d k_d|; p is off by at most 2 e_m ln 2
            relative, plus 2^-20 for ex2 and the sum;
  o2        bf16, P rounded before the product: (half + 2 e_2 + 2^-18) A_2 + half |o2|;
            f32: (2 e_2 + 2^-17) A_2 + half |o2|;
  o         the same of the first map plus |lam| times that of the second, without their own
            rounding (the difference is formed in fp32, within 2^-18 A), and half |o|;
  lse       the largest score error plus 2^-18 plus 2^-23 |lse|.
  P_m       rebuilt: relative E_m = 3 e_m + 2^-17 + 2^-22 |lse_m| (the score's error, the
            lse's, ex2's);
  Y, delta  e_d = 2^-17 (sum_d |dout_d v_d| + sum_d |dout_d| (|o_d| + 2 |lam o2_d|));
  dz_m      F_m = (half + E_m + sums) |dz_m| + w_m P_m e_d,  w = 1, |lam|;
  dq, dk    scale sum F_m |k_m|, scale sum F_m |q_m|, and half of the result;
  dv        sum_s sum_m (half + E_m + sums) w_m P_m |dout|, and half of the result;
  dlam      sum P_2 ((E_2 + sums) |Y| + e_d) over its rows: no rounding to the stored type;
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
BAD_INDEX = 5
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


def inputs(B, Sq, Sk, h, hk, D, dtype, seed=0, packed=False, spread=1.2, one=False):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[dtype]

    def draw(*shape, s=spread):
        return (torch.randn(*shape, generator=g) * s).to(dt).to(DEV)

    lam = (0.6 + 0.4 * torch.randn(1 if one else h, generator=g)).to(DEV)
    if packed == "heads":  # everything heads before tokens
        q, k, v, do = [draw(*s).transpose(1, 2) for s in
                       ((B, h, Sq, D), (B, hk, Sk, D), (B, hk, Sk, D), (B, h, Sq, D))]
        return q, k, v, lam, do * 0.5
    if packed:  # q's maps as pairs of heads between other columns, k and v in one projection
        q = draw(B, Sq, (2 * h + 2) * (D // 2))[..., D:].unflatten(-1, (h, D))
        kv = draw(B, Sk, 2, hk, D)
        k, v = kv[:, :, 0], kv[:, :, 1]
    else:
        q, k, v = draw(B, Sq, h, D), draw(B, Sk, hk, D), draw(B, Sk, hk, D)
    return q, k, v, lam, draw(B, Sq, h, D, s=0.5)


def maps(Q, K, scale):
    """Per map: columns, weights P, the score's error bound, |lse|."""
    d = Q.shape[1] // 2
    for at in (slice(0, d), slice(d, 2 * d)):
        z = scale * (Q[:, at] @ K[:, at].T)
        m = z.max(1, keepdims=True)
        p = np.exp(z - m)
        t = p.sum(1, keepdims=True)
        e = 2.0 ** -17 * abs(scale) * 1.4427 * (np.abs(Q[:, at]) @ np.abs(K[:, at]).T)
        yield at, p / t, e, np.abs((m + np.log(t)) / math.log(2.0))


def check_forward(o, o2, lse, q, k, v, lam, lens, scale):
    Q, K, V = f64(q), f64(k), f64(v)
    B, Sq, h, D = Q.shape
    G, L = h // K.shape[2], np.broadcast_to(f64(lam), (h,))
    half = torch.finfo(o.dtype).eps / 2
    for b, n in enumerate(lens):
        K[b, n:] = V[b, n:] = 0.0
    ref, ref2, rl = O.diff_attention(Q, K, V, f64(lam), lens, scale)
    tol, tol2, ez = np.zeros(Q.shape), np.zeros(Q.shape), np.zeros((B, h, 2, Sq))
    for b in range(B):
        n = int(lens[b])
        for i in range(h if n else 0):
            for m, (_, P, e, _) in enumerate(maps(Q[b, :, i], K[b, :n, i // G], scale)):
                A = P @ np.abs(V[b, :n, i // G])
                ez[b, i, m] = e.max(1)
                t = (2 * ez[b, i, m][:, None] + (half + 2.0 ** -18 if half > 1e-3
                                                 else 2.0 ** -17)) * A
                tol[b, :, i] += t * (abs(L[i]) if m else 1.0) * (1 + 2.0 ** -18)
                tol2[b, :, i] = t
    for got, r, t in ((o, ref, tol), (o2, ref2, tol2)):
        if got is not None:
            err = np.abs(f64(got) - r)
            assert np.all(err <= t + half * np.abs(r) + 1e-37), (err - t - half * np.abs(r)).max()
    if lse is not None:
        got, dead = f64(lse), np.isneginf(rl)
        assert np.array_equal(dead, np.isneginf(got))
        live = ~dead
        assert np.all(np.abs(got[live] - rl[live]) <=
                      (ez + 2.0 ** -18)[live] + 2.0 ** -23 * np.abs(rl[live]))


def check_backward(got, q, k, v, lam, o, o2, dout, lens, scale):
    half = torch.finfo(q.dtype).eps / 2
    Q, K, V, Oo, O2, g = (f64(t) for t in (q, k, v, o, o2, dout))
    B, Sq, h, D = Q.shape
    G, L = h // K.shape[2], np.broadcast_to(f64(lam), (h,))
    for b, n in enumerate(lens):  # what lies behind the lengths is not part of the problem
        K[b, n:] = V[b, n:] = 0.0
    ref = O.diff_attention_bwd(Q, K, V, f64(lam), g, lens, scale, o=Oo, o2=O2)
    tq, tk, tv, tl = np.zeros(Q.shape), np.zeros(K.shape), np.zeros(K.shape), np.zeros(h)
    for b in range(B):
        n = int(lens[b])
        for i in range(h if n else 0):
            j, gi = i // G, g[b, :, i]
            Ki, Vi, a = K[b, :n, j], V[b, :n, j], np.abs(gi)
            second = O2[b, :, i]
            first = Oo[b, :, i] + L[i] * second
            Y = gi @ Vi.T
            ed = 2.0 ** -17 * (a @ np.abs(Vi).T + (a * (np.abs(Oo[b, :, i]) + 2 * np.abs(
                L[i] * second) + np.abs(second))).sum(1, keepdims=True))
            for m, (at, P, e, l) in enumerate(maps(Q[b, :, i], Ki, scale)):
                by, t = (abs(L[i]), second) if m else (1.0, first)
                E = 3 * e + 2.0 ** -17 + 2.0 ** -22 * l
                dz = np.abs(by * P * (Y - (gi * t).sum(1, keepdims=True)))
                F = (half + E + SUMS) * dz + by * P * ed
                tq[b, :, i, at] = abs(scale) * (F @ np.abs(Ki[:, at]))
                tk[b, :n, j, at] += abs(scale) * (F.T @ np.abs(Q[b, :, i, at]))
                tv[b, :n, j] += ((half + E + SUMS) * by * P).T @ a
                if m:
                    tl[i] += (P * ((E + SUMS) * np.abs(Y) + ed)).sum()
    if lam.numel() == 1:
        tl = tl.sum(keepdims=True)
    for name, x, r, t, own in zip(("dq", "dk", "dv", "dlam"), got, ref, (tq, tk, tv, tl),
                                  (half, half, half, 2.0 ** -24)):
        err = np.abs(f64(x) - r)
        worst = (err - t - own * np.abs(r)).max()
        assert worst <= 1e-37, (name, err.max(), worst)
    for b, n in enumerate(lens):
        assert (got[1][b, n:] == 0).all() and (got[2][b, n:] == 0).all()


def lengths(lens):
    return torch.tensor(lens, dtype=torch.int32, device=DEV)


CASES = [  # B, Sq, Sk, h, hk, D, lens, packed
    (1, 1, 1, 1, 1, 64, None, False),
    (1, 1, 2, 4, 1, 128, None, False),
    (2, 300, 77, 3, 3, 128, [77, 16], False),      # text of 77 states
    (3, 129, 128, 2, 2, 64, [128, 0, 1], True),    # full tiles, an empty batch, one state
    (2, 40, 300, 6, 2, 128, [257, 128], True),     # three heads a group (21 tokens a subtile)
    (2, 23, 130, 10, 2, 64, [129, 127], False),    # five heads a group
    (4, 1, 2000, 24, 8, 128, [2000, 1999, 130, 0], False),   # a serving step
    (1, 1, 8192, 2, 2, 64, None, False),           # two rows in all, runs of states
    (1, 5, 700, 64, 1, 64, [641], False),          # 64 heads on one key head
    (2, 1, 1900, 14, 2, 128, [1900, 385], True),   # seven heads a group, runs
    (1, 1537, 513, 2, 1, 128, None, True),
    (2, 333, 150, 4, 2, 128, [150, 90], "heads"),
    (3, 17, 300, 6, 2, 64, [300, 0, 65], True),
    (160, 2, 70, 2, 1, 64, None, False),           # more units than SMs
    (2, 900, 64, 14, 2, 128, [64, 50], False),
    (3, 6, 2300, 4, 4, 128, [2300, 700, 0], True),   # few rows, runs of states
    (2, 2100, 200, 12, 12, 128, [199, 64], False),   # several units a CTA
    (1, 2, 1300, 3, 3, 64, [1290], True),            # two rows a key head
    (3, 4, 700, 2, 2, 64, [700, 0, 3], "heads"),     # four
    (2, 2, 1100, 4, 2, 128, [1100, 513], True),      # two tokens of two heads
    (70, 1, 600, 3, 1, 128, None, False),            # three
    (2, 4900, 1100, 2, 2, 64, [1100, 70], False),    # 156 units in 152 pieces
    (1, 9800, 1030, 2, 2, 128, None, False),         # 154
    (2, 10000, 1030, 2, 2, 64, [1030, 800], False),  # 316: 152 go round, the others are cut
    (40, 3, 1100, 4, 2, 128, [1100, 0, 5, 700, 64] * 8, False),  # 80 units of all lengths
    (3, 40, 5000, 4, 2, 64, [5000, 0, 4321], True),  # few long units, each in many parts
]


def fill_behind(k, v, lens):
    for b, m in enumerate(lens or []):
        k[b, m:] = float("nan")
        v[b, m:] = float("inf") if b % 2 else float("nan")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,Sq,Sk,h,hk,D,lens,packed", CASES)
def test_forward(nabla, B, Sq, Sk, h, hk, D, lens, packed, dtype):
    q, k, v, lam, _ = inputs(B, Sq, Sk, h, hk, D, dtype, seed=Sk, packed=packed, one=Sk % 2 == 1)
    n = None if lens is None else lengths(lens)
    fill_behind(k, v, lens)  # what lies behind the lengths must not matter
    o, o2, lse = nabla.nabla_diff_attn_fwd_lse(q, k, v, lam, kv_len=n)
    assert nabla.nabla_get_last_device_status() == 0
    check_forward(o, o2, lse, q, k, v, lam, lens or [Sk] * B, math.sqrt(2 / D))
    assert torch.equal(nabla.nabla_diff_attn_fwd(q, k, v, lam, kv_len=n), o)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,Sq,Sk,h,hk,D,lens,packed", CASES)
def test_backward(nabla, B, Sq, Sk, h, hk, D, lens, packed, dtype):
    q, k, v, lam, dout = inputs(B, Sq, Sk, h, hk, D, dtype, seed=Sk, packed=packed,
                                one=Sk % 2 == 1)
    n = None if lens is None else lengths(lens)
    fill_behind(k, v, lens)
    o, o2, lse = nabla.nabla_diff_attn_fwd_lse(q, k, v, lam, kv_len=n)
    if packed == "heads":
        o, o2 = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (o, o2))
    got = nabla.nabla_diff_attn_bwd(q, k, v, lam, o, o2, lse, dout, kv_len=n)
    assert nabla.nabla_get_last_device_status() == 0
    check_backward(got, q, k, v, lam, o, o2, dout, lens or [Sk] * B, math.sqrt(2 / D))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale,weight", [(0.0, 0.5), (-0.3, -1.5), (1.1, 0.0), (0.2, 30.0)])
def test_scales_and_weights(nabla, dtype, scale, weight):
    q, k, v, lam, dout = inputs(2, 70, 200, 2, 2, 64, dtype, seed=7, spread=0.8)
    lam.fill_(weight)
    n = lengths([200, 73])
    o, o2, lse = nabla.nabla_diff_attn_fwd_lse(q, k, v, lam, kv_len=n, scale=scale)
    check_forward(o, o2, lse, q, k, v, lam, [200, 73], scale)
    got = nabla.nabla_diff_attn_bwd(q, k, v, lam, o, o2, lse, dout, kv_len=n, scale=scale)
    check_backward(got, q, k, v, lam, o, o2, dout, [200, 73], scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scores_that_jump(nabla, dtype):
    """Scores that rise by hundreds of base-2 units from tile to tile, in one map and in rows
    apart: the running bias has to be raised and O rescaled, in each map for itself."""
    q, k, v, lam, _ = inputs(1, 200, 640, 2, 2, 64, dtype, seed=8, spread=0.5)
    k[0, 130:140, 0, :32] *= 12.0
    k[0, 300, 0] *= 60.0
    k[0, 520:600, 1, 32:] *= 40.0
    q[0, ::3] *= 8.0
    q[0, 5] = 0.0
    o, o2, lse = nabla.nabla_diff_attn_fwd_lse(q, k, v, lam)
    assert nabla.nabla_get_last_device_status() == 0
    check_forward(o, o2, lse, q, k, v, lam, [640], math.sqrt(2 / 64))


def test_equal_maps_leave_nothing(nabla):
    """q_1 = q_2, k_1 = k_2, lam = 1: the same sums in both maps, o = 0 to the bit in bf16."""
    q, k, v, lam, _ = inputs(1, 300, 500, 2, 1, 128, "bf16", seed=3)
    q[..., 64:], k[..., 64:] = q[..., :64].clone(), k[..., :64].clone()
    lam.fill_(1.0)
    o, o2, lse = nabla.nabla_diff_attn_fwd_lse(q, k, v, lam)
    assert torch.equal(lse[:, :, 0], lse[:, :, 1])
    assert float(o.abs().max()) <= 2.0 ** -22 * float(o2.abs().max())


def test_bad_lengths_are_clamped_and_reported(nabla):
    q, k, v, lam, dout = inputs(3, 20, 50, 2, 2, 64, "bf16", seed=9)
    good, bad = lengths([50, 0, 50]), lengths([51, -1, 50])
    want = nabla.nabla_diff_attn_fwd_lse(q, k, v, lam, kv_len=good)
    grads = nabla.nabla_diff_attn_bwd(q, k, v, lam, *want, dout, kv_len=good)
    assert nabla.nabla_get_last_device_status() == 0
    got = nabla.nabla_diff_attn_fwd_lse(q, k, v, lam, kv_len=bad)
    assert nabla.nabla_get_last_device_status() == BAD_INDEX
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    got = nabla.nabla_diff_attn_bwd(q, k, v, lam, *want, dout, kv_len=bad)
    assert nabla.nabla_get_last_device_status() == BAD_INDEX
    assert all(torch.equal(a, b) for a, b in zip(grads, got))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Sq,Sk", [(1, 3000), (600, 300)])
def test_repeats_streams_and_graphs(nabla, Sq, Sk, dtype):
    """Same bits from call to call, on another stream, and from two graphs with a workspace
    each; a replay reads the lengths anew."""
    B, h, hk, D = 2, 6, 2, 128
    q, k, v, lam, dout = inputs(B, Sq, Sk, h, hk, D, dtype, seed=10)
    n = lengths([Sk, Sk // 2 + 1])

    def call(**kw):
        f = nabla.nabla_diff_attn_fwd_lse(q, k, v, lam, kv_len=n, workspace=kw.get("fws"),
                                          stream=kw.get("stream"))
        return [*f, *nabla.nabla_diff_attn_bwd(q, k, v, lam, *f, dout, kv_len=n,
                                               workspace=kw.get("bws"), stream=kw.get("stream"))]

    def same(a, b):
        return all(torch.equal(x, y) for x, y in zip(a, b))

    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = call(stream=side)
    side.synchronize()
    assert same(want, other) and same(want, call())
    sizes = (q.dtype, B, Sq, Sk, h, hk, D)
    graphs = []
    for _ in range(2):
        fws = torch.empty(max(nabla.nabla_diff_attn_fwd_workspace_bytes(*sizes), 1),
                          dtype=torch.uint8, device=DEV)
        bws = torch.empty(nabla.nabla_diff_attn_bwd_workspace_bytes(*sizes), dtype=torch.uint8,
                          device=DEV)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            outs = call(fws=fws, bws=bws)
        graphs.append((g, outs, fws, bws))
    with torch.cuda.stream(side):
        graphs[0][0].replay()
    graphs[1][0].replay()
    torch.cuda.synchronize()
    assert same(want, graphs[0][1]) and same(want, graphs[1][1])
    n.copy_(lengths([1, 3 * Sk // 4]))
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert same(graphs[0][1], call())


@pytest.mark.parametrize("which", range(4))
def test_gradients_along_directions_against_differences(nabla, which):
    """fp32: the change of <dout, o>, formed in 64 bits, along a random direction.  o is off
    by at most 2^-16 of about 3 an element, so the quotient by 2 * 3 * 2^-16 * sum |dout| /
    step at most, and by a hundredth of that where the errors' signs differ; the third-order
    term is below 1e-3 of the change at this step."""
    q, k, v, lam, dout = inputs(2, 9, 40, 4, 2, 64, "f32", seed=12, spread=0.8)
    n = lengths([40, 23])
    o, o2, lse = nabla.nabla_diff_attn_fwd_lse(q, k, v, lam, kv_len=n)
    grads = nabla.nabla_diff_attn_bwd(q, k, v, lam, o, o2, lse, dout, kv_len=n)
    x = [q, k, v, lam]
    d = torch.randn(x[which].shape, generator=torch.Generator().manual_seed(which)).to(DEV)
    step = 2.0 ** -9

    def loss(by):
        y = list(x)
        y[which] = x[which] + by * d
        return float((nabla.nabla_diff_attn_fwd(*y, kv_len=n).double() * dout).sum())

    got = (loss(step) - loss(-step)) / (2 * step)
    want = float((grads[which].double() * d).sum())
    room = 2 * 3 * 2.0 ** -16 * float(dout.abs().sum()) / step / 100
    assert abs(got - want) <= room + 1e-3 * float((grads[which].double() * d).abs().sum())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_past_32_bits(nabla, dtype):
    """Rows more than 2^31 elements apart give the bits of the dense call."""
    n, h, D = 260, 2, 64
    pitch = 2 ** 31 // (n - 1) // 8 * 8 + 64
    q, k, v, lam, dout = inputs(1, n, n, h, h, D, dtype, seed=5)

    def far(t):
        room = torch.empty((n - 1) * pitch + h * D, dtype=t.dtype, device=DEV)
        view = room.as_strided((1, n, h, D), (room.numel(), pitch, D, 1))
        view.copy_(t)
        return view

    want = nabla.nabla_diff_attn_fwd_lse(q, k, v, lam)
    fq, fk, fv = far(q), far(k), far(v)
    got = nabla.nabla_diff_attn_fwd_lse(fq, fk, fv, lam)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    grads = nabla.nabla_diff_attn_bwd(q, k, v, lam, *want, dout)
    got = nabla.nabla_diff_attn_bwd(fq, fk, fv, lam, far(want[0]), far(want[1]), want[2],
                                    far(dout))
    assert all(torch.equal(a, b) for a, b in zip(grads, got))
    assert nabla.nabla_get_last_device_status() == 0
