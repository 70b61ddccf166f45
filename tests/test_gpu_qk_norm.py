"""Per-head RMS norm with rotation on the GPU vs the fp64 oracle, through the binding.

Tolerances, from the arithmetic (eps24 = 2^-24, the largest relative error of one fp32
operation; half = half a step of the stored type, 2^-8 for bf16 and 2^-24 for fp32):
  forward   r: a tree of 8 + log2(D/8) <= 12 additions, halved by the root, plus the
            reciprocal root (2 ulp = 4 eps24); r w, x (r w) and the rotation's two
            products and sum: at most 6 + 4 + 2 + 3 = 15 eps24 of |a c| + |b s|, below
            2^-20 of |a| + |b|; then half of the result for the store.
  dx        two such sums, and up to 8 more operations: below 2^-18 of
            r (|g| + |x| r^2 mean|g x|); then half.
  dw        a lane adds at most 24 rows an item here, two items, then 8 + 32 + 32
            partial sums: a chain of at most 128 additions, 2^-17 of sum |dy x r| (the
            terms' own error is within it); then half.
"""
import numpy as np
import pytest
import torch

from oracle import nabla_oracle as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


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


def half(dt):
    return torch.finfo(dt).eps / 2


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def table(rows, R, seed=0):
    rng = np.random.default_rng(seed)
    a = rng.uniform(-1000.0, 1000.0, (rows, R // 2))
    return (torch.from_numpy(np.cos(a)).float().to(DEV),
            torch.from_numpy(np.sin(a)).float().to(DEV))


def inputs(B, S, hq, hk, D, dtype, seed=0, packed=False, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[dtype]
    if packed == "heads":  # heads before tokens
        q = (torch.randn(B, hq, S, D, generator=g) * spread).to(dt).to(DEV).transpose(1, 2)
        k = (torch.randn(B, hk, S, D, generator=g) * spread).to(dt).to(DEV).transpose(1, 2)
    elif packed:  # views of one projection
        x = (torch.randn(B, S, (hq + 2 * hk) * D, generator=g) * spread).to(dt).to(DEV)
        q = x[..., :hq * D].view(B, S, hq, D)
        k = x[..., hq * D:(hq + hk) * D].view(B, S, hk, D) if hk else None
    else:
        q = (torch.randn(B, S, hq, D, generator=g) * spread).to(dt).to(DEV)
        k = (torch.randn(B, S, hk, D, generator=g) * spread).to(dt).to(DEV) if hk else None
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(dt).to(DEV) for _ in range(2)]
    return q, k, w[0], w[1] if hk else None


def tokens(cos, sin, pos, B, S, R):
    """The oracle's angles [B or 1, S, R/2]."""
    if cos is None:
        return np.zeros((1, S, 0)), np.zeros((1, S, 0))
    c, s = f64(cos), f64(sin)
    return (c[None, :S], s[None, :S]) if pos is None else (c[pos.cpu().numpy()],
                                                          s[pos.cpu().numpy()])


def pair_size(y, R, pairs):
    """|a| + |b| of every column's pair (|y| for columns that are not rotated)."""
    a = np.abs(y).copy()
    if pairs:
        s = a[..., 0:R:2] + a[..., 1:R:2]
        a[..., 0:R:2] = a[..., 1:R:2] = s
    else:
        s = a[..., :R // 2] + a[..., R // 2:R]
        a[..., :R // 2] = a[..., R // 2:R] = s
    return a


def check_forward(z, x, w, c, s, pairs, eps=EPS):
    ref = O.qk_norm_rope(f64(x), f64(w), c, s, pairs, eps)
    none = np.zeros((1, x.shape[1], 0))
    size = pair_size(O.qk_norm_rope(f64(x), f64(w), none, none, pairs, eps), 2 * c.shape[-1],
                     pairs)
    err = np.abs(f64(z) - ref)
    assert np.all(err <= half(z.dtype) * np.abs(ref) + 2.0 ** -20 * size + 1e-38)


def check_backward(dx, dw, x, w, dz, c, s, pairs, eps=EPS):
    X, W, Z = f64(x), f64(w), f64(dz)
    rx, rw = O.qk_norm_rope_bwd(X, W, Z, c, s, pairs, eps)
    dy = O.rotate(Z, c, -s, pairs)
    size_dy = pair_size(Z, 2 * c.shape[-1], pairs)
    r = 1 / np.sqrt((X * X).mean(-1, keepdims=True) + eps)
    g = size_dy * (1.0 if W is None else np.abs(W))
    size = r * (g + np.abs(X) * r * r * (g * np.abs(X)).mean(-1, keepdims=True))
    assert np.all(np.abs(f64(dx) - rx) <= half(dx.dtype) * np.abs(rx) + 2.0 ** -18 * size + 1e-38)
    if W is None:
        assert dw is None
        return
    terms = (np.maximum(np.abs(dy), size_dy * 2.0 ** -20) * np.abs(X) * r).sum((0, 1, 2))
    assert np.all(np.abs(f64(dw) - rw) <= half(dw.dtype) * np.abs(rw) + 2.0 ** -17 * terms)


CASES = [  # B, S, hq, hk, D, R, dtype, pairs, packed, positions
    (1, 1, 1, 1, 64, 64, "bf16", True, False, False),      # one token, one head
    (3, 1, 24, 8, 128, 128, "bf16", False, False, True),   # a serving step
    (2, 37, 5, 3, 128, 96, "bf16", True, True, False),     # odd everything, in the projection
    (2, 37, 5, 3, 128, 96, "f32", False, True, True),
    (1, 130, 7, 2, 64, 16, "f32", True, False, True),      # only 16 columns rotated
    (1, 130, 7, 2, 64, 48, "bf16", False, True, False),
    (2, 9, 4, 4, 128, 0, "bf16", True, False, False),      # norm alone
    (1, 257, 6, 0, 64, 32, "bf16", False, False, False),   # q alone
    (2, 300, 24, 24, 128, 128, "f32", True, False, False),
    (2, 50, 6, 3, 64, 64, "bf16", True, "heads", False),
    (5, 1, 3, 1, 64, 64, "bf16", False, False, True),      # few heads: runs of tokens
    (3, 37, 2, 1, 128, 96, "bf16", True, True, True),
    (1, 130, 1, 1, 64, 16, "f32", False, True, True),
    (2, 61, 4, 1, 128, 128, "f32", True, "heads", False),
]


@pytest.mark.parametrize("B,S,hq,hk,D,R,dtype,pairs,packed,positions", CASES)
def test_forward_and_backward(nabla, B, S, hq, hk, D, R, dtype, pairs, packed, positions):
    q, k, wq, wk = inputs(B, S, hq, hk, D, dtype, seed=S, packed=packed)
    cos, sin = table(max(S, 500) if positions else S, R) if R else (None, None)
    pos = None
    if positions and R:
        pos = torch.randint(0, cos.shape[0], (B, S), dtype=torch.int32,
                            generator=torch.Generator().manual_seed(1)).to(DEV)
    c, s = tokens(cos, sin, pos, B, S, R)
    zq, zk = nabla.nabla_qk_norm_rope(q, k, wq, wk, cos, sin, pos=pos, interleaved=pairs, eps=EPS)
    check_forward(zq, q, wq, c, s, pairs)
    if hk:
        check_forward(zk, k, wk, c, s, pairs)
    dzq, dzk, _, _ = inputs(B, S, hq, hk, D, dtype, seed=S + 1, packed=packed, spread=0.3)
    dq, dk, dwq, dwk = nabla.nabla_qk_norm_rope_bwd(q, k, wq, wk, dzq, dzk, cos, sin, pos=pos,
                                                    interleaved=pairs, eps=EPS)
    check_backward(dq, dwq, q, wq, dzq, c, s, pairs)
    if hk:
        check_backward(dk, dwk, k, wk, dzk, c, s, pairs)
    assert nabla.nabla_get_last_device_status() == 0


def test_no_weights_and_mixed_weight_type(nabla):
    q, k, wq, wk = inputs(2, 33, 4, 2, 128, "bf16")
    cos, sin = table(33, 128)
    c, s = tokens(cos, sin, None, 2, 33, 128)
    zq, zk = nabla.nabla_qk_norm_rope(q, k, None, None, cos, sin)
    check_forward(zq, q, None, c, s, True)
    check_forward(zk, k, None, c, s, True)
    dq, dk, dwq, dwk = nabla.nabla_qk_norm_rope_bwd(q, k, None, None, zq, zk, cos, sin)
    assert dwq is None and dwk is None
    check_backward(dq, None, q, None, zq, c, s, True)
    w32 = wq.float() * 1.001  # fp32 weights of a bf16 tensor, and one side without any
    dq, dk, dwq, dwk = nabla.nabla_qk_norm_rope_bwd(q, k, w32, None, zq, zk, cos, sin)
    assert dwq.dtype == torch.float32 and dwk is None
    check_backward(dq, dwq, q, w32, zq, c, s, True)
    check_backward(dk, None, k, None, zk, c, s, True)


def test_rows_of_zeros_and_extremes(nabla):
    q, _, wq, _ = inputs(1, 8, 2, 0, 64, "f32")
    q[0, 0] = 0.0                       # x = 0: z = 0, and dx = g / sqrt(eps)
    q[0, 1] *= 1e-15                    # mean square below eps
    q[0, 2] *= 1e15
    q[0, 3, 0, 5] = float("nan")        # stays in its row
    q[0, 4, 1, 7] = float("inf")
    cos, sin = table(8, 64)
    c, s = tokens(cos, sin, None, 1, 8, 64)
    z, _ = nabla.nabla_qk_norm_rope(q, None, wq, None, cos, sin)
    good = torch.ones(8, 2, dtype=torch.bool)
    good[3, 0] = good[4, 1] = False
    assert torch.isfinite(z[0].cpu()[good]).all()
    assert torch.isnan(z[0, 3, 0]).any() and torch.isnan(z[0, 4, 1]).any()
    keep = [0, 1, 2, 5, 6, 7]
    check_forward(z[:, keep], q[:, keep], wq, c[:, keep], s[:, keep], True)
    dz = torch.randn(1, 8, 2, 64, device=DEV)
    q[0, 3, 0, 5] = q[0, 4, 1, 7] = 0.25
    dx, _, dw, _ = nabla.nabla_qk_norm_rope_bwd(q, None, wq, None, dz, None, cos, sin)
    check_backward(dx, dw, q, wq, dz, c, s, True)


def test_strided_outputs_and_untouched_columns(nabla):
    """dq and dk written into one packed gradient: dv's columns stay as they were."""
    B, S, h, D = 2, 41, 3, 64
    q, k, wq, wk = inputs(B, S, h, h, D, "bf16", packed=True)
    cos, sin = table(S, D)
    dzq, dzk, _, _ = inputs(B, S, h, h, D, "bf16", seed=5)
    want = nabla.nabla_qk_norm_rope_bwd(q, k, wq, wk, dzq, dzk, cos, sin)
    pack = torch.full((B, S + 2, 3 * h * D), 7.0, dtype=torch.bfloat16, device=DEV)
    view = pack[:, :S]  # batches two tokens further apart than they need
    dq = view[..., :h * D].unflatten(-1, (h, D))
    dk = view[..., h * D:2 * h * D].unflatten(-1, (h, D))
    got = nabla.nabla_qk_norm_rope_bwd(q, k, wq, wk, dzq, dzk, cos, sin, dq=dq, dk=dk)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert (pack[:, S:] == 7).all() and (pack[..., 2 * h * D:] == 7).all()


def test_bad_position_is_reported_and_not_rotated(nabla):
    q, k, wq, wk = inputs(1, 6, 2, 2, 64, "bf16")
    cos, sin = table(10, 64)
    pos = torch.tensor([[0, 9, 10, -1, 3, 4]], dtype=torch.int32, device=DEV)
    zq, _ = nabla.nabla_qk_norm_rope(q, k, wq, wk, cos, sin, pos=pos)
    assert nabla.nabla_get_last_device_status() == 5  # NABLA_ERR_BAD_INDEX
    c, s = f64(cos), f64(sin)
    at = [0, 9, 0, 0, 3, 4]
    c, s = c[at][None].copy(), s[at][None].copy()
    c[0, 2:4], s[0, 2:4] = 1.0, 0.0
    check_forward(zq, q, wq, c, s, True)
    nabla.nabla_qk_norm_rope(q, k, wq, wk, cos, sin)  # six tokens, ten rows
    assert nabla.nabla_get_last_device_status() == 0


def test_weight_gradient_repeats_and_replays(nabla):
    """Same bits from call to call, on another stream and from a captured graph."""
    q, k, wq, wk = inputs(2, 1100, 6, 6, 128, "bf16")
    dzq, dzk, _, _ = inputs(2, 1100, 6, 6, 128, "bf16", seed=9)
    cos, sin = table(1100, 128)

    def call(**kw):
        return nabla.nabla_qk_norm_rope_bwd(q, k, wq, wk, dzq, dzk, cos, sin, **kw)

    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = call()
    torch.cuda.current_stream().wait_stream(side)
    outs = [torch.empty_like(t) for t in want]
    ws = torch.empty(nabla.nabla_qk_norm_rope_bwd_workspace_bytes(128), dtype=torch.uint8,
                     device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call(dq=outs[0], dk=outs[1], dwq=outs[2], dwk=outs[3], workspace=ws)
    for _ in range(2):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(want, other, outs):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_gradient_against_differences(nabla):
    """Central differences of sum(dz * z) with the forward itself, fp32.  The loss is
    formed in 64 bits from z, each element off by at most e = 2^-20 (|a| + |b|), so the
    quotient is off by sum |dz| e / step; the third-order term is below 1e-4 at this
    step and row size."""
    q, _, wq, _ = inputs(1, 2, 1, 0, 64, "f32", seed=3)
    cos, sin = table(2, 64)
    dz = torch.randn(1, 2, 1, 64, device=DEV)
    dx, _, dw, _ = nabla.nabla_qk_norm_rope_bwd(q, None, wq, None, dz, None, cos, sin)

    def loss(q, w):
        z, _ = nabla.nabla_qk_norm_rope(q, None, w, None, cos, sin)
        return float((z.double() * dz.double()).sum())

    step = 2.0 ** -6
    size = float((dz.abs().sum() * 2 * 4.0)) * 2.0 ** -20 / step
    for j in (0, 1, 31, 32, 63):
        e = torch.zeros_like(q)
        e[0, 1, 0, j] = step
        got = (loss(q + e, wq) - loss(q - e, wq)) / (2 * step)
        assert abs(got - float(dx[0, 1, 0, j])) <= size + 1e-4
        e = torch.zeros_like(wq)
        e[j] = step
        got = (loss(q, wq + e) - loss(q, wq - e)) / (2 * step)
        assert abs(got - float(dw[j])) <= size + 1e-4


def same_as_dense(nabla, q, k, wq, wk, qo, ko, room, marked):
    """Forward and backward into the views qo, ko of `room` give the dense calls' bits and
    write nothing else of it."""
    B, S, _, D = q.shape
    cos, sin = table(S, D)
    wanted = list(nabla.nabla_qk_norm_rope(q, k, wq, wk, cos, sin))
    dzq, dzk = (torch.randn(t.shape, generator=torch.Generator().manual_seed(1)).to(t.dtype)
                .to(DEV) for t in (q, k))
    wanted += nabla.nabla_qk_norm_rope_bwd(q, k, wq, wk, dzq, dzk, cos, sin)
    before = room.clone()
    got = list(nabla.nabla_qk_norm_rope(q, k, wq, wk, cos, sin, q_out=qo, k_out=ko))
    got = [t.clone() for t in got]
    got += nabla.nabla_qk_norm_rope_bwd(q, k, wq, wk, dzq, dzk, cos, sin, dq=qo, dk=ko)
    assert len(got) == len(wanted) == 6
    assert all(torch.equal(a, b) for a, b in zip(got, wanted))
    assert torch.equal(room[~marked], before[~marked])
    assert nabla.nabla_get_last_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_outputs_between_each_other(nabla, dtype):
    """q's and k's heads in one tensor, heads before tokens, batch after batch."""
    B, S, h, hk, D = 3, 21, 4, 2, 64
    q, k, wq, wk = inputs(B, S, h, hk, D, dtype)
    room = torch.full((B, h + hk + 1, S, D), 3.0, dtype=q.dtype, device=DEV)
    marked = torch.zeros_like(room, dtype=torch.bool)
    marked[:, 1:] = True
    same_as_dense(nabla, q, k, wq, wk, room[:, 1:1 + h].transpose(1, 2),
                  room[:, 1 + h:].transpose(1, 2), room, marked)


def test_outputs_in_tokens_of_an_odd_batch_pitch(nabla):
    """Batches apart by no whole number of tokens."""
    B, S, h, D = 2, 9, 2, 64
    q, k, wq, wk = inputs(B, S, h, h, D, "bf16")
    pitch = (2 * h + 1) * D
    room = torch.full((B * (S * pitch + 72),), 3.0, dtype=q.dtype, device=DEV)
    marked = torch.zeros_like(room, dtype=torch.bool)

    def views(x):
        st = (S * pitch + 72, pitch, D, 1)
        return x.as_strided((B, S, h, D), st), x[h * D:].as_strided((B, S, h, D), st)

    for x in views(marked):
        x.fill_(True)
    same_as_dense(nabla, q, k, wq, wk, *views(room), room, marked)


def test_outputs_beside_the_inputs(nabla):
    """q, k, v and the outputs side by side in one tensor of five."""
    B, S, h, D = 2, 37, 3, 128
    q, k, wq, wk = inputs(B, S, h, h, D, "bf16")
    room = torch.full((B, S, 5, h, D), 3.0, dtype=q.dtype, device=DEV)
    room[:, :, 0], room[:, :, 1] = q, k
    marked = torch.zeros_like(room, dtype=torch.bool)
    marked[:, :, 3:] = True
    same_as_dense(nabla, room[:, :, 0], room[:, :, 1], wq, wk, room[:, :, 3], room[:, :, 4], room,
                  marked)
