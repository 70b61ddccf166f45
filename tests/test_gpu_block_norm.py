"""The gated sum with adaptive norm on the GPU vs the fp64 oracle, through the binding.

Tolerances, from the arithmetic (eps24 = 2^-24, half = half a step of the stored type).  A
row's sum is a chain of at most 16 additions in a thread, 5 in a warp and 16 over the warps:
37 eps24 of the sum of magnitudes, so a mean is off by at most 2^-18 mean|t|, and with the
squares about it, the root and the products a normed value n = (t - mean) r by less than
2^-17 N, N = r (|t| + mean|t|).
  s         2^-17 of S = |x| + |rs gate pw| N(u);  then half of it for the store.
  y         s's error times r, what it changes of the mean and of r (at most the root mean
            square of it, times 1 + |n|), and the norm's own: 2^-16 of
            |w (1 + scale)| (r S + (1 + |n|) r rms(S)) + |shift|;  then half.
  dx        three such sums of products: 2^-16 of T = |dsum| + r (g + mean g + N mean(g N)),
            g = |dy w (1 + scale)|;  then half.
  du        the same of e = |rs gate pw| T: 2^-15 of r (e + mean e + N mean(e N));  then half.
  sums      a term is off by 2^-15 of its size with T and N as above; a run here has at most
            48 rows, runs are added in chains of at most 32 + 32: 128 eps24 more.  2^-14 of
            the sum of the terms' sizes;  then half.
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


def half(t):
    return torch.finfo(t.dtype).eps / 2


def f64(t):
    return None if t is None else t.double().cpu().numpy()


class Case:
    """Inputs of one call; mod: None, "one", "batch", or the modulation rows of a batch."""

    def __init__(self, B, S, C, dtype, norm, post, mod, mtype="f32", weights=True, branch=True,
                 rs=0.7, seed=0, mean=0.4, views=False):
        g = torch.Generator().manual_seed(seed)
        dt, mt = TYPES[dtype], TYPES[mtype]

        def draw(*shape, s=1.0, m=0.0, kind=dt):
            return (torch.randn(*shape, generator=g) * s + m).to(kind).to(DEV)

        def plane(**kw):
            if not views:
                return draw(B, S, C, **kw)
            return draw(B, S + 3, 2, C, **kw)[:, :S, 1]  # batches and tokens further apart

        self.norm, self.post, self.rs = norm, post, rs
        self.x, self.u = plane(s=1.5, m=mean), plane(s=0.9, m=-mean) if branch else None
        rows = {None: None, "one": (), "batch": (B,)}.get(mod, (B, mod))
        p = None if rows is None else draw(*rows, 3, C, s=0.4, kind=mt)  # one projection
        at = [None] * 3 if p is None else [p[..., i, :] for i in range(3)]
        self.gate = at[0] if branch else None
        self.scale, self.shift = at[1:] if norm else (None, None)
        self.w = draw(C, s=0.2, m=1.0) if weights and norm else None
        self.pw = draw(C, s=0.2, m=1.0) if weights and post else None
        self.dsum, self.dy = plane(), plane() if norm else None

    def args(self):
        return dict(gate=self.gate, scale=self.scale, shift=self.shift, weight=self.w,
                    post_weight=self.pw, norm=self.norm, post_norm=self.post,
                    residual_scale=self.rs, eps=EPS)

    def host(self):
        return [f64(t) for t in (self.gate, self.scale, self.shift, self.w, self.pw)]


def magnitudes(t, kind):
    """r and N = r (|t| + mean|t|) of the rows of t."""
    _, r = O.normed(t, kind, EPS)
    a = np.abs(t)
    return r, r * (a + (a.mean(-1, keepdims=True) if kind == "layer" else 0.0))


def factor(B, S, *parts):
    """The product of |weights| and |1 + scale| or |gate| over the tokens."""
    out = np.ones((B, S, 1))
    for p in parts:
        if p is not None:
            out = out * np.abs(O.over_tokens(p, B, S))
    return out


def mean(t):
    return t.mean(-1, keepdims=True)


def check_forward(c, s, y):
    x, u = f64(c.x), f64(c.u)
    B, S, _ = x.shape
    gate, scale, shift, w, pw = c.host()
    rs_, ry = O.block_norm(x, u, gate, scale, shift, w, pw, c.norm, c.post, c.rs, EPS)
    size = np.abs(x)
    if u is not None:
        size = size + c.rs * factor(B, S, gate, pw) * magnitudes(u, c.post)[1]
        assert s.shape == c.x.shape and s.dtype == c.x.dtype
        assert np.all(np.abs(f64(s) - rs_) <= half(s) * np.abs(rs_) + 2.0 ** -17 * size)
    if c.norm is None:
        assert y is None
        return
    n, r = O.normed(rs_, c.norm, EPS)
    up = factor(B, S, w, None if scale is None else 1.0 + scale)
    size = up * (r * size + (1 + np.abs(n)) * r * np.sqrt(mean(size * size)))
    size = size + (0.0 if shift is None else np.abs(O.over_tokens(shift, B, S)))
    assert np.all(np.abs(f64(y) - ry) <= half(y) * np.abs(ry) + 2.0 ** -16 * size)


def check_backward(c, s, got):
    s, u, dsum, dy = (f64(t) for t in (s, c.u, c.dsum, c.dy))
    B, S, C = s.shape
    gate, scale, shift, w, pw = c.host()
    want = O.block_norm_bwd(s, u, dsum, dy, gate, scale, shift, w, pw, c.norm, c.post, c.rs, EPS)
    up = factor(B, S, w, None if scale is None else 1.0 + scale)
    T = 0.0 if dsum is None else np.abs(dsum)
    sizes = [None] * 7
    if c.norm is not None:
        r, N = magnitudes(s, c.norm)
        g = np.abs(dy) * up
        T = T + r * (g + mean(g) + N * mean(g * N))
        terms = np.abs(dy) * N
        if scale is not None:
            sizes[3] = O.by_rows(terms * factor(B, S, w), scale.shape)
            sizes[4] = O.by_rows(np.abs(dy), scale.shape)
        if w is not None:
            sizes[5] = (terms * factor(B, S, None if scale is None else 1.0 + scale)).sum((0, 1))
    sizes[0] = T
    if u is not None:
        e = c.rs * factor(B, S, gate, pw) * T
        r, M = magnitudes(u, c.post)
        sizes[1] = e if c.post is None else r * (e + mean(e) + M * mean(e * M))
        if gate is not None:
            sizes[2] = O.by_rows(c.rs * factor(B, S, pw) * T * M, gate.shape)
        if pw is not None:
            sizes[6] = (c.rs * factor(B, S, gate) * T * M).sum((0, 1))
    like = (c.x, c.u, c.gate, c.scale, c.shift, c.w, c.pw)
    for a, ref, size, t, tol in zip(got, want, sizes, like, (-16, -15) + (-14,) * 5):
        assert (a is None) == (ref is None) == (t is None)
        if a is not None:
            assert a.shape == t.shape and a.dtype == t.dtype
            err = np.abs(f64(a) - ref)
            assert np.all(err <= half(a) * np.abs(ref) + 2.0 ** tol * size + 1e-38)


CASES = [  # B, S, C, dtype, norm, post, modulations, their type, weights, branch
    (1, 1, 8, "bf16", "rms", None, "batch", "f32", True, True),        # the smallest row
    (16, 1, 2048, "bf16", "rms", None, "batch", "f32", True, True),    # a serving step
    (2, 37, 64, "f32", "layer", "rms", "one", "f32", True, True),      # a team of 8 lanes
    (3, 41, 72, "bf16", "layer", "layer", "batch", "bf16", True, True),
    (2, 30, 128, "bf16", "rms", "rms", 10, "f32", True, True),
    (1, 203, 256, "f32", "layer", None, 29, "bf16", False, True),
    (2, 50, 264, "bf16", "layer", "rms", 50, "f32", True, True),       # a row a token
    (2, 33, 1112, "f32", "layer", "rms", 11, "f32", True, True),
    (1, 700, 1536, "bf16", "layer", None, "batch", "bf16", False, False),  # the norm alone
    (2, 310, 2048, "bf16", "layer", None, "batch", "bf16", False, True),
    (1, 64, 2056, "bf16", "rms", "layer", "one", "f32", True, True),   # the last warp nearly empty
    (2, 350, 2152, "bf16", "layer", "rms", 5, "bf16", True, True),     # several rows a block
    (1, 640, 2560, "bf16", "rms", "layer", "batch", "f32", True, True),
    (1, 640, 2560, "f32", "layer", "layer", "batch", "bf16", True, True),
    (2, 200, 512, "bf16", "layer", None, 25, "f32", True, True),       # 4 to 16 tokens a row
    (2, 640, 1024, "bf16", "rms", "rms", 160, "f32", True, True),
    (1, 19, 4096, "f32", "rms", "rms", None, "f32", True, True),
    (2, 9, 4104, "bf16", "layer", "rms", 3, "f32", True, True),        # two vectors a thread
    (1, 11, 8192, "f32", "layer", "layer", "batch", "f32", True, True),
    (1, 300, 512, "bf16", None, "rms", "batch", "f32", True, True),    # the sum alone
    (2, 5, 320, "f32", None, None, "batch", "f32", False, True),
    (4, 3000, 64, "bf16", "layer", None, 6, "f32", True, True),        # rows over many runs
]


@pytest.mark.parametrize("B,S,C,dtype,norm,post,mod,mtype,weights,branch", CASES)
@pytest.mark.parametrize("views", [False, True])
def test_forward_and_backward(nabla, B, S, C, dtype, norm, post, mod, mtype, weights, branch,
                              views):
    c = Case(B, S, C, dtype, norm, post, mod, mtype, weights, branch, seed=S + C, views=views)
    s, y = nabla.nabla_block_norm(c.x, c.u, **c.args())
    check_forward(c, s, y)
    got = nabla.nabla_block_norm_bwd(s, c.u, c.dsum, c.dy, **c.args())
    check_backward(c, s, got)
    again = nabla.nabla_block_norm_bwd(s, c.u, c.dsum, c.dy, **c.args())
    assert all(a is b or torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_mean_that_dwarfs_the_spread(nabla, dtype):
    """Rows of 300 + noise: squares about the mean, not a difference of squares.  (The
    oracle takes the stored values; N of the tolerance holds the mean.)"""
    c = Case(2, 21, 1024, dtype, "layer", "layer", "batch", mean=300.0)
    s, y = nabla.nabla_block_norm(c.x, c.u, **c.args())
    check_forward(c, s, y)
    check_backward(c, s, nabla.nabla_block_norm_bwd(s, c.u, c.dsum, c.dy, **c.args()))


def test_rows_of_zeros_and_of_no_number(nabla):
    c = Case(1, 6, 512, "f32", "layer", "rms", "batch")
    c.x[0, 0] = 0.0
    c.u[0, 0] = 0.0          # s = 0: y = shift
    c.u[0, 3, 5] = float("nan")  # stays in its row
    c.x[0, 4, 7] = float("inf")
    s, y = nabla.nabla_block_norm(c.x, c.u, **c.args())
    assert torch.equal(y[0, 0], c.shift[0])
    assert torch.isnan(y[0, 3]).all() and torch.isnan(y[0, 4]).any()
    good = [1, 2, 5]
    c.x, c.u = c.x[:, good].contiguous(), c.u[:, good].contiguous()
    check_forward(c, s[:, good], y[:, good])


def test_no_residual_gradient(nabla):
    c = Case(2, 13, 320, "bf16", "rms", "rms", "batch")
    s, _ = nabla.nabla_block_norm(c.x, c.u, **c.args())
    c.dsum = None
    check_backward(c, s, nabla.nabla_block_norm_bwd(s, c.u, None, c.dy, **c.args()))


def test_in_place(nabla):
    """x_out over x, dx over dsum, and outputs between others that stay as they were."""
    c = Case(2, 45, 640, "bf16", "layer", "rms", "batch")
    s, y = nabla.nabla_block_norm(c.x, c.u, **c.args())
    grads = nabla.nabla_block_norm_bwd(s, c.u, c.dsum, c.dy, **c.args())
    room = torch.full((2, 45, 3, 640), 5.0, dtype=torch.bfloat16, device=DEV)
    x = c.x.clone()
    s2, y2 = nabla.nabla_block_norm(x, c.u, x_out=x, y=room[:, :, 1], **c.args())
    assert s2 is x and torch.equal(x, s) and torch.equal(y2, y)
    assert (room[:, :, 0] == 5).all() and (room[:, :, 2] == 5).all()
    d = c.dsum.clone()
    again = nabla.nabla_block_norm_bwd(x, c.u, d, c.dy, dx=d, du=room[:, :, 2], **c.args())
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    assert (room[:, :, 0] == 5).all() and torch.equal(room[:, :, 1], y)


@pytest.mark.parametrize("C", [64, 1536])
def test_streams_and_graphs(nabla, C):
    """The same bits on another stream and from a graph whose inputs change."""
    c, e = (Case(2, 500, C, "bf16", "layer", "rms", 4, seed=i) for i in (1, 2))
    e.gate, e.scale, e.shift, e.w, e.pw = c.gate, c.scale, c.shift, c.w, c.pw

    def call(t):
        s, y = nabla.nabla_block_norm(t.x, t.u, **t.args())
        return [s, y, *nabla.nabla_block_norm_bwd(s, t.u, t.dsum, t.dy, **t.args())]

    want = [call(t) for t in (c, e)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = call(e)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want[1], other))
    s, y = nabla.nabla_block_norm(e.x, e.u, stream=side, **e.args())
    side.synchronize()
    assert torch.equal(s, want[1][0]) and torch.equal(y, want[1][1])
    live = Case(2, 500, C, "bf16", "layer", "rms", 4, seed=1)
    live.gate, live.scale, live.shift, live.w, live.pw = c.gate, c.scale, c.shift, c.w, c.pw
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = call(live)
    for new, ref in ((e, want[1]), (c, want[0])):
        for n in ("x", "u", "dsum", "dy"):
            getattr(live, n).copy_(getattr(new, n))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, outs))


def test_gradients_against_differences(nabla):
    """Central differences of <dsum, s> + <dy, y> with the forward itself in fp32, formed in
    64 bits: s and y are off by at most 2^-16 of about 8 here, so the quotient by
    2 * 96 * 8 * 2^-16 / step; the third-order term is below 2e-3 at this step."""
    c = Case(1, 2, 48, "f32", "layer", "rms", "batch", rs=1.0)
    s, _ = nabla.nabla_block_norm(c.x, c.u, **c.args())
    got = nabla.nabla_block_norm_bwd(s, c.u, c.dsum, c.dy, **c.args())
    step = 2.0 ** -5
    bound = 2 * 96 * 8 * 2.0 ** -16 / step + 2e-3

    def loss():
        s, y = nabla.nabla_block_norm(c.x, c.u, **c.args())
        return float((s.double() * c.dsum).sum() + (y.double() * c.dy).sum())

    for name, grad in zip(("x", "u", "gate", "scale", "shift", "w", "pw"), got):
        t = getattr(c, name)
        for j in (0, 7, 8, 47):
            at = (0,) * (t.dim() - 1) + (j,)
            keep = t[at].clone()
            t[at] = keep + step
            hi = loss()
            t[at] = keep - step
            lo = loss()
            t[at] = keep
            assert abs((hi - lo) / (2 * step) - float(grad[at])) <= bound, (name, j)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_past_32_bits(nabla, dtype):
    """Rows more than 2^31 elements apart give the bits of the dense call."""
    n, C = 260, 128
    pitch = 2 ** 31 // (n - 1) // 8 * 8 + 64
    c = Case(1, n, C, dtype, "layer", "rms", 5)

    def far(t):
        room = torch.empty((n - 1) * pitch + C, dtype=t.dtype, device=DEV)
        view = room.as_strided((1, n, C), (room.numel(), pitch, 1))
        view.copy_(t)
        return view

    s, y = nabla.nabla_block_norm(c.x, c.u, **c.args())
    want = nabla.nabla_block_norm_bwd(s, c.u, c.dsum, c.dy, **c.args())
    x, u = far(c.x), far(c.u)
    fs, fy = nabla.nabla_block_norm(x, u, y=far(y), **c.args())
    assert torch.equal(fs, s) and torch.equal(fy, y)
    got = nabla.nabla_block_norm_bwd(far(s), u, far(c.dsum), far(c.dy), dx=x, **c.args())
    assert all(torch.equal(a, b) for a, b in zip(want, got))
