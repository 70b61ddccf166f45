"""The gated sum with norm in 64 bits on the inputs' own device (rows by the ten thousand are
too many for the oracle), its gradient by automatic differentiation, and for each element the
size that the fp32 kernels' errors are proportional to:

  s     2^-17 of |x| + |rs gate pw| N(u), N(t) = r (|t| + mean|t|) (rms: r |t|);
  y     2^-16 of |w (1 + scale)| (r S + (1 + |n|) r rms(S)) + |shift|, S the size of s;
  dx    2^-16 of T = |dsum| + r (g + mean g + N mean(g N)), g = |dy w (1 + scale)|;
  du    2^-15 of r (e + mean e + N mean(e N)), e = |rs gate pw| T (no post norm: of e);
  sums  2^-14 of the sum of the terms' sizes;
each plus half a step of the stored type.  A row's sum is a chain of at most 16 additions in a
thread, 5 in a warp and 16 over warps, 2^-24 each, so a mean is off by less than 2^-18 mean|t|
and a normed value by 2^-17 N; a gradient is three such sums; a sum over tokens adds at most
500 additions in a chain (a run, then the runs 32 at a time) to its terms' 2^-15."""
import torch

EPS = 1e-6
TOLERANCE = dict(s=-17, y=-16, dx=-16, du=-15, dgate=-14, dscale=-14, dshift=-14, dw=-14, dpw=-14)


class Inputs:
    """Inputs of a call on [B, S, C]; rows: modulation rows of a batch; branch: "" for none, "u",
    or the post norm's name; weights: the norms have some."""

    def __init__(self, B, S, C, dtype, norm, branch, rows, mtype=torch.float32, weights=True,
                 rs=0.7, seed=0, device="cuda:0"):
        g = torch.Generator(device=device).manual_seed(seed)

        def draw(*shape, s=1.0, m=0.0, kind=dtype):
            return (torch.randn(*shape, generator=g, device=device) * s + m).to(kind)

        self.norm, self.post, self.rs = norm, branch if branch not in ("", "u") else None, rs
        self.x, self.u = draw(B, S, C, s=1.5, m=0.4), draw(B, S, C, s=0.9) if branch else None
        self.dsum, self.dy = draw(B, S, C), draw(B, S, C)
        p = draw(B, rows, 3, C, s=0.4, kind=mtype)  # one projection
        self.gate = p[:, :, 0] if branch else None
        self.scale, self.shift = p[:, :, 1], p[:, :, 2]
        self.w = draw(C, s=0.2, m=1.0) if weights else None
        self.pw = draw(C, s=0.2, m=1.0) if weights and self.post else None

    def args(self):
        return dict(gate=self.gate, scale=self.scale, shift=self.shift, weight=self.w,
                    post_weight=self.pw, norm=self.norm, post_norm=self.post,
                    residual_scale=self.rs, eps=EPS)


def wide(t):
    return None if t is None else t.detach().double()


def tokens(m, S):
    """Rows of the modulations over the tokens."""
    return m.repeat_interleave(S // m.shape[1], 1)


def by_rows(t, m):
    B, rows, C = m.shape
    return t.reshape(B, rows, -1, C).sum(2)


def normed(t, kind):
    if kind == "layer":
        t = t - t.mean(-1, keepdim=True)
    return t * (t * t).mean(-1, keepdim=True).add(EPS).rsqrt()


def magnitudes(t, kind):
    a = t.abs()
    if kind is None:
        return torch.ones_like(t[..., :1]), a
    c = t - t.mean(-1, keepdim=True) if kind == "layer" else t
    r = (c * c).mean(-1, keepdim=True).add(EPS).rsqrt()
    return r, r * (a + a.mean(-1, keepdim=True) if kind == "layer" else a)


def mean(t):
    return t.mean(-1, keepdim=True)


def branch_part(c, u, gate, pw):
    b = normed(u, c.post) if c.post else u
    return c.rs * tokens(gate, u.shape[1]) * (b if pw is None else b * pw)


def norm_part(c, s, w, scale, shift):
    n = normed(s, c.norm)
    n = n if w is None else n * w
    return n * (1.0 + tokens(scale, s.shape[1])) + tokens(shift, s.shape[1])


def forward(c):
    """{name: (value, size)} of s (where there is a branch) and y."""
    x, u, gate, scale, shift, w, pw = (
        wide(t) for t in (c.x, c.u, c.gate, c.scale, c.shift, c.w, c.pw))
    S = x.shape[1]
    out, s, size = {}, x, x.abs()
    if u is not None:
        s = x + branch_part(c, u, gate, pw)
        by = c.rs * tokens(gate, S).abs()
        size = size + (by if pw is None else by * pw.abs()) * magnitudes(u, c.post)[1]
        out["s"] = s, size
    n, (r, _) = normed(s, c.norm), magnitudes(s, c.norm)
    up = (1.0 + tokens(scale, S)).abs()
    up = up if w is None else up * w.abs()
    of_y = up * (r * size + (1 + n.abs()) * r * mean(size * size).sqrt()) + tokens(shift, S).abs()
    out["y"] = norm_part(c, s, w, scale, shift), of_y
    return out


def backward(c, s):
    """{name: (value, size)} of the gradients, from the sum s that the forward left."""
    s, u, dsum, dy, gate, scale, shift, w, pw = (wide(t) for t in (
        s, c.u, c.dsum, c.dy, c.gate, c.scale, c.shift, c.w, c.pw))
    S = s.shape[1]
    leaves = dict(dx=s, dscale=scale, dshift=shift, dw=w)
    leaves = {k: t.requires_grad_() for k, t in leaves.items() if t is not None}
    y = norm_part(c, s, w, scale, shift)
    got = dict(zip(leaves, torch.autograd.grad((y * dy).sum(), list(leaves.values()))))
    ds = got["dx"] = got["dx"] + dsum
    leaves = {k: t.requires_grad_() for k, t in dict(du=u, dgate=gate, dpw=pw).items()
              if t is not None}
    if u is not None:
        b = branch_part(c, u, gate, pw)
        got.update(zip(leaves, torch.autograd.grad((b * ds).sum(), list(leaves.values()))))
    with torch.no_grad():
        r, N = magnitudes(s, c.norm)
        a = 1.0 if w is None else w.abs()
        more = (1.0 + tokens(scale, S)).abs()
        g = dy.abs() * more * a
        T = dsum.abs() + r * (g + mean(g) + N * mean(g * N))
        sizes = dict(dx=T, dscale=by_rows(dy.abs() * N * a, scale), dshift=by_rows(dy.abs(), shift),
                     dw=(dy.abs() * N * more).sum((0, 1)))
        if u is not None:
            by = c.rs * tokens(gate, S).abs()
            pa = 1.0 if pw is None else pw.abs()
            r, M = magnitudes(u, c.post)
            e = by * pa * T
            sizes.update(du=e if c.post is None else r * (e + mean(e) + M * mean(e * M)),
                         dgate=by_rows(c.rs * pa * T * M, gate), dpw=(by * T * M).sum((0, 1)))
    return {k: (t, sizes[k]) for k, t in got.items()}


GRADS = ("dx", "du", "dgate", "dscale", "dshift", "dw", "dpw")


def check(name, got, value, size):
    assert got.shape == value.shape, name
    half = torch.finfo(got.dtype).eps / 2
    room = half * value.abs() + 2.0 ** TOLERANCE[name] * size + 1e-38
    over = (got.double() - value).abs() - room
    assert bool((over <= 0).all()), (name, float(over.max()), int((over > 0).sum()))
