"""More operators of a video diffusion transformer block, as cases that can be timed
and compared:

  * "norm": what lies between two of the block's branches: the gated, optionally normed,
            scaled sum of the residual and a branch's output, and the adaptive norm that
            the next branch reads, and their gradient;
  * "diff": differential attention, the difference of two softmax maps with learned
            weights, of tokens to states of any length, and its gradient.

run() computes them in elementary torch operations in 32 bits, or, where `own`
is true, through the framework's entry points.  exact() is the operators'
definition in 64 bits.
"""
import math

import torch

own = False  # run() calls the framework's kernels where this is true

DEV = "cuda"
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
LOG2E = 1.4426950408889634


# ------------------------------------------------------------------ the cases

def norm_case(name, B, S, C, dtype="bf16", grad=False, norm="layer", post="", branch=True,
              mod="batch", frames=1, mtype="f32", weight=False, rscale=1.0):
    """norm, post: "rms", "layer" or "" (none), of the sum and of the branch's output;
    branch: there is one, with a gate; mod: the gate's, scale's and shift's rows: "one"
    for all tokens, one a "batch", or one for each of `frames` equal runs of a batch's
    tokens ("frames"); weight: the norms have learned weights too."""
    case = dict(op="norm", grad=grad, dtype=dtype, B=B, S=S, C=C, norm=norm, post=post,
                branch=branch, mod=mod, frames=frames, mtype=mtype, weight=weight, rscale=rscale)
    return dict(case, name=name) if name else case


def diff_case(name, B, Sq, Sk, h, hk, D, dtype="bf16", grad=False, lens=False, packed=False,
              each=True):
    """D: columns of a head's values, and of its two queries or keys of D / 2 together;
    lens: the batch's states have different lengths (lengths()); packed: k and v are views
    of one projection [B, Sk, 2, hk, D]; each: a learned weight for each head, else one."""
    case = dict(op="diff", grad=grad, dtype=dtype, B=B, Sq=Sq, Sk=Sk, h=h, hk=hk, D=D,
                lens=lens, packed=packed, each=each)
    return dict(case, name=name) if name else case


def listed():
    return [
        # one token for each of 16 requests between two branches: latency
        norm_case("norm step", 16, 1, 2048, norm="rms", weight=True),
        # the 480p latent (32768 tokens) before the first branch: the norm alone
        norm_case("norm 480p first", 1, 32768, 2048, branch=False),
        # the 720p latent between two branches, norms before and after them
        norm_case("norm 720p", 1, 98304, 1536, norm="rms", post="rms", weight=True),
        # the training step's backward at 480p, prompt and negative prompt
        norm_case("norm 480p grad", 2, 32768, 2048, grad=True, mtype="bf16"),
        # a 32-bit check of a small model, a row of modulations for each frame, odd sizes
        norm_case("norm frames f32 grad", 2, 1001, 1112, dtype="f32", grad=True, norm="layer",
                  post="rms", mod="frames", frames=13, weight=True, rscale=0.7),
        # one token for each of 16 requests against long states, shared heads
        diff_case("diff step", 16, 1, 4096, 24, 8, 128, lens=True),
        # prompt and negative prompt together (guidance): text padded to 512 states
        diff_case("diff 480p", 2, 32768, 512, 12, 12, 128, lens=True, packed=True),
        # every token of a short clip to every other
        diff_case("diff self", 1, 8192, 8192, 12, 12, 128, each=False),
        # the training step's backward at 480p
        diff_case("diff 480p grad", 1, 32768, 512, 12, 12, 128, grad=True),
        # a small model with shared heads of 64, ragged prompts of an odd length
        diff_case("diff ragged grad", 3, 1000, 333, 12, 4, 64, grad=True, lens=True),
        # 32-bit checks of a small model
        diff_case("diff f32", 1, 1024, 257, 2, 2, 64, dtype="f32"),
        diff_case("diff f32 grad", 2, 500, 77, 6, 2, 128, dtype="f32", grad=True, lens=True,
                  each=False),
    ]


def _log(rng, lo, hi):
    """A whole number, uniform over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    grad, dtype = rng.random() < 0.5, "f32" if rng.random() < 0.25 else "bf16"
    if rng.random() < 0.45:
        C = 8 * _log(rng, 8, 1024)
        B = _log(rng, 1, 16)
        most = 65536 * 2048 // (2 if dtype == "f32" else 1)
        S = _log(rng, 1, max(1, min(98304, most // (B * C))))
        branch, norm = rng.random() < 0.8, rng.choice(("rms", "layer", "layer"))
        post = rng.choice(("", "", "rms", "layer")) if branch else ""
        mod = rng.choice(("one", "batch", "batch", "frames"))
        frames = rng.choice([m for m in range(1, min(S, 64) + 1) if S % m == 0] + [S] * (S < 4096))
        return norm_case(None, B, S, C, dtype, grad, norm, post, branch, mod,
                         frames if mod == "frames" else 1, rng.choice(("f32", "bf16")),
                         rng.random() < 0.5, rng.choice((1.0, 0.5)))
    D = rng.choice((64, 128))
    hk = rng.choice((1, 2, 3, 4, 5, 8, 12, 16))
    h = hk * rng.choice([g for g in (1, 1, 2, 3, 4, 8) if g * hk <= 24])
    B = _log(rng, 1, 16)
    most = 12 * 128 * 512 * 32768 * (1 if grad else 4)  # B h Sq Sk D of the listed ones
    if dtype == "f32":
        most //= 64
    # one state alone has no gradient to compare: its softmax is constant, dq = dk = 0
    few = 2 if grad else 1
    Sk = _log(rng, few, max(few, min(8192, most // (B * h * D))))
    Sq = _log(rng, 1, max(1, min(98304, most // (B * h * D * max(Sk, 512)))))
    return diff_case(None, B, Sq, Sk, h, hk, D, dtype, grad, rng.random() < 0.6,
                     rng.random() < 0.3, rng.random() < 0.7)


def lengths(case):
    """The states each batch has: the first all of them, the others spread over the
    range (prompts of different lengths; 0 occurs where Sk is small)."""
    if not case["lens"]:
        return [case["Sk"]] * case["B"]
    return [case["Sk"] if b == 0 else int(case["Sk"] * ((b * 0.6180339887) % 1.0))
            for b in range(case["B"])]


def mod_shape(case):
    B, C = case["B"], case["C"]
    return {"one": (C,), "batch": (B, C), "frames": (B, case["frames"], C)}[case["mod"]]


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    dt = TYPES[case["dtype"]]

    def normal(*shape, spread=1.0, mean=0.0, kind=dt):
        return (torch.randn(*shape, generator=g, device=DEV) * spread + mean).to(kind)

    if case["op"] == "norm":
        B, S, C, mt = case["B"], case["S"], case["C"], TYPES[case["mtype"]]
        s = dict(op="norm", grad=case["grad"], norm=case["norm"], post=case["post"],
                 rscale=case["rscale"], u=None, gate=None, w=None, pw=None)
        s["x"] = normal(B, S, C, spread=1.7, mean=0.3)  # a residual that has grown
        rows = mod_shape(case)
        # one projection of the time embedding holds the modulations side by side
        n = 3 if case["branch"] else 2
        p = normal(*rows[:-1], n, C, spread=0.4, kind=mt) if case["mod"] != "one" else normal(
            n, C, spread=0.4, kind=mt)
        s["scale"], s["shift"] = p[..., 0, :], p[..., 1, :]
        if case["branch"]:
            s["u"], s["gate"] = normal(B, S, C, spread=0.9), p[..., 2, :]
        if case["weight"]:
            s["w"] = normal(C, spread=0.2, mean=1.0)
            if case["post"]:
                s["pw"] = normal(C, spread=0.2, mean=1.0)
        if case["grad"]:  # x is the sum that the forward left behind
            s["dy"], s["dsum"] = normal(B, S, C), normal(B, S, C)
        return s
    B, h, hk, D, Sq, Sk = (case[n] for n in ("B", "h", "hk", "D", "Sq", "Sk"))
    q = normal(B, Sq, h, D, spread=1.2)  # normed queries and keys with their weights
    if case["packed"]:
        kv = normal(B, Sk, 2, hk, D, spread=1.2)
        k, v = kv[:, :, 0], kv[:, :, 1]
    else:
        k, v = normal(B, Sk, hk, D, spread=1.2), normal(B, Sk, hk, D)
    lam = normal(h if case["each"] else 1, spread=0.1, mean=0.5, kind=torch.float32)
    s = dict(op="diff", grad=case["grad"], q=q, k=k, v=v, lam=lam, lens=None)
    if case["lens"]:
        s["lens"] = torch.tensor(lengths(case), dtype=torch.int32, device=DEV)
    if case["grad"]:  # what the forward of the training step left behind
        s["o"], s["o2"], s["lse"] = plain_diff(s, all_of_it=True)
        s["dout"] = normal(B, Sq, h, D)
    return s


# ------------------------------------------------------------------ plain forms: norm

def spread_rows(m, x):
    """A modulation's rows in 32 bits, over the tokens of x [B, S, C]."""
    B, S, C = x.shape
    f = m.float()
    if f.dim() == 3 and f.shape[1] != S:
        f = f.repeat_interleave(S // f.shape[1], 1)
    return f[:, None] if f.dim() == 2 else f


def gather_rows(t, m, x):
    """The transpose of spread_rows: the tokens' sums for each of a modulation's rows."""
    B, S, C = x.shape
    if m.dim() == 1:
        return t.sum((0, 1))
    if m.dim() == 2:
        return t.sum(1)
    return t.view(B, m.shape[1], S // m.shape[1], C).sum(2)


def center(f, kind):
    """The normed rows and what they were multiplied by."""
    if kind == "layer":
        f = f - f.mean(-1, keepdim=True)
    r = torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
    return f * r, r


def center_grad(d, n, r, kind):
    """The gradient of center() at its outputs n, r for the gradient d of n."""
    g = d - n * (d * n).mean(-1, keepdim=True)
    if kind == "layer":
        g = g - d.mean(-1, keepdim=True)
    return g * r


def plain_norm(s):
    x = s["x"]
    a = x.float()
    outs = []
    if s["u"] is not None:
        b = s["u"].float()
        if s["post"]:
            b = center(b, s["post"])[0]
            if s["pw"] is not None:
                b = b * s["pw"].float()
        a = a + s["rscale"] * spread_rows(s["gate"], x) * b
        outs.append(a.to(x.dtype))
    n = center(a, s["norm"])[0]
    if s["w"] is not None:
        n = n * s["w"].float()
    y = n * (1.0 + spread_rows(s["scale"], x)) + spread_rows(s["shift"], x)
    return outs + [y.to(x.dtype)]


def plain_norm_grad(s):
    x, w, pw = s["x"], s["w"], s["pw"]
    dy = s["dy"].float()
    n, r = center(x.float(), s["norm"])
    up = 1.0 + spread_rows(s["scale"], x)
    wf = 1.0 if w is None else w.float()
    ds = s["dsum"].float() + center_grad(dy * up * wf, n, r, s["norm"])
    out = dict(dx=ds.to(x.dtype))
    if s["u"] is not None:
        b, rb = s["u"].float(), None
        gate = s["rscale"] * spread_rows(s["gate"], x)
        if s["post"]:
            b, rb = center(b, s["post"])
        pf = 1.0 if pw is None else pw.float()
        db = ds * gate
        out["dgate"] = gather_rows(ds * b * (s["rscale"] * pf), s["gate"], x).to(s["gate"].dtype)
        if pw is not None:
            out["dpw"] = (db * b).sum((0, 1)).to(pw.dtype)
        if s["post"]:
            db = center_grad(db * pf, b, rb, s["post"])
        out["du"] = db.to(x.dtype)
    out["dscale"] = gather_rows(dy * n * wf, s["scale"], x).to(s["scale"].dtype)
    out["dshift"] = gather_rows(dy, s["shift"], x).to(s["shift"].dtype)
    if w is not None:
        out["dw"] = (dy * up * n).sum((0, 1)).to(w.dtype)
    return [out[k] for k in NORM_GRADS if k in out]


NORM_GRADS = ("dx", "du", "dgate", "dscale", "dshift", "dw", "dpw")


# ------------------------------------------------------------------ plain forms: diff

def heads(x, hk):
    """[B, S, h, D] -> [B, hk, S h / hk, D] in 32 bits: the rows that share a key head."""
    B, S, h, D = x.shape
    return x.float().reshape(B, S, hk, h // hk, D).permute(0, 2, 1, 3, 4).reshape(B, hk, -1, D)


def rows(x, S, h):
    """heads() undone: [B, hk, S h / hk, D] -> [B, S, h, D]."""
    B, hk, _, D = x.shape
    return x.reshape(B, hk, S, h // hk, D).permute(0, 2, 1, 3, 4).reshape(B, S, h, D)


def weights(s):
    """The learned weights of the rows of heads(): [1, hk, S h / hk, 1]."""
    S, h = s["q"].shape[1:3]
    hk = s["k"].shape[2]
    lam = s["lam"].expand(h).reshape(1, hk, 1, h // hk)
    return lam.expand(1, hk, S, h // hk).reshape(1, hk, -1, 1)


def plain_map(s, which):
    """Softmax of one map over each batch's states (rows without any: all 0) and the
    scores' base-2 log-sum-exp."""
    d = s["k"].shape[-1] // 2
    k = s["k"].float().transpose(1, 2)[..., which * d:(which + 1) * d]
    q = heads(s["q"], k.shape[1])[..., which * d:(which + 1) * d]
    z = q @ k.transpose(-1, -2) * (1.0 / math.sqrt(d))
    if s["lens"] is not None:
        out = torch.arange(k.shape[2], device=DEV) >= s["lens"][:, None, None, None]
        z = z.masked_fill(out, -math.inf)
    m = z.amax(-1, keepdim=True).clamp_min(-3e38)
    p = (z - m).exp()
    total = p.sum(-1, keepdim=True)
    return p / total.clamp_min(1e-37), ((m + total.log()) * LOG2E)[..., 0]


def plain_diff(s, all_of_it=False):
    S, h = s["q"].shape[1:3]
    v, kind = s["v"].float().transpose(1, 2), s["q"].dtype
    p1, l1 = plain_map(s, 0)
    p2, l2 = plain_map(s, 1)
    if not all_of_it:
        return rows((p1 - weights(s) * p2) @ v, S, h).to(kind)
    o2 = p2 @ v
    o = p1 @ v - weights(s) * o2
    B, hk = l1.shape[:2]
    lse = torch.stack([t.reshape(B, hk, S, h // hk).transpose(2, 3).reshape(B, h, S)
                       for t in (l1, l2)], 2).contiguous()  # [B, h, 2, S]
    return rows(o, S, h).to(kind), rows(o2, S, h).to(kind), lse


def plain_diff_grad(s):
    S, h = s["q"].shape[1:3]
    hk, D = s["k"].shape[2:]
    d, kind, lam = D // 2, s["q"].dtype, weights(s)
    dout, k, q = heads(s["dout"], hk), s["k"].float().transpose(1, 2), heads(s["q"], hk)
    dp = dout @ s["v"].float().permute(0, 2, 3, 1)
    t2 = (dout * heads(s["o2"], hk)).sum(-1, keepdim=True)
    t1 = (dout * heads(s["o"], hk)).sum(-1, keepdim=True) + lam * t2
    p, _ = plain_map(s, 0)
    total = p
    dq, dk = [], []
    for which, t, by in ((0, t1, 1.0), (1, t2, -lam)):
        if which:
            p, _ = plain_map(s, 1)
            total = total - lam * p
        dz = p * (dp - t) * by * (1.0 / math.sqrt(d))
        dq.append(dz @ k[..., which * d:(which + 1) * d])
        dk.append(dz.transpose(-1, -2) @ q[..., which * d:(which + 1) * d])
    dv = total.transpose(-1, -2) @ dout
    # from the map itself: o2 is rounded to the inputs' type, lam's gradient is not
    dlam = -rows((p * dp).sum(-1, keepdim=True).double(), S, h).sum((0, 1))[:, 0]
    if s["lam"].numel() == 1:
        dlam = dlam.sum(0, keepdim=True)
    dlam = dlam.float()
    return [rows(torch.cat(dq, -1), S, h).to(kind), torch.cat(dk, -1).transpose(1, 2).to(kind),
            dv.transpose(1, 2).to(kind), dlam]


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    if own:
        from block_sparse_attention_nablat_gb300 import nabla

        if s["op"] == "norm":
            args = dict(gate=s["gate"], scale=s["scale"], shift=s["shift"], weight=s["w"],
                        post_weight=s["pw"], norm=s["norm"], post_norm=s["post"] or None,
                        residual_scale=s["rscale"], eps=EPS)
            if s["grad"]:
                return [t for t in nabla.nabla_block_norm_bwd(s["x"], s["u"], s["dsum"], s["dy"],
                                                              **args) if t is not None]
            total, y = nabla.nabla_block_norm(s["x"], s["u"], **args)
            return [y] if s["u"] is None else [total, y]
        if s["grad"]:
            return list(nabla.nabla_diff_attn_bwd(s["q"], s["k"], s["v"], s["lam"], s["o"],
                                                  s["o2"], s["lse"], s["dout"], kv_len=s["lens"]))
        return nabla.nabla_diff_attn_fwd(s["q"], s["k"], s["v"], s["lam"], kv_len=s["lens"])
    if s["op"] == "norm":
        return plain_norm_grad(s) if s["grad"] else plain_norm(s)
    return plain_diff_grad(s) if s["grad"] else plain_diff(s)


# ------------------------------------------------------------------ cost

def work(case):
    e, B = SIZE[case["dtype"]], case["B"]
    if case["op"] == "norm":
        x, m = B * case["S"] * case["C"], SIZE[case["mtype"]]
        side = (3 if case["branch"] else 2) * math.prod(mod_shape(case)) * m
        side += case["weight"] * (2 if case["post"] else 1) * case["C"] * e
        if case["grad"]:  # sum, u, dsum, dy in; dx, du out; modulations and their gradients
            return {"bytes": (6 if case["branch"] else 4) * x * e + 2 * side,
                    "flops": (30 if case["branch"] else 16) * x}
        return {"bytes": (4 if case["branch"] else 2) * x * e + side,
                "flops": (10 if case["branch"] else 6) * x}
    h, hk, D = case["h"], case["hk"], case["D"]
    rows_, keys = case["Sq"] * h * D, sum(lengths(case))
    pairs = case["Sq"] * h * D * keys  # a product over all of D: 2 flops each
    if case["grad"]:  # q, o, o2, dout in, dq out; k, v in; dk, dv out over the padded length
        b = (5 * B * rows_ + 2 * keys * hk * D + 2 * B * case["Sk"] * hk * D) * e
        # scores, dout v, dv, dq, dk: the two maps' halves make up a whole product each
        return {"bytes": b + 8 * B * h * case["Sq"], "flops": 10 * pairs}
    # scores (two halves), and the difference of the maps times v: one product each
    return {"bytes": (2 * B * rows_ + 2 * keys * hk * D) * e, "flops": 4 * pairs}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return exact_norm(s) if case["op"] == "norm" else exact_diff(s, case)


def exact_norm(s):
    """sum = x + rscale gate N(u) pw, y = N(sum) w (1 + scale) + shift with N(t) = (t - mean)
    / sqrt(var + eps), or t / sqrt(mean t^2 + eps), a batch at a time; the gradient by
    automatic differentiation of that."""
    x = s["x"]
    B, S, C = x.shape

    def normed(t, kind):
        if kind == "layer":
            return (t - t.mean(-1, keepdim=True)) / (t.var(-1, keepdim=True, unbiased=False)
                                                      + EPS).sqrt()
        return t / (t.pow(2).mean(-1, keepdim=True) + EPS).sqrt()

    names = [n for n in ("gate", "scale", "shift", "w", "pw") if s[n] is not None]
    par = {n: s[n].double().requires_grad_(s["grad"]) for n in names}
    sums, ys, dxs, dus = [], [], [], []
    for b in range(B):
        def row(n):
            m = par[n]
            if m.dim() == 1:
                return m
            m = m[b:b + 1] if m.dim() == 2 else m[b]
            return m[:, None].expand(-1, S // m.shape[0], -1).reshape(S, C)

        total = x[b].double().requires_grad_(s["grad"])
        y = normed(total, s["norm"])
        inner = total
        if s["u"] is not None:
            u = s["u"][b].double().requires_grad_(s["grad"])
            branch = normed(u, s["post"]) if s["post"] else u
            if "pw" in par:
                branch = branch * par["pw"]
            branch = branch * row("gate") * s["rscale"]
            if not s["grad"]:
                inner = total + branch
                sums.append(inner)
                y = normed(inner, s["norm"])
        if "w" in par:
            y = y * par["w"]
        y = y * (1 + row("scale")) + row("shift")
        if not s["grad"]:
            ys.append(y)
            continue
        dy, ds = s["dy"][b].double(), s["dsum"][b].double()
        y.backward(dy)
        ds = ds + total.grad  # x's gradient, and the sum's, which goes on to the branch
        dxs.append(ds)
        if s["u"] is not None:
            branch.backward(ds)
            dus.append(u.grad)
    if not s["grad"]:
        return ([torch.stack(sums)] if sums else []) + [torch.stack(ys)]
    out = [torch.stack(dxs)] + ([torch.stack(dus)] if dus else [])
    return out + [par[n].grad for n in names]


def exact_diff(s, case):
    """o = (softmax(q1 k1^T / sqrt(d)) - lam softmax(q2 k2^T / sqrt(d))) v over each batch's
    states, a batch's head at a time; the gradient by automatic differentiation of that."""
    B, S, h, D = s["q"].shape
    hk, d = s["k"].shape[2], D // 2
    kind = dict(dtype=torch.float64, device=DEV)
    o, dq = torch.zeros(B, S, h, D, **kind), torch.zeros(B, S, h, D, **kind)
    dk = torch.zeros(*s["k"].shape, **kind)
    dv = torch.zeros_like(dk)
    dlam = torch.zeros(s["lam"].numel(), **kind)
    for b, n in enumerate(lengths(case)):
        for i in range(h if n else 0):
            j, at = i // (h // hk), min(i, s["lam"].numel() - 1)
            leaf = [t.double().requires_grad_(s["grad"]) for t in (
                s["q"][b, :, i], s["k"][b, :n, j], s["v"][b, :n, j], s["lam"][at])]
            q, k, v, lam = leaf
            first = torch.softmax(q[:, :d] @ k[:, :d].T / math.sqrt(d), -1)
            second = torch.softmax(q[:, d:] @ k[:, d:].T / math.sqrt(d), -1)
            out = (first - lam * second) @ v
            if s["grad"]:
                out.backward(s["dout"][b, :, i].double())
                dq[b, :, i] = q.grad
                dk[b, :n, j] += k.grad
                dv[b, :n, j] += v.grad
                dlam[at] += lam.grad
            else:
                o[b, :, i] = out
    return [dq, dk, dv, dlam] if s["grad"] else o
