"""The operators around the block-sparse self-attention of a video diffusion
transformer block, as cases that can be timed and compared:

  * "qk":    RMS norm of queries and keys per head, with the position rotation
             in the same pass, and its gradient (input, weights);
  * "cross": attention of the video tokens to an encoder's states of another
             length (padded prompts, shared key/value heads), and its gradient.

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

def qk_case(name, B, S, h, hk, D, R, dtype="bf16", grad=False, pairs=True, packed=False,
            pos=False):
    """pairs: rotate (2i, 2i + 1), else (i, i + R / 2); packed: q and k are views of
    one projection [B, S, (h + 2 hk) D]; pos: the tokens' rows of the rotation
    table are given ([B, S]), else token s takes row s."""
    case = dict(op="qk", grad=grad, dtype=dtype, B=B, S=S, h=h, hk=hk, D=D, R=R, pairs=pairs,
                packed=packed, pos=pos)
    return dict(case, name=name) if name else case


def cross_case(name, B, Sq, Sk, h, hk, D, dtype="bf16", grad=False, lens=False, packed=False):
    """lens: the batch's states have different lengths (lengths()); packed: k and v
    are views of one projection [B, Sk, 2, hk, D]."""
    case = dict(op="cross", grad=grad, dtype=dtype, B=B, Sq=Sq, Sk=Sk, h=h, hk=hk, D=D,
                lens=lens, packed=packed)
    return dict(case, name=name) if name else case


def listed():
    return [
        # one token for each of 16 requests, keys on fewer heads, positions given: latency
        qk_case("qk step", 16, 1, 24, 8, 128, 128, pairs=False, pos=True),
        # the 480p latent's self-attention inputs (8x8x8 blocks of 64 tokens, 24 heads)
        qk_case("qk 480p", 1, 32768, 24, 24, 128, 128),
        # the 720p latent, queries and keys still lying in the packed projection
        qk_case("qk 720p packed", 1, 98304, 24, 24, 128, 128, packed=True),
        # the training step's backward at 480p
        qk_case("qk 480p grad", 1, 32768, 24, 24, 128, 128, grad=True),
        # a 32-bit check of a small model: odd length, odd heads, half of the head rotated
        qk_case("qk f32 grad", 2, 1001, 5, 3, 64, 32, dtype="f32", grad=True, pairs=False),
        # one token for each of 16 requests against long encoder states, shared heads
        cross_case("cross step", 16, 1, 4096, 24, 8, 128, lens=True),
        # prompt and negative prompt together (guidance): text padded to 512 states
        cross_case("cross 480p", 2, 32768, 512, 24, 24, 128, lens=True, packed=True),
        # the 720p latent against one full-length prompt
        cross_case("cross 720p", 1, 98304, 512, 24, 24, 128),
        # the training step's backward at 480p
        cross_case("cross 480p grad", 1, 32768, 512, 24, 24, 128, grad=True),
        # a small model with shared heads of 64, ragged prompts of an odd length
        cross_case("cross ragged grad", 3, 1000, 333, 12, 4, 64, grad=True, lens=True),
        # 32-bit checks of a small model against a 257-state image encoding
        cross_case("cross f32", 1, 1024, 257, 2, 2, 64, dtype="f32"),
        cross_case("cross f32 grad", 2, 500, 77, 6, 2, 128, dtype="f32", grad=True, lens=True),
    ]


def _log(rng, lo, hi):
    """A whole number, uniform over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    grad, dtype = rng.random() < 0.5, "f32" if rng.random() < 0.25 else "bf16"
    D = rng.choice((64, 128))
    hk = rng.choice((1, 2, 3, 4, 5, 8, 12, 16, 24))
    h = hk * rng.choice([g for g in (1, 1, 2, 3, 4, 8) if g * hk <= 32])
    B = _log(rng, 1, 16)
    if rng.random() < 0.4:
        # at most the elements of the listed 480p (with its gradient) or 720p latent
        most = (32768 if grad else 98304) * 48 * 128 // (2 if dtype == "f32" else 1)
        S = _log(rng, 1, max(1, min(98304, most // (B * (h + hk) * D))))
        R = rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= D] + [D, D])
        return qk_case(None, B, S, h, hk, D, R, dtype, grad, rng.random() < 0.5,
                       rng.random() < 0.5, rng.random() < 0.3)
    most = 24 * 128 * 512 * (32768 if grad else 98304)  # B h Sq Sk D of the listed ones
    if dtype == "f32":
        most //= 64
    # one state alone has no gradient to compare: its softmax is constant, dq = dk = 0
    few = 2 if grad else 1
    Sk = _log(rng, few, max(few, min(8192, most // (B * h * D))))
    Sq = _log(rng, 1, max(1, min(98304, most // (B * h * D * max(Sk, 512)))))
    return cross_case(None, B, Sq, Sk, h, hk, D, dtype, grad, rng.random() < 0.6,
                      rng.random() < 0.3)


def lengths(case):
    """The states each batch has: the first all of them, the others spread over the
    range (prompts of different lengths; 0 occurs where Sk is small)."""
    if not case["lens"]:
        return [case["Sk"]] * case["B"]
    return [case["Sk"] if b == 0 else int(case["Sk"] * ((b * 0.6180339887) % 1.0))
            for b in range(case["B"])]


# ------------------------------------------------------------------ inputs

def table(case):
    """cos and sin [rows, R / 2], angles in 64 bits, kept in 32."""
    rows = max(case["S"], 4096) if case["pos"] else case["S"]
    n = case["R"] // 2
    freq = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=DEV),
                     -torch.arange(n, dtype=torch.float64, device=DEV) / n)
    a = torch.arange(rows, dtype=torch.float64, device=DEV)[:, None] * freq
    return a.cos().float().contiguous(), a.sin().float().contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    dt = TYPES[case["dtype"]]
    B, h, hk, D = case["B"], case["h"], case["hk"], case["D"]

    def normal(*shape, spread=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device=DEV) * spread + mean).to(dt)

    if case["op"] == "qk":
        S = case["S"]
        if case["packed"]:
            x = normal(B, S, (h + 2 * hk) * D, spread=1.3)
            q = x[..., :h * D].view(B, S, h, D)
            k = x[..., h * D:(h + hk) * D].view(B, S, hk, D)
        else:
            q, k = normal(B, S, h, D, spread=1.3), normal(B, S, hk, D, spread=0.8)
        cos, sin = table(case)
        s = dict(op="qk", grad=case["grad"], pairs=case["pairs"], q=q, k=k, cos=cos, sin=sin,
                 wq=normal(D, spread=0.2, mean=1.0), wk=normal(D, spread=0.2, mean=1.0), pos=None)
        if case["pos"]:
            s["pos"] = torch.randint(0, cos.shape[0], (B, S), generator=g, device=DEV,
                                     dtype=torch.int32)
        if case["grad"]:
            s["dq"], s["dk"] = normal(B, S, h, D), normal(B, S, hk, D)
        return s
    Sq, Sk = case["Sq"], case["Sk"]
    q = normal(B, Sq, h, D, spread=1.2)  # normed queries and keys with their weights
    if case["packed"]:
        kv = normal(B, Sk, 2, hk, D, spread=1.2)
        k, v = kv[:, :, 0], kv[:, :, 1]
    else:
        k, v = normal(B, Sk, hk, D, spread=1.2), normal(B, Sk, hk, D)
    s = dict(op="cross", grad=case["grad"], q=q, k=k, v=v, lens=None)
    if case["lens"]:
        s["lens"] = torch.tensor(lengths(case), dtype=torch.int32, device=DEV)
    if case["grad"]:  # what the forward of the training step left behind
        s["o"], s["lse"] = plain_cross(s, lse=True)
        s["dout"] = normal(B, Sq, h, D)
    return s


# ------------------------------------------------------------------ plain forms

def rotate(x, c, s, pairs):
    """The first 2 c.shape[-1] columns of x rotated by the angles' cos and sin."""
    n = c.shape[-1]
    if pairs:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        r = torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        r = torch.cat((a * c - b * s, a * s + b * c), -1)
    return torch.cat((r, x[..., 2 * n:]), -1)


def angles(s, which):
    """cos or sin of every token's angles, [B or 1, S, 1, R / 2]."""
    t = s[which]
    return (t[s["pos"].long()] if s["pos"] is not None else t[None])[:, :, None]


def plain_qk(s):
    c, n = angles(s, "cos"), angles(s, "sin")
    return [plain_norm(s["q"], s["wq"], c, n, s["pairs"]),
            plain_norm(s["k"], s["wk"], c, n, s["pairs"])]


def plain_norm(x, w, c, n, pairs):
    f = x.float()
    y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS) * w.float()
    return rotate(y, c, n, pairs).to(x.dtype)


def plain_norm_grad(x, w, dz, c, n, pairs):
    f = x.float()
    dy = rotate(dz.float(), c, -n, pairs)  # the rotation's transpose
    r = torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
    xh = f * r
    g = dy * w.float()
    dx = r * (g - xh * (g * xh).mean(-1, keepdim=True))
    return dx.to(x.dtype), (dy * xh).sum((0, 1, 2)).to(w.dtype)


def heads(x, hk):
    """[B, S, h, D] -> [B, hk, S h / hk, D] in 32 bits: the rows that share a key head."""
    B, S, h, D = x.shape
    return x.float().reshape(B, S, hk, h // hk, D).permute(0, 2, 1, 3, 4).reshape(B, hk, -1, D)


def rows(x, S, h):
    """heads() undone: [B, hk, S h / hk, D] -> [B, S, h, D]."""
    B, hk, _, D = x.shape
    return x.reshape(B, hk, S, h // hk, D).permute(0, 2, 1, 3, 4).reshape(B, S, h, D)


def plain_probs(s):
    """Softmax over each batch's states (rows without any: all 0) and the scores'
    base-2 log-sum-exp."""
    k = s["k"].float().transpose(1, 2)
    z = heads(s["q"], k.shape[1]) @ k.transpose(-1, -2) * (1.0 / math.sqrt(k.shape[-1]))
    if s["lens"] is not None:
        out = torch.arange(k.shape[2], device=DEV) >= s["lens"][:, None, None, None]
        z = z.masked_fill(out, -math.inf)
    m = z.amax(-1, keepdim=True).clamp_min(-3e38)
    p = (z - m).exp()
    total = p.sum(-1, keepdim=True)
    lse = (m + total.log()) * LOG2E
    return p / total.clamp_min(1e-37), lse[..., 0]


def plain_cross(s, lse=False):
    S, h = s["q"].shape[1:3]
    p, l2 = plain_probs(s)
    o = rows(p @ s["v"].float().transpose(1, 2), S, h).to(s["q"].dtype)
    if not lse:
        return o
    B, hk = l2.shape[:2]
    return o, l2.reshape(B, hk, S, h // hk).transpose(2, 3).reshape(B, h, S).contiguous()


def plain_cross_grad(s):
    S, h = s["q"].shape[1:3]
    hk, D = s["k"].shape[2:]
    scale = 1.0 / math.sqrt(D)
    p, _ = plain_probs(s)
    dout = heads(s["dout"], hk)
    dv = p.transpose(-1, -2) @ dout
    dp = dout @ s["v"].float().permute(0, 2, 3, 1)
    dz = p * (dp - (dout * heads(s["o"], hk)).sum(-1, keepdim=True)) * scale
    dq = dz @ s["k"].float().transpose(1, 2)
    dk = dz.transpose(-1, -2) @ heads(s["q"], hk)
    kind = s["q"].dtype
    return [rows(dq, S, h).to(kind), dk.transpose(1, 2).to(kind), dv.transpose(1, 2).to(kind)]


def run(state):
    s = state
    if own:
        from block_sparse_attention_nablat_gb300 import nabla

        if s["op"] == "qk":
            if s["grad"]:
                return nabla.nabla_qk_norm_rope_bwd(
                    s["q"], s["k"], s["wq"], s["wk"], s["dq"], s["dk"], s["cos"], s["sin"],
                    pos=s["pos"], interleaved=s["pairs"], eps=EPS)
            return nabla.nabla_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"],
                                            pos=s["pos"], interleaved=s["pairs"], eps=EPS)
        if s["grad"]:
            return nabla.nabla_cross_attn_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["dout"],
                                              kv_len=s["lens"])
        return nabla.nabla_cross_attn_fwd(s["q"], s["k"], s["v"], kv_len=s["lens"])
    if s["op"] == "qk":
        if not s["grad"]:
            return plain_qk(s)
        c, n = angles(s, "cos"), angles(s, "sin")
        dq, dwq = plain_norm_grad(s["q"], s["wq"], s["dq"], c, n, s["pairs"])
        dk, dwk = plain_norm_grad(s["k"], s["wk"], s["dk"], c, n, s["pairs"])
        return [dq, dk, dwq, dwk]
    return plain_cross_grad(s) if s["grad"] else plain_cross(s)


# ------------------------------------------------------------------ cost

def work(case):
    e, B, h, hk, D = SIZE[case["dtype"]], case["B"], case["h"], case["hk"], case["D"]
    if case["op"] == "qk":
        x = B * case["S"] * (h + hk) * D
        tokens = case["S"] * (B if case["pos"] else 1)
        side = tokens * case["R"] * 4 + (4 * B * case["S"] if case["pos"] else 0) + 2 * D * e
        if case["grad"]:  # x, dz in, dx out; squares, two products, rotation, dw
            return {"bytes": 3 * x * e + side + 2 * D * e, "flops": 16 * x}
        return {"bytes": 2 * x * e + side, "flops": 8 * x}
    rows_, keys = case["Sq"] * h * D, sum(lengths(case))
    scores = case["Sq"] * h * D * keys  # one product over all scores: 2 flops each
    if case["grad"]:  # q, o, dout in, dq out; k, v in; dk, dv out over the whole padded length
        b = (4 * B * rows_ + 2 * keys * hk * D + 2 * B * case["Sk"] * hk * D) * e
        return {"bytes": b + 4 * B * h * case["Sq"], "flops": 10 * scores}
    return {"bytes": (2 * B * rows_ + 2 * keys * hk * D) * e, "flops": 4 * scores}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return exact_qk(s) if case["op"] == "qk" else exact_cross(s, case)


def exact_qk(s):
    """z = Rot(w x / sqrt(mean x^2 + eps)) by complex products; its gradient by the
    chain rule, a head at a time."""
    turn = torch.complex(s["cos"].double(), s["sin"].double())
    turn = turn[s["pos"].long()] if s["pos"] is not None else turn[None]
    n = turn.shape[-1]

    def turned(y, by):
        out = y.clone()
        if s["pairs"]:
            first, second = slice(0, 2 * n, 2), slice(1, 2 * n, 2)
        else:
            first, second = slice(0, n), slice(n, 2 * n)
        z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * by
        out[..., first], out[..., second] = z.real, z.imag
        return out

    def one(x, w, dz):
        a, w = x.double(), w.double()
        size = (a.pow(2).sum(-1, keepdim=True) / a.shape[-1] + EPS).sqrt()
        if dz is None:
            return turned(w * a / size, turn), None
        dy = turned(dz.double(), turn.conj())
        inner = (dy * w * a).sum(-1, keepdim=True)
        dx = dy * w / size - a * inner / (a.shape[-1] * size.pow(3))
        return dx, (dy * a / size).sum((0, 1))

    outs = []
    for x, w, d in (("q", "wq", "dq"), ("k", "wk", "dk")):
        got = [one(s[x][:, :, i], s[w], s[d][:, :, i] if s["grad"] else None)
               for i in range(s[x].shape[2])]
        outs.append((torch.stack([a for a, _ in got], 2),
                     torch.stack([b for _, b in got]).sum(0) if s["grad"] else None))
    (a, dwa), (b, dwb) = outs
    return [a, b, dwa, dwb] if s["grad"] else [a, b]


def exact_cross(s, case):
    """o = softmax(q k^T / sqrt(D)) v over each batch's states, and its gradient, a
    batch's head at a time; the gradients of a shared key head are added up."""
    B, S, h, D = s["q"].shape
    hk = s["k"].shape[2]
    kind = dict(dtype=torch.float64, device=DEV)
    o, dq = torch.zeros(B, S, h, D, **kind), torch.zeros(B, S, h, D, **kind)
    dk = torch.zeros(*s["k"].shape, **kind)
    dv = torch.zeros_like(dk)
    for b, n in enumerate(lengths(case)):
        for i in range(h if n else 0):
            j = i // (h // hk)
            q, k, v = s["q"][b, :, i].double(), s["k"][b, :n, j].double(), s["v"][b, :n, j].double()
            p = torch.softmax(q @ k.T / math.sqrt(D), -1)
            o[b, :, i] = p @ v
            if s["grad"]:
                do = s["dout"][b, :, i].double()
                dp = do @ v.T
                dz = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(D)
                dq[b, :, i] = dz @ k
                dk[b, :n, j] += dz.T @ q
                dv[b, :n, j] += p.T @ do
    return [dq, dk, dv] if s["grad"] else o
