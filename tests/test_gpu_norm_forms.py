"""The gated sum with norm in every form that its launch rules choose by type, columns, tokens,
branch and modulation rows, with several rows a warp and the backward's ring filled more than
twice, against 64 bits (norm_plain: tolerances, derived there)."""
import ctypes

import numpy as np
import pytest
import torch

import norm_plain as plain
from oracle import nabla_oracle as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SMS = 152


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


def case(C, T, each, dtype, norm, branch, **kw):
    """About T tokens, `each` of them a row of the modulations (0: a batch of two thirds)."""
    if not each:
        return plain.Inputs(3, -(-T // 3), C, TYPES[dtype], norm, branch, 1, seed=C, **kw)
    rows = -(-T // each)
    return plain.Inputs(1, rows * each, C, TYPES[dtype], norm, branch, rows, seed=C, **kw)


def check_forward(nabla, c):
    s, y = nabla.nabla_block_norm(c.x, c.u, **c.args())
    want = plain.forward(c)
    if c.u is not None:
        plain.check("s", s, *want["s"])
    plain.check("y", y, *want["y"])
    assert nabla.nabla_get_last_device_status() == 0
    return s


# Columns, and the tokens from which on a team has two rows and more: 152 SMs hold `blocks` of
# `teams` rows each.
#         C     blocks, teams
FORWARD = {
    "bf16": [(40, 4, 32), (104, 4, 16), (200, 4, 8),              # 8, 16, 32 lanes a row
             (456, 3, 8), (1000, 2, 8), (1320, 2, 8), (2040, 2, 8),  # 2, 4, 6, 8 vectors a lane
             (2312, 3, 1), (4000, 3, 1), (4408, 3, 1), (8192, 3, 1)],  # two warps a row, and more
    "f32": [(40, 4, 32), (104, 4, 16), (200, 4, 8), (456, 3, 8), (1000, 2, 8),
            (1504, 4, 1), (4096, 4, 1), (8192, 2, 1)],
}


@pytest.mark.parametrize("branch", ["", "u", "layer"])
@pytest.mark.parametrize("each", [3, 13])  # too few to lay the modulations out, and enough
@pytest.mark.parametrize("dtype,C,blocks,teams", [(d, *f) for d in FORWARD for f in FORWARD[d]])
def test_forward(nabla, dtype, C, blocks, teams, each, branch):
    norm = "rms" if branch == "layer" else "layer"
    check_forward(nabla, case(C, SMS * blocks * (2 * teams + 1) + 5, each, dtype, norm, branch))


@pytest.mark.parametrize("branch", ["", "rms"])
@pytest.mark.parametrize("C,T", [(520, 500), (2312, 400), (4096, 608), (4408, 304), (8192, 60)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_of_few_rows(nabla, dtype, C, T, branch):
    check_forward(nabla, case(C, T, 4, dtype, "layer", branch))


# Columns, teams on the 152 SMs, and rows of each team: a ring's four stages filled more than
# twice; teams of a warp or less have none.
BACKWARD = {
    "bf16": [(40, 64, 4), (104, 32, 4), (200, 16, 4),        # 8, 16, 32 lanes a row
             (264, 8, 9), (1504, 2, 9), (2048, 2, 10),         # a block a row
             (2152, 2, 9), (2560, 2, 11),                      # two of them on an SM
             (2600, 1, 9), (4096, 1, 10),
             (4104, 1, 9), (6144, 1, 9), (6400, 1, 9), (8192, 1, 9)],  # two vectors a thread
    "f32": [(40, 64, 4), (104, 32, 4), (200, 16, 4), (264, 8, 9), (1112, 3, 9), (2312, 1, 10),
            (4096, 1, 9), (4104, 1, 9), (6144, 1, 9), (6400, 1, 5), (8192, 1, 5)],
}


@pytest.mark.parametrize("branch,each,weights", [
    ("", 7, False), ("u", 0, True),  # rows of the modulations that cross runs, and long ones
    ("layer", 7, True), ("rms", 0, False), ("rms", 3, True),
])
@pytest.mark.parametrize("dtype,C,teams,L", [(d, *f) for d in BACKWARD for f in BACKWARD[d]])
def test_backward(nabla, dtype, C, teams, L, branch, each, weights):
    norm = "rms" if branch == "layer" else "layer"
    c = case(C, SMS * teams * L - 3 * teams, each, dtype, norm, branch, weights=weights,
             mtype=torch.bfloat16 if each == 3 else torch.float32)
    s = (c.x.float() + 0.5 * c.u.float()).to(c.x.dtype) if branch else c.x
    got = nabla.nabla_block_norm_bwd(s, c.u, c.dsum, c.dy, **c.args())
    assert nabla.nabla_get_last_device_status() == 0
    want = plain.backward(c, s)
    for name, t in zip(plain.GRADS, got):
        assert (t is None) == (name not in want), name
        if t is not None:
            plain.check(name, t, *want[name])
    again = nabla.nabla_block_norm_bwd(s, c.u, c.dsum, c.dy, **c.args())
    assert all(a is b or torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("C", [40, 200, 1504, 4104])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_of_an_absent_branch_output(nabla, dtype, C):
    """Through the C entry point, du = rs gate ds without u (which only its norm and its gate's
    gradient need), and dx beside it or not."""
    T = 700
    c = case(C, T, 0, dtype, "layer", "u", weights=False)
    S = c.x.shape[1]
    lib, vp = nabla.load(), ctypes.c_void_p
    outs = torch.empty_like(c.x), torch.empty_like(c.x)

    def call(dx):
        code = nabla.NABLA_BF16 if dtype == "bf16" else nabla.NABLA_F32
        gate, scale = c.gate.contiguous(), c.scale.contiguous()
        return lib.nabla_block_norm_bwd(
            c.x.data_ptr(), None, None, None, c.dsum.data_ptr(), None, c.dy.data_ptr(), None, code,
            3, S, C, 2, 0, None, None, nabla.NABLA_F32, gate.data_ptr(), C, scale.data_ptr(), C,
            nabla.NABLA_F32, 3, c.rs, plain.EPS, dx, None, outs[1].data_ptr(), None, None, None,
            None, None, None, None, 0, vp(torch.cuda.current_stream().cuda_stream))

    want = plain.backward(c, c.x)
    for dx in (outs[0].data_ptr(), None):
        outs[0].zero_(), outs[1].zero_()
        assert call(dx) == 0
        assert nabla.nabla_get_last_device_status() == 0
        plain.check("du", outs[1], *want["du"])
        if dx:
            plain.check("dx", outs[0], *want["dx"])
        else:
            assert (outs[0] == 0).all()


@pytest.mark.parametrize("norm,branch", [("layer", "rms"), ("rms", "layer"), ("rms", "u")])
def test_gradients_along_directions_against_differences(nabla, norm, branch):
    """<grad, d> of whole tensors along random directions against central differences of the
    oracle's forward in 64 bits.  Room: the kernels' (norm_plain, times |d|), and the change from
    one step to twice that, three times what the third derivative makes of it.  No gradient could
    be missing: the room is less than an eighth of what is compared."""
    c = plain.Inputs(2, 3, 72, torch.float32, norm, branch, 3, rs=1.0, seed=5)
    s = plain.forward(c)["s"][0].float()
    got = nabla.nabla_block_norm_bwd(s, c.u, c.dsum, c.dy, **c.args())
    sizes = plain.backward(c, s)
    names = dict(zip(plain.GRADS, ("x", "u", "gate", "scale", "shift", "w", "pw")))
    at = {k: getattr(c, k) for k in names.values()}
    at = {k: None if t is None else t.double().cpu().numpy() for k, t in at.items()}
    dsum, dy = c.dsum.double().cpu().numpy(), c.dy.double().cpu().numpy()

    def loss(t):
        s, y = O.block_norm(t["x"], t["u"], t["gate"], t["scale"], t["shift"], t["w"], t["pw"],
                            c.norm, c.post, c.rs, plain.EPS)
        return float((s * dsum).sum() + (y * dy).sum())

    for i, (grad, k) in enumerate(names.items()):
        if at[k] is None:
            continue
        g = got[i].double().cpu().numpy()
        # a random direction, leaning towards the gradient so that what is compared is not small
        d = np.random.default_rng(i).standard_normal(g.shape)
        value, size = (t.cpu().numpy() for t in sizes[grad])
        d += value / np.abs(value).mean()

        def difference(step):
            hi, lo = ({**at, k: at[k] + by * d} for by in (step, -step))
            return (loss(hi) - loss(lo)) / (2 * step)

        near, far = difference(2.0 ** -10), difference(2.0 ** -9)
        room = 2.0 ** -24 * np.abs(value) + 2.0 ** plain.TOLERANCE[grad] * size
        room = (np.abs(d) * room).sum() + abs(near - far)
        assert abs((g * d).sum() - near) <= room, grad
        assert room < abs(near) / 8, grad
