"""Calls on several streams that allocate their own scratch and outputs give the bits of
the same calls one after the other, while the current stream allocates and writes memory
of the same sizes, and outputs are dropped as soon as they have been copied."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


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


def operators(N, seed, dtype):
    """Calls that take a stream; their inputs are made here."""
    g = torch.Generator().manual_seed(seed)

    def draw(*shape):
        return torch.randn(*shape, generator=g).to(dtype).to(DEV)

    q, k, v, dout = (draw(1, 2048, 2, 64) for _ in range(4))
    ek, ev, w = draw(1, 300, 2, 64), draw(1, 300, 2, 64), draw(64)
    sq, sk, sv = draw(2, 1, 6, 128), draw(2, 3000, 2, 128), draw(2, 3000, 2, 128)
    sta = torch.ones(32, 32, dtype=torch.uint8, device=DEV).tril().triu(-2)
    nb, inds = N.nabla_build_mask(q, k, sta, 0.6)
    o1, lse1 = N.nabla_attn_fwd_lse(q, k, v, nb, inds)
    o, lse = N.nabla_cross_attn_fwd_lse(q, ek, ev)
    torch.cuda.synchronize()
    return [
        lambda s: (N.nabla_build_mask(q, k, sta, 0.6, stream=s)[0],),
        lambda s: N.nabla_attn_bwd(q, k, v, o1, dout, nb, inds, lse=lse1, stream=s),
        lambda s: N.nabla_qk_norm_rope_bwd(q, k, w, w, dout, v, stream=s),
        lambda s: N.nabla_cross_attn_fwd_lse(sq, sk, sv, stream=s),
        lambda s: N.nabla_cross_attn_bwd(q, ek, ev, o, lse, dout, stream=s),
    ]


def copies(outs):
    return [t.clone() for t in outs]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("handles", [False, True], ids=["objects", "handles"])
def test_overlapping_calls_keep_their_memory(nabla, dtype, handles):
    sides = [torch.cuda.Stream() for _ in range(3)]
    ops = [operators(nabla, i, dtype) for i in range(3)]
    want = [[copies(f(None)) for f in fs] for fs in ops]
    torch.cuda.synchronize()
    sizes = sorted({t.numel() * t.element_size() for f in want[0] for t in f} |
                   {nabla.nabla_cross_attn_bwd_workspace_bytes(dtype, 1, 2048, 300, 2, 2, 64),
                    nabla.nabla_cross_attn_fwd_workspace_bytes(dtype, 2, 1, 3000, 6, 2, 128),
                    nabla.nabla_qk_norm_rope_bwd_workspace_bytes(64)})
    got = [[[] for _ in fs] for fs in ops]
    for _ in range(6):
        for i in range(len(ops[0])):
            for j, side in enumerate(sides):
                outs = ops[j][i](side.cuda_stream if handles else side)
                with torch.cuda.stream(side):
                    got[j][i].append(copies(outs))
                del outs
                for n in sizes:
                    torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0xff)
    torch.cuda.synchronize()
    for j in range(3):
        for ref, runs in zip(want[j], got[j]):
            for run in runs:
                assert all(torch.equal(a, b) for a, b in zip(ref, run))
    assert nabla.nabla_get_last_device_status() == 0


def test_outputs_outlive_their_last_use_on_the_current_stream(nabla):
    """An output of a call on another stream, read on the current one and dropped there
    while that read is pending, is not handed to the next call on the other stream."""
    f, g = operators(nabla, 5, torch.bfloat16)[4], operators(nabla, 6, torch.bfloat16)[4]
    want, side = copies(f(None)), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        outs = f(side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(4_000_000)  # a few milliseconds of pending work
        read = copies(outs)
        del outs
        for _ in range(3):
            g(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(read, want))


def test_default_stream_from_another_one(nabla):
    """The default stream by number, and by its other name, while another is current."""
    f, side = operators(nabla, 7, torch.bfloat16)[4], torch.cuda.Stream()
    want = copies(f(None))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = [f(0), f(1), f(torch.cuda.default_stream())]
    torch.cuda.synchronize()
    for outs in got:
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("op", range(1, 5), ids=["attn_bwd", "qk_norm_bwd", "cross_lse",
                                                 "cross_bwd"])
def test_calls_on_a_forked_stream_are_captured(nabla, op):
    """Two calls on a stream forked from the capturing one, their scratch and outputs
    allocated in the capture and the first's outputs dropped there."""
    f, g = (operators(nabla, i, torch.bfloat16)[op] for i in (8, 9))
    want = [copies(x(None)) for x in (f, g)]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        current = torch.cuda.current_stream()
        side.wait_stream(current)
        outs = f(side)
        current.wait_stream(side)
        first = copies(outs)
        del outs
        second = g(side)
        current.wait_stream(side)
    for _ in range(3):
        for t in first + list(second):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in ((first, want[0]), (second, want[1])):
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
