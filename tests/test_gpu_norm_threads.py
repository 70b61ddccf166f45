"""The gated sum with norm called by several host threads at once, at two widths that one
compiled kernel serves with different amounts of shared memory: no call is refused, and the
results are those of one thread."""
import ctypes
import pathlib
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
HERE = pathlib.Path(__file__).resolve().parent
THREADS, TIMES, S = 6, 2000, 320  # half of the threads call each width
vp = ctypes.c_void_p


class NormCall(ctypes.Structure):  # as in norm_threads.cpp
    _fields_ = [("ins", vp * 4), ("outs", vp * 2), ("weight", vp), ("post_weight", vp),
                ("dweight", vp), ("dpost_weight", vp), ("workspace", vp),
                ("ws_bytes", ctypes.c_size_t), ("stream", vp), ("S", ctypes.c_int),
                ("C", ctypes.c_int), ("dt", ctypes.c_int), ("grad", ctypes.c_int)]


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


@pytest.fixture(scope="module")
def threads(tmp_path_factory):
    """norm_threads(calls, times) over the C entry points."""
    so = tmp_path_factory.mktemp("threads") / "norm_threads.so"
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-pthread",
                    f"-I{HERE.parent / 'include'}", str(HERE / "norm_threads.cpp"), "-o", str(so)],
                   check=True)
    return ctypes.CDLL(str(so)).norm_threads


class Program:
    """A thread's call and its arrays, on a stream of its own."""

    def __init__(self, nabla, grad, C, weights, dtype, seed):
        g = torch.Generator().manual_seed(seed)
        self.ins = [torch.randn(1, S, C, generator=g).to(dtype).to(DEV) for _ in range(4)]
        w = torch.rand(2, C, generator=g).to(DEV) + 0.5 if weights else None
        self.outs = [torch.empty_like(self.ins[0]) for _ in range(2)]
        self.small = torch.zeros(2, C, device=DEV)
        self.ws = torch.empty(nabla.nabla_block_norm_bwd_workspace_bytes(1, S, C),
                              dtype=torch.uint8, device=DEV)
        self.stream = torch.cuda.Stream()
        self.stream.wait_stream(torch.cuda.current_stream())
        self.keep = w

        def at(t, i, on=True):
            return t[i].data_ptr() if t is not None and on else None

        self.call = NormCall(
            (vp * 4)(*(t.data_ptr() for t in self.ins)),
            (vp * 2)(*(t.data_ptr() for t in self.outs)),
            at(w, 0), at(w, 1), at(self.small, 0, weights and grad),
            at(self.small, 1, weights and grad), self.ws.data_ptr(), self.ws.numel(),
            self.stream.cuda_stream, S, C,
            nabla.NABLA_BF16 if dtype == torch.bfloat16 else nabla.NABLA_F32, int(grad))

    def results(self):
        return [t.clone() for t in (*self.outs, self.small)]


@pytest.mark.parametrize("grad,dtype,one,other", [  # (columns, weights)
    (False, torch.bfloat16, (5120, True), (8192, True)),
    (False, torch.float32, (4104, False), (8192, False)),
    (True, torch.bfloat16, (6400, False), (8192, True)),
    (True, torch.float32, (640, True), (2048, True)),
])
def test_threads_of_different_widths(nabla, threads, grad, dtype, one, other):
    lib = nabla.load()
    fns = [ctypes.cast(f, vp) for f in (lib.nabla_block_norm, lib.nabla_block_norm_bwd)]
    programs = [Program(nabla, grad, *(one, other)[i % 2], dtype, seed=i) for i in range(THREADS)]
    want = []
    for p in programs:
        assert threads(*fns, ctypes.byref(p.call), 1, 1) == 0
        torch.cuda.synchronize()
        want.append(p.results())
    calls = (NormCall * THREADS)(*(p.call for p in programs))
    error = threads(*fns, calls, THREADS, TIMES)
    torch.cuda.synchronize()
    assert error == 0
    for p, ref in zip(programs, want):
        assert all(torch.equal(a, b) for a, b in zip(p.results(), ref))
    assert nabla.nabla_get_last_device_status() == 0
