"""The fused norm's ring of rows: a wait that runs out ends the threads that wait, with the
status set, and the block's others and the context go on."""
import ctypes
import subprocess
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TIMEOUT = 4  # NABLA_ERR_TIMEOUT


def test_a_row_that_does_not_come(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as build

    so, here = tmp_path / "ring_wait.so", __file__.rsplit("/", 1)[0]
    subprocess.run([build._nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-shared",
                    f"{here}/ring_wait.cu", "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    row = torch.arange(1024, dtype=torch.float32, device=DEV)
    out = torch.zeros(65, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    ptr = [ctypes.c_void_p(t.data_ptr()) for t in (row, out, status)]
    assert lib.ring_wait(*ptr, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 1.0
    assert int(status) == TIMEOUT
    assert float(out[0]) == float(row.sum())
    assert (out[1:33] == 0).all() and (out[33:] == 1).all()
    assert float(row.sum()) == 1023 * 512
