"""Probabilities and verification after a device wait that ran out (what should end it is left
out by a test's own launch, with a limit of milliseconds): a status, nothing read that did not
arrive, and an end."""
import ctypes
import os
import subprocess

import pytest
import torch

import lm_head_gumbel_gb300 as fs
from lm_head_gumbel_gb300 import build as libbuild

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    out = str(tmp_path_factory.mktemp("wait") / "wait_runs_out.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "wait_runs_out.cu")
    subprocess.run([libbuild.nvcc_path(), *libbuild.ARCH_FLAGS, "-O1", "-std=c++17", "-Xcompiler", "-fPIC",
                    f"-I{libbuild.INCLUDE}", f"-I{libbuild.CSRC}", "-shared", "-o", out, src], check=True)
    lib = ctypes.CDLL(out)
    lib.stale_draw.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                               ctypes.c_uint64, ctypes.c_void_p, ctypes.c_void_p]
    lib.half_probs.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                               ctypes.c_uint64, ctypes.c_void_p]
    return lib


@pytest.mark.parametrize("mode", [0, 1, 2])  # from p, from max(p - q, 0), from p without an id
@pytest.mark.parametrize("V", [1, 1024, 5000, 300000])
def test_nothing_is_drawn_from_sums_that_did_not_arrive(lib, V, mode):
    p = torch.full((V,), 1.0 / V, device="cuda")
    q = p * 0.5
    out = torch.full((4,), 77, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    word = lib.stale_draw(p.data_ptr(), q.data_ptr(), V, mode, 2_000_000, out.data_ptr(),
                          torch.cuda.current_stream().cuda_stream)
    drawn, gave_up, segment, kept = out.tolist()
    assert word == 1 and gave_up == 1
    assert drawn == -1
    assert 0 <= segment < -(-V // 1024)
    assert kept == 1


@pytest.mark.parametrize("N,clusters", [(1, 1), (2, 1), (5, 2), (400, 100)])
def test_probabilities_end_after_a_wait_that_ran_out(lib, N, clusters):
    """A status, an end, and nothing outside the rows is written."""
    x = torch.randn((N, 8000), device="cuda")
    out = torch.full((N + 2, 8000), 77.0, device="cuda")
    torch.cuda.synchronize()
    word = lib.half_probs(x.data_ptr(), out[1:].data_ptr(), N, clusters, 2_000_000,
                          torch.cuda.current_stream().cuda_stream)
    assert word == 1
    assert bool((out[0] == 77.0).all()) and bool((out[N + 1] == 77.0).all())
    # The device is as it was.
    assert torch.allclose(fs.fs_probs(x), torch.softmax(x, 1), rtol=1e-5)
    assert fs.fs_last_device_error() == (fs.FS_OK, 0)
