"""Overlapping calls behind a kernel that lets its dependents start long before it writes."""
import ctypes
import os
import subprocess

import pytest
import torch

import lm_head_gumbel_gb300 as fs
from gpu_cases import assert_no_device_error
from lm_head_gumbel_gb300 import build as libbuild

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fs.load_library()
    yield
    assert_no_device_error()


@pytest.fixture(scope="module")
def late_copy(tmp_path_factory):
    """to.copy_(source), `ms` after its dependents may start; both contiguous, of one size."""
    out = str(tmp_path_factory.mktemp("dependents") / "dependents.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "dependents.cu")
    subprocess.run([libbuild.nvcc_path(), *libbuild.ARCH_FLAGS, "-O2", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-shared", "-o", out, src], check=True)
    lib = ctypes.CDLL(out)
    lib.late_copy.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint64,
                              ctypes.c_void_p]

    def run(to, source, ms):
        assert to.is_contiguous() and source.is_contiguous() and to.nbytes == source.nbytes
        assert lib.late_copy(source.data_ptr(), to.data_ptr(), to.nbytes, int(ms * 1e6),
                             torch.cuda.current_stream().cuda_stream) == 0
    return run


def head(V, d, seed):
    gen = torch.Generator().manual_seed(seed)
    return fs.fs_quantize((torch.randn((V, d), generator=gen) / d ** 0.5).bfloat16().cuda(), 128)


def hidden(M, d, seed):
    gen = torch.Generator().manual_seed(seed)
    return fs.fs_quantize(torch.randn((M, d), generator=gen).bfloat16().cuda())


@pytest.mark.parametrize("M", [3, 200])
@pytest.mark.parametrize("flag", [False, True])
def test_product_starts_nothing_before_its_predecessor_has_ended(late_copy, flag, M):
    """A kernel writes a head; a product with another head, with and without the flag; an
    overlapping product with the first head, whose kernel before is the other product."""
    d = 512
    a, b = hidden(M, d, 1), hidden(4, d, 2)
    w, other = head(3000, d, 3), head(200, d, 4)
    want, want_other = fs.fs_matmul_fp8(*a, *w), fs.fs_matmul_fp8(*b, *other)
    written = torch.zeros_like(w.values)
    for ms in (0.1, 1.0, 20.0):
        written.zero_()
        torch.cuda.synchronize()
        late_copy(written, w.values, ms)
        got_other = fs.fs_matmul_fp8(*b, *other, overlap_previous=flag)
        got = fs.fs_matmul_fp8(*a, written, w.scale, overlap_previous=True)
        torch.cuda.synchronize()
        assert torch.equal(got_other, want_other) and torch.equal(got, want)


@pytest.mark.parametrize("M", [3, 200])
def test_product_waits_as_long_as_its_predecessor_takes(late_copy, M):
    """The limit of a device wait (2 s) is not for the kernel that makes A."""
    a, w = hidden(M, 512, 1), head(3000, 512, 3)
    want = fs.fs_matmul_fp8(*a, *w)
    A = torch.zeros_like(a.values)
    torch.cuda.synchronize()
    late_copy(A, a.values, 2600)
    got = fs.fs_matmul_fp8(A, a.scale, *w, overlap_previous=True)
    torch.cuda.synchronize()
    assert fs.fs_last_device_error() == (fs.FS_OK, 0)
    assert torch.equal(got, want)


@pytest.mark.parametrize("B", [4, 200])
@pytest.mark.parametrize("call", ["sample", "logprobs"])
def test_sampler_and_logprobs_wait_as_long_as_their_predecessor_takes(late_copy, call, B):
    """The same of the kernel that makes H, for single CTAs and pairs."""
    gen = torch.Generator().manual_seed(B)
    H = torch.randn((B, 256), generator=gen).bfloat16().cuda()
    W = (torch.randn((3000, 256), generator=gen) * 0.1).bfloat16().cuda()
    ids = torch.randint(0, 3000, (B,), generator=gen).cuda()

    def run(h, overlap):
        if call == "sample":
            return fs.fs_sample(h, W, seed=5, offset=1, overlap_previous=overlap)
        return fs.fs_logprobs(h, W, ids, overlap_previous=overlap).logp

    want = run(H, False)
    late = torch.zeros_like(H)
    torch.cuda.synchronize()
    late_copy(late, H, 2600)
    got = run(late, True)
    torch.cuda.synchronize()
    assert fs.fs_last_device_error() == (fs.FS_OK, 0)
    assert torch.equal(got, want)
