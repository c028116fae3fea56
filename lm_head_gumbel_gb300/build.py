"""Build the CUDA library ``libfs.so`` in-tree with nvcc, for sm_103a only, and
the argument-marshalling module ``_marshal.so`` with the host compiler."""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBRARY = os.path.join(PKG, "libfs.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
MARSHAL_DEPENDS = [os.path.join(CSRC, "fs_marshal.cpp")] + [
    os.path.join(INCLUDE, f) for f in ("fs_sample.h", "fs_vocab.h",
                                                  "fs_speculate.h")]
SOURCES = [os.path.join(CSRC, f) for f in ("fs_sample.cu", "fs_merge.cu", "fs_logprobs.cu",
                                          "fs_embed.cu", "fs_fp8.cu", "fs_verify.cu")]
DEPENDS = SOURCES + [os.path.join(CSRC, f) for f in ("fs_kernels.cuh", "fs_ptx.cuh",
                                                    "fs_noise.cuh", "fs_contract.cuh",
                                                    "fs_pieces.h")] + [
    os.path.join(INCLUDE, f) for f in ("fs_sample.h", "fs_vocab.h",
                                                  "fs_speculate.h")]

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfs.so")
    return cand


def command(output: str = LIBRARY, extra=()) -> list:
    return [nvcc_path(), *ARCH_FLAGS, "--threads", "0", "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
            "-shared", f"-I{INCLUDE}", *extra, "-o", output, *SOURCES]


def marshal_command(output: str = MARSHAL) -> list:
    import torch
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            f'-DFS_TORCH_VERSION="{torch.__version__}"', f"-I{INCLUDE}",
            f"-I{home}/include", f"-I{home}/include/torch/csrc/api/include",
            f"-I{sysconfig.get_path('include')}", f"-I{cuda}/include", "-o", output,
            MARSHAL_DEPENDS[0], f"-L{home}/lib", "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-ltorch_cuda", "-lc10", "-lc10_cuda"]


def marshal_depends() -> list:
    """The module's sources, and torch: one installed behind the build is not the one
    that the module was built for."""
    import torch
    return MARSHAL_DEPENDS + [torch.version.__file__]


def up_to_date(output: str = LIBRARY, depends=tuple(DEPENDS)) -> bool:
    if not os.path.exists(output):
        return False
    t = os.path.getmtime(output)
    return all(os.path.getmtime(f) <= t for f in depends)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libfs.so and _marshal.so, each unless it is newer than every
    source it depends on; both at the same time."""
    jobs = []
    if force or not up_to_date():
        tmp = LIBRARY + f".tmp{os.getpid()}"
        jobs.append((LIBRARY, tmp, command(tmp, ["-Xptxas", "-v"] if verbose else [])))
    if force or not up_to_date(MARSHAL, marshal_depends()):
        tmp = MARSHAL + f".tmp{os.getpid()}"
        jobs.append((MARSHAL, tmp, marshal_command(tmp)))
    running = [(job, subprocess.Popen(job[2], stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                      text=True)) for job in jobs]
    done = [(job, proc.communicate()[0], proc.returncode) for job, proc in running]
    for (output, tmp, cmd), text, status in done:
        if status != 0:
            raise RuntimeError(f"{os.path.basename(output)} build failed:\n{' '.join(cmd)}\n{text}")
        os.replace(tmp, output)
        if verbose:
            print(text)
    return LIBRARY


if __name__ == "__main__":
    print(build(force=True, verbose=True))
