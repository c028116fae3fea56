"""The operators of include/fs_speculate.h without a GPU: the library exports them,
the binding's structures match the header's and bad arguments are rejected on the
host before any device work."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fs_speculate.h")
INVALID = 1
UNSUPPORTED = 2  # no device


@pytest.fixture(scope="module")
def lib():
    from lm_head_gumbel_gb300 import build as libbuild
    try:
        libbuild.build()
    except RuntimeError as e:  # no nvcc on this machine
        pytest.skip(str(e))
    import lm_head_gumbel_gb300 as fs
    return fs.load_library()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(fs_[a-z_0-9]+)\s*\(", text)))
    assert names == ["fs_matmul_fp8", "fs_probs", "fs_quantize", "fs_verify"]
    for name in names:
        assert hasattr(lib, name), name


@pytest.mark.parametrize("struct,mirror", [("fs_matmul_fp8_args", "FsMatmulFp8Args"),
                                           ("fs_probs_args", "FsProbsArgs"),
                                           ("fs_verify_args", "FsVerifyArgs")])
def test_structures_match_the_header(tmp_path, struct, mirror):
    """Field offsets and size of the ctypes mirror against the C compiler's."""
    import lm_head_gumbel_gb300 as fs
    cls = getattr(fs, mirror)
    fields = [f[0] for f in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "fs_speculate.h"\n'
                   "int main(void){"
                   + "".join(f'printf("%zu ", offsetof({struct}, {f}));' for f in fields)
                   + f'printf("%zu\\n", sizeof({struct}));return 0;}}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == [getattr(cls, f).offset for f in fields] + [ctypes.sizeof(cls)]


def _quantize(lib, **kw):
    a = dict(x=0x10000, N=4, d=256, ldx=256, dtype=0, block=1, values=0x20000, ldv=256,
             scale=0x30000, lds=2)
    a.update(kw)
    return lib.fs_quantize(a["x"], a["N"], a["d"], a["ldx"], a["dtype"], a["block"], a["values"],
                           a["ldv"], a["scale"], a["lds"], None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(values=None), dict(scale=None), dict(N=-1), dict(N=2**31 - 128), dict(d=0),
    dict(d=2**31 - 1, ldx=2**31, ldv=2**31), dict(ldx=255), dict(ldv=255), dict(lds=1),
    dict(dtype=2), dict(dtype=-1), dict(block=0), dict(block=64), dict(x=0x10001),
    dict(x=0x10002, dtype=1), dict(scale=0x30002), dict(N=300, block=128, lds=1),
    dict(N=2**30, d=2**20, ldx=2**20, ldv=2**20, lds=2**13),
])
def test_quantize_bad_arguments(lib, kw):
    assert _quantize(lib, **kw) == INVALID


def test_quantize_of_nothing(lib):
    assert _quantize(lib, N=0, x=None, values=None, scale=None) == 0


def _matmul(**kw):
    import lm_head_gumbel_gb300 as fs
    base = dict(A=0x10000, a_scale=0x20000, W=0x30000, w_scale=0x40000, M=4, d=300, V=1000,
                lda=304, lda_scale=3, ldw=304, ldw_scale=3, out=0x50000, ldo=1000, out_dtype=0)
    base.update(kw)
    return fs.FsMatmulFp8Args(**base)


@pytest.mark.parametrize("kw", [
    dict(A=None), dict(a_scale=None), dict(W=None), dict(w_scale=None), dict(out=None),
    dict(M=-1), dict(M=2**31 - 1), dict(d=0), dict(V=0), dict(V=2**31 - 1), dict(lda=299),
    dict(lda=300), dict(lda=308), dict(ldw=288), dict(ldw=305), dict(lda_scale=2),
    dict(ldw_scale=2), dict(ldo=999), dict(out_dtype=2), dict(A=0x10008), dict(W=0x30001),
    dict(a_scale=0x20002), dict(w_scale=0x40001), dict(out=0x50001), dict(out=0x50002, out_dtype=1),
    dict(flags=2), dict(flags=0x80000000),
    dict(M=2**30, V=2**30, ldo=2**30),  # 32-bit counts of tiles
])
def test_matmul_bad_arguments(lib, kw):
    assert lib.fs_matmul_fp8(ctypes.byref(_matmul(**kw)), None) == INVALID


def _probs(**kw):
    import lm_head_gumbel_gb300 as fs
    base = dict(logits=0x10000, N=4, V=1000, ldl=1000, out=0x90000, ldo=1000, dtype=0, out_dtype=1)
    base.update(kw)
    return fs.FsProbsArgs(**base)


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(out=None), dict(N=-1), dict(N=2**31), dict(V=0), dict(V=2**31 - 65536),
    dict(ldl=999), dict(ldo=999), dict(dtype=2), dict(out_dtype=-1), dict(logits=0x10001),
    dict(logits=0x10002, dtype=1), dict(out=0x90002), dict(temperature=0x20002),
    dict(vocab_mask=0x30000, mask_ld=31), dict(vocab_mask=0x30002, mask_ld=32),
    dict(out=0x10000),                                   # in place, but of another type
    dict(out=0x10000, out_dtype=0, ldo=1008),            # and with another stride
])
def test_probs_bad_arguments(lib, kw):
    assert lib.fs_probs(ctypes.byref(_probs(**kw)), None) == INVALID


def _verify(**kw):
    import lm_head_gumbel_gb300 as fs
    base = dict(p=0x10000, q=0x20000, draft_ids=0x30000, u=0x40000, B=4, K=3, V=1000, p_seq=4000,
                p_pos=1000, q_seq=3000, q_pos=1000, ld_ids=3, ldu=4, out_ids=0x50000, ld_out=4,
                out_accepted=0x60000, dtype=1)
    base.update(kw)
    return fs.FsVerifyArgs(**base)


@pytest.mark.parametrize("kw", [
    dict(p=None), dict(u=None), dict(out_ids=None), dict(draft_ids=None), dict(B=-1),
    dict(B=2**24), dict(K=-1), dict(K=1025, ld_ids=2000, ldu=2000, ld_out=2000), dict(V=0),
    dict(V=2**31 - 65536), dict(p=0x10002), dict(q=0x20001), dict(draft_ids=0x30004),
    dict(u=0x40002), dict(out_ids=0x50004), dict(out_accepted=0x60004), dict(ld_ids=2), dict(ldu=3),
    dict(ld_out=3), dict(p_seq=-1), dict(q_pos=-8), dict(dtype=2),
])
def test_verify_bad_arguments(lib, kw):
    assert lib.fs_verify(ctypes.byref(_verify(**kw)), None) == INVALID


def test_nothing_to_do_and_null_arguments(lib):
    assert lib.fs_matmul_fp8(ctypes.byref(_matmul(M=0, A=None, out=None)), None) == 0
    assert lib.fs_probs(ctypes.byref(_probs(N=0, logits=None, out=None)), None) == 0
    assert lib.fs_verify(ctypes.byref(_verify(B=0, p=None, out_ids=None)), None) == 0
    assert lib.fs_matmul_fp8(None, None) == INVALID
    assert lib.fs_probs(None, None) == INVALID
    assert lib.fs_verify(None, None) == INVALID


def test_the_module_refuses_what_the_library_cannot_see(lib):
    """Types, shapes and devices; CPU tensors never reach the library."""
    import lm_head_gumbel_gb300 as fs
    import torch
    bad = [
        lambda: fs.fs_quantize(torch.zeros(4, 8)),                       # not on a GPU
        lambda: fs.fs_quantize([1.0]),
        lambda: fs.fs_quantize(torch.zeros(4, 8, dtype=torch.float16)),
        lambda: fs.fs_matmul_fp8(*[torch.zeros(4, 16)] * 4),
        lambda: fs.fs_matmul_fp8(*[torch.zeros(4, 16)] * 4, out_dtype=torch.float16),
        lambda: fs.fs_probs(torch.zeros(4, 8)),
        lambda: fs.fs_probs(torch.zeros(4, 8), out=torch.zeros(4, 8), out_dtype=torch.bfloat16),
        lambda: fs.fs_verify(torch.zeros(2, 3, 8), torch.zeros(2, 2), torch.zeros(2, 3)),
    ]
    for call in bad:
        with pytest.raises(fs.FsError) as e:
            call()
        assert e.value.status == INVALID


@pytest.mark.parametrize("V,ld", [(1, 1), (1000, 1000), (300000, 300000)])
def test_probs_takes_every_documented_number_of_rows(lib, V, ld):
    """0 <= N < 2^28: one row more is refused, as an argument; the largest number is not."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the pointers are made up")
    for N, status in ((2**28, INVALID), (2**28 - 1, UNSUPPORTED), (2**27, UNSUPPORTED)):
        assert lib.fs_probs(ctypes.byref(_probs(N=N, V=V, ldl=ld, ldo=ld)), None) == status


PIECES = r"""
#include <cstdio>
#include "fs_pieces.h"
using namespace fs::fp8;
// Every piece that is read whole, of every small matrix, ends inside it: N rows of d elements,
// ldx apart, have (N - 1) ldx + d.
int main() {
  int bad = 0, whole = 0;
  for (int size = 2; size <= 4; size += 2)
    for (int N = 1; N <= 5; ++N)
      for (int d = 1; d <= 40; ++d)
        for (int ldx = d; ldx <= d + 20; ++ldx) {
          if (!whole_pieces(0x1000, N, N > 1 ? ldx : 0, size)) continue;
          for (int row = 0; row < N; ++row)
            for (int col = 0; col < d; col += kPiece) {
              if (!whole_piece(d - col, row == N - 1)) continue;
              ++whole;
              if (row * ldx + col + kPiece > (N - 1) * ldx + d) {
                if (bad++ < 5) printf("size %d: [%d, %d], stride %d, row %d, column %d\n", size, N, d, ldx, row, col);
              }
            }
        }
  if (whole == 0) printf("no piece\n");
  return bad != 0 || whole == 0;
}
"""


def test_quantisation_reads_inside_its_matrix(tmp_path):
    src, exe = tmp_path / "pieces.cpp", tmp_path / "pieces"
    src.write_text(PIECES)
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "lm_head_gumbel_gb300", "csrc"),
                    str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
