"""The operators of include/fs_vocab.h without a GPU: the library exports them,
the binding's structures match the header's, sizes come out as documented and
bad arguments are rejected on the host before any device work."""
import ctypes
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fs_vocab.h")
INVALID, WORKSPACE = 1, 5


@pytest.fixture(scope="module")
def lib():
    from lm_head_gumbel_gb300 import build as libbuild
    try:
        libbuild.build()
    except RuntimeError as e:  # no nvcc on this machine
        pytest.skip(str(e))
    import lm_head_gumbel_gb300 as fs
    return fs.load_library()


def declared_functions():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(fs_[a-z_0-9]+)\s*\(", text)))


def test_every_declared_symbol_is_exported(lib):
    names = declared_functions()
    assert names == ["fs_embed", "fs_embed_grad", "fs_embed_grad_workspace_size", "fs_logprobs",
                     "fs_logprobs_grad", "fs_logprobs_grad_workspace_size",
                     "fs_logprobs_workspace_size"]
    for name in names:
        assert hasattr(lib, name), name


@pytest.mark.parametrize("struct,mirror", [("fs_logprobs_args", "FsLogprobsArgs"),
                                           ("fs_logprobs_grad_args", "FsLogprobsGradArgs")])
def test_structures_match_the_header(tmp_path, struct, mirror):
    """Field offsets and size of the ctypes mirror against the C compiler's."""
    import lm_head_gumbel_gb300 as fs
    cls = getattr(fs, mirror)
    fields = [f[0] for f in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "fs_vocab.h"\nint main(void){'
                   + "".join(f'printf("%zu ", offsetof({struct}, {f}));' for f in fields)
                   + f'printf("%zu\\n", sizeof({struct}));return 0;}}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                          check=True).stdout.split()]
    assert got == [getattr(cls, f).offset for f in fields] + [ctypes.sizeof(cls)]


def test_workspace_sizes(lib):
    import lm_head_gumbel_gb300 as fs
    for bad in ((0, 100, 0), (65536, 100, 0), (4, 0, 0), (4, 2**31, 0), (4, 100, -1),
                (4, 100, 21)):
        assert fs.fs_logprobs_workspace_size(*bad) == 0
    # Small vocabularies: units of 64 ids, 2 slots each; a slot is 16 bytes and its two lists.
    assert fs.fs_logprobs_workspace_size(1, 100, 0) == 256
    assert fs.fs_logprobs_workspace_size(64, 256, 4) == 64 * 8 * 16 + 2 * 64 * 8 * 8 * 4
    # 594 vocabulary blocks: a group per SM for up to 128 rows.
    assert fs.fs_logprobs_workspace_size(128, 151936, 20) == 128 * 304 * (16 + 24 * 8)
    # 4 pair blocks of 256 rows: 19 groups of 4 pairs.
    assert fs.fs_logprobs_workspace_size(1024, 151936, 5) == 1024 * 38 * (16 + 16 * 8)
    # Above 5 pair blocks the rows go in several launches, each reusing it.
    assert (fs.fs_logprobs_workspace_size(65535, 151936, 5)
            <= 1280 * 50 * (16 + 24 * 8))
    for bad in ((0, 64, 100), (65536, 64, 100), (4, 0, 100), (4, 64, 0)):
        assert fs.fs_logprobs_grad_workspace_size(*bad) == 0
    # G in bf16, its rows padded to 8 ids, its rounding at the tokens, where they are, and
    # dH's partial tiles (one k slice: unsplit).
    assert fs.fs_logprobs_grad_workspace_size(3, 64, 64) == 512 + 256 + 256
    assert fs.fs_logprobs_grad_workspace_size(1024, 4096, 151936) >= 1024 * 151936 * 2
    assert fs.fs_embed_grad_workspace_size(0, 64) == 0
    assert fs.fs_embed_grad_workspace_size(5, 0) == 0
    assert fs.fs_embed_grad_workspace_size(64, 10) == 4 * 256 + 256  # 2 runs x 2 x 16 floats
    assert fs.fs_embed_grad_workspace_size(1, 8) == 4 * 256 + 256


def _logprobs(**kw):
    import lm_head_gumbel_gb300 as fs
    base = dict(H=0x10000, W=0x20000, tokens=0x30000, B=4, d=256, V=4096, ldh=256, ldw=256, K=5,
                out_logp=0x40000, out_entropy=0x50000, out_lse=0x60000, out_topk_idx=0x70000,
                out_topk_logp=0x80000, workspace=0x90000, workspace_bytes=1 << 30)
    base.update(kw)
    return fs.FsLogprobsArgs(**base)


@pytest.mark.parametrize("kw,want", [
    (dict(H=None), INVALID), (dict(W=None), INVALID), (dict(H=0x10008), INVALID),
    (dict(W=0x20002), INVALID), (dict(B=0), INVALID), (dict(B=65536), INVALID),
    (dict(d=0), INVALID), (dict(V=0), INVALID), (dict(V=2**31), INVALID),
    (dict(ldh=255), INVALID), (dict(ldh=260), INVALID), (dict(ldw=248), INVALID),
    (dict(K=-1), INVALID), (dict(K=21), INVALID),
    (dict(K=0), INVALID),                        # alternatives' outputs without K
    (dict(out_topk_idx=None), INVALID), (dict(out_topk_logp=None), INVALID),
    (dict(tokens=None), INVALID), (dict(out_logp=None), INVALID),
    (dict(tokens=0x30004), INVALID), (dict(out_topk_idx=0x70004), INVALID),
    (dict(out_lse=0x60002), INVALID), (dict(temperature=0x30002), INVALID),
    (dict(vocab_mask=0xA0000, mask_ld=127), INVALID), (dict(vocab_mask=0xA0002, mask_ld=128), INVALID),
    (dict(vocab_offset=-1), INVALID), (dict(vocab_offset=2**31 - 4096), INVALID),
    (dict(flags=2), INVALID), (dict(flags=0x80000000), INVALID),
    (dict(tokens=None, out_logp=None, out_entropy=None, out_lse=None, K=0, out_topk_idx=None,
          out_topk_logp=None), INVALID),         # nothing asked for
    (dict(workspace=None), WORKSPACE), (dict(workspace=0x90080), WORKSPACE),
    (dict(workspace_bytes=255), WORKSPACE),
])
def test_logprobs_bad_arguments(lib, kw, want):
    assert lib.fs_logprobs(ctypes.byref(_logprobs(**kw)), None) == want


def _grad(**kw):
    import lm_head_gumbel_gb300 as fs
    base = dict(H=0x10000, W=0x20000, tokens=0x30000, lse=0x40000, grad_logp=0x50000, B=4, d=256,
                V=4096, ldh=256, ldw=256, out_dH=0x60000, out_dW=0x70000, lddh=256, lddw=256,
                workspace=0x90000, workspace_bytes=1 << 30)
    base.update(kw)
    return fs.FsLogprobsGradArgs(**base)


@pytest.mark.parametrize("kw,want", [
    (dict(H=None), INVALID), (dict(W=None), INVALID), (dict(tokens=None), INVALID),
    (dict(lse=None), INVALID), (dict(grad_logp=None), INVALID),
    (dict(out_dH=None, out_dW=None), INVALID),
    (dict(entropy=0x80000), INVALID), (dict(grad_entropy=0x80000), INVALID),  # both or neither
    (dict(entropy=0x80000, grad_entropy=0x80002), INVALID),
    (dict(lddh=255), INVALID), (dict(lddh=260), INVALID), (dict(lddw=0), INVALID),
    (dict(out_dH=0x60008), INVALID), (dict(out_dW=0x70004), INVALID),
    (dict(tokens=0x30004), INVALID), (dict(lse=0x40001), INVALID),
    (dict(B=0), INVALID), (dict(d=0), INVALID), (dict(V=2**31), INVALID),
    (dict(vocab_offset=-8), INVALID), (dict(vocab_mask=0xA0000, mask_ld=0), INVALID),
    (dict(B=65535, V=2**31 - 1, d=8, ldh=8, ldw=8, lddh=8, lddw=8), INVALID),  # 32-bit counts
    (dict(workspace=None), WORKSPACE), (dict(workspace=0x90010), WORKSPACE),
    (dict(workspace_bytes=4 * 4096 * 2 - 1), WORKSPACE),
])
def test_logprobs_grad_bad_arguments(lib, kw, want):
    assert lib.fs_logprobs_grad(ctypes.byref(_grad(**kw)), None) == want


def test_null_arguments(lib):
    assert lib.fs_logprobs(None, None) == INVALID
    assert lib.fs_logprobs_grad(None, None) == INVALID


def _call_embed(lib, **kw):
    a = dict(ids=0x10000, N=4, E=0x20000, V=100, d=64, lde=64, dtype=0, scale=1.0,
             vocab_offset=0, out=0x30000, ldo=64)
    a.update(kw)
    return lib.fs_embed(a["ids"], a["N"], a["E"], a["V"], a["d"], a["lde"], a["dtype"],
                        a["scale"], a["vocab_offset"], a["out"], a["ldo"], None)


@pytest.mark.parametrize("kw", [
    dict(ids=None), dict(E=None), dict(out=None), dict(N=-1), dict(N=2**31), dict(V=0),
    dict(V=2**31), dict(d=0), dict(lde=63), dict(ldo=63), dict(dtype=2), dict(dtype=-1),
    dict(vocab_offset=-1), dict(vocab_offset=2**31 - 100), dict(ids=0x10004), dict(E=0x20001),
    dict(E=0x20002, dtype=1), dict(out=0x30002, dtype=1), dict(N=2**30, d=2**30, lde=2**30, ldo=2**30),
])
def test_embed_bad_arguments(lib, kw):
    assert _call_embed(lib, **kw) == INVALID


def test_embed_of_nothing(lib):
    assert _call_embed(lib, N=0, ids=None, out=None) == 0


def _call_grad(lib, **kw):
    a = dict(ids=0x10000, N=4, dY=0x20000, V=100, d=64, ldy=64, yt=0, scale=1.0, vocab_offset=0,
             dE=0x30000, lde=64, et=0, accumulate=0, ws=0x40000, wsb=1 << 30)
    a.update(kw)
    return lib.fs_embed_grad(a["ids"], a["N"], a["dY"], a["V"], a["d"], a["ldy"], a["yt"],
                             a["scale"], a["vocab_offset"], a["dE"], a["lde"], a["et"],
                             a["accumulate"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(ids=None), INVALID), (dict(dY=None), INVALID), (dict(dE=None), INVALID),
    (dict(N=-1), INVALID), (dict(N=2**31 - 65536), INVALID), (dict(V=0), INVALID),
    (dict(d=0), INVALID), (dict(ldy=63), INVALID), (dict(lde=0), INVALID), (dict(yt=3), INVALID),
    (dict(et=-1), INVALID), (dict(yt=1, et=0), INVALID), (dict(ids=0x10001), INVALID),
    (dict(dY=0x20001), INVALID), (dict(dE=0x30002, et=1), INVALID),
    (dict(vocab_offset=2**31 - 100), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=0x40001), WORKSPACE), (dict(wsb=1000), WORKSPACE),
])
def test_embed_grad_bad_arguments(lib, kw, want):
    assert _call_grad(lib, **kw) == want


def test_embed_grad_of_nothing_added(lib):
    assert _call_grad(lib, N=0, ids=None, dY=None, accumulate=1, ws=None, wsb=0) == 0


def test_matrix_reads_stay_in_the_ring(tmp_path):
    """An MMA reads 128 rows of A, 16 KB, however few the box in shared memory holds:
    the last slice's read ends inside the ring for every box height and unit width."""
    from lm_head_gumbel_gb300 import build as libbuild
    src = tmp_path / "ring.cu"
    src.write_text("""
#include <cstdio>
#include "fs_contract.cuh"
using namespace fs::vocab;
template <int N, bool kSt> struct Epi { static constexpr int kN = N; static constexpr bool kStaged = kSt; };
template <class E, bool kPair> void print() {
  for (unsigned rows = 8; rows <= 128; rows += 8)
    std::printf("%d %d %u %u %u %d\\n", E::kN, int(kPair), rows, ring_stages<E, kPair>(rows * 128u),
                ring_bytes<E>(), slices<E>());
}
int main() {
  print<Epi<64, false>, false>(); print<Epi<128, false>, false>(); print<Epi<256, false>, false>();
  print<Epi<256, false>, true>(); print<Epi<128, true>, false>(); print<Epi<256, true>, false>();
  print<Epi<256, true>, true>();
}
""")
    exe = tmp_path / "ring"
    try:
        nvcc = libbuild.nvcc_path()
    except RuntimeError as e:
        pytest.skip(str(e))
    subprocess.run([nvcc, *libbuild.ARCH_FLAGS, "-std=c++17", f"-I{libbuild.CSRC}",
                    f"-I{libbuild.INCLUDE}", "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    lines = [[int(x) for x in line.split()] for line in out.splitlines()]
    assert len(lines) == 7 * 16
    for n, pair, rows, stages, ring, slices in lines:
        piece = rows * 128 + (n // 2 if pair else n) * 128  # A's box and B's columns, bf16 x 64
        last = (stages * slices - 1) * piece
        assert 2 <= stages <= 8
        assert last + max(piece, 128 * 128) <= ring, (n, pair, rows)


def _without_marshal(code):
    """Runs `code` in a new process where _marshal cannot be imported."""
    head = ("import sys; sys.path.insert(0, %r)\n"
            "sys.modules['lm_head_gumbel_gb300._marshal'] = None\n"
            "import torch, lm_head_gumbel_gb300 as fs\n" % ROOT)
    return subprocess.run([sys.executable, "-c", head + code], capture_output=True, text=True)


def test_the_sampler_needs_no_marshalling_module(lib):
    """Only libfs.so: the sampler's functions and the sizes work from the first call on."""
    r = _without_marshal("print(fs.fs_num_tiles(300), fs.fs_workspace_size(4, 1000) > 0,\n"
                         "      fs.fs_status_string(0), fs.fs_embed_grad_workspace_size(1, 8))")
    assert r.returncode == 0, r.stderr
    assert r.stdout.split()[:2] == ["3", "True"] and r.stdout.split()[-1] == "1280"


def test_the_operators_say_that_the_module_is_missing(lib):
    """FsError, on the first call and on every later one."""
    r = _without_marshal("""
t = torch.zeros(1)
for _ in range(2):
    for call in (lambda: fs.fs_embed(t, t), lambda: fs.fs_embed_grad(t, t, 4),
                 lambda: fs.fs_logprobs(t, t, t), lambda: fs.fs_logprobs_grad(t, t, t, t, t)):
        try:
            call()
        except fs.FsError as e:
            assert e.status == fs.FS_ERR_UNSUPPORTED and "_marshal" in str(e), str(e)
        else:
            raise SystemExit("no error")
""")
    assert r.returncode == 0, r.stderr + r.stdout


def test_a_module_for_another_torch_is_refused(lib):
    r = _without_marshal("""
import types
sys.modules['lm_head_gumbel_gb300._marshal'] = types.SimpleNamespace(torch_version="0.1")
try:
    fs.fs_embed(torch.zeros(1), torch.zeros(1))
except fs.FsError as e:
    assert e.status == fs.FS_ERR_UNSUPPORTED and "0.1" in str(e), str(e)
else:
    raise SystemExit("no error")
""")
    assert r.returncode == 0, r.stderr + r.stdout


def test_the_module_is_built_again_for_another_torch(lib):
    from lm_head_gumbel_gb300 import build as libbuild
    import torch
    assert torch.version.__file__ in libbuild.marshal_depends()
    assert libbuild.up_to_date(libbuild.MARSHAL, libbuild.marshal_depends())
    import lm_head_gumbel_gb300 as fs
    from lm_head_gumbel_gb300 import _binding
    assert _binding.load_marshal().torch_version == torch.__version__
    with pytest.raises(fs.FsError):                       # refused by the module itself
        fs.fs_embed(torch.zeros(1, dtype=torch.int64), torch.zeros(4, 4))


def test_out_dtype_is_not_ignored(lib):
    import lm_head_gumbel_gb300 as fs
    import torch
    ids, dY = torch.zeros(2, dtype=torch.int64), torch.zeros(2, 8)
    with pytest.raises(fs.FsError, match="out_dtype"):
        fs.fs_embed_grad(ids, dY, 4, out=torch.zeros(4, 8), out_dtype=torch.bfloat16)
    with pytest.raises(fs.FsError, match="out_dtype"):
        fs.fs_embed_grad(ids, dY.bfloat16(), 4, out=torch.zeros(4, 8).bfloat16(),
                         out_dtype=torch.float32, accumulate=True)
