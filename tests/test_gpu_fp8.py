"""Quantisation to 8 bits with a scale for each block of 128, and the product of such
matrices, on the GPU against the forms of speculate_ref."""
import pytest
import torch

import lm_head_gumbel_gb300 as fs
import speculate_ref as ref
from gpu_cases import assert_no_device_error

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fs.load_library()
    yield
    assert_no_device_error()


def matrix(n, d, dtype, *, ld=None, shift=0, seed=0, std=1.0):
    """[n, d] normal values with row stride ld, `shift` elements into a buffer."""
    ld = ld or d
    gen = torch.Generator().manual_seed(seed)
    buf = torch.full((n * ld + shift + 16,), 5.0, device="cuda").to(dtype)
    view = buf[shift:shift + n * ld].view(n, ld)[:, :d]
    view.copy_((torch.randn((n, d), generator=gen) * std).to(dtype))
    return view, buf


def same_bits(a, b, bits):
    """Equal bit by bit, one NaN being as good as another."""
    a, b = a.cpu().contiguous(), b.contiguous()
    nan = a.float().isnan()
    assert torch.equal(nan, b.float().isnan())
    assert torch.equal(a.view(bits)[~nan], b.view(bits)[~nan])


def check_quantized(x, block, **kw):
    got = fs.fs_quantize(x, block, **kw)
    values, scale = ref.quantize(x, block)
    same_bits(got.scale, scale, torch.int32)
    same_bits(got.values, values, torch.uint8)
    return got


# (N, d, row stride, offset): blocks that end early both ways, rows off 16 bytes, one element.
SHAPES = [(1, 1, 1, 0), (1, 128, 128, 0), (3, 130, 136, 8), (130, 257, 257, 0), (129, 1000, 1003, 3),
          (257, 384, 384, 0), (64, 4096, 4096, 0), (500, 100, 104, 0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("N,d,ld,shift", SHAPES)
def test_quantize(N, d, ld, shift, block, dtype):
    x, _ = matrix(N, d, dtype, ld=ld, shift=shift, seed=N + d, std=3.0)
    check_quantized(x, block)
    # Into given tensors: nothing outside them is written.
    n, k = -(-N // block), -(-d // 128)
    out, buf = matrix(N, d, torch.float8_e4m3fn, ld=ld + 5, shift=shift, seed=1)
    scale = torch.full((n, k + 3), 7.0, device="cuda")
    guard = buf.clone().view(torch.uint8)
    got = check_quantized(x, block, out=out, out_scale=scale[:, :k])
    assert got.values is out and bool((scale[:, k:] == 7.0).all())
    inside = torch.zeros_like(buf, dtype=torch.bool)
    inside[shift:shift + N * (ld + 5)].view(N, ld + 5)[:, :d] = True
    assert torch.equal(buf.view(torch.uint8)[~inside], guard[~inside])


@pytest.mark.parametrize("block", [1, 128])
def test_quantize_extremes(block):
    """Blocks of zeros, of one tiny or subnormal value, of the largest, of NaN and infinity;
    values that fall on and next to the middle between two steps."""
    x = torch.zeros((260, 700), device="cuda")
    x[0, 5] = 1e-42
    x[130, 129] = 1e-29
    x[130, 130] = -3e-30
    x[1, 260:300] = 3.4e38
    x[1, 300:310] = 1e30
    x[140, 390] = float("nan")
    x[3, 520] = float("inf")
    x[4, 650], x[4, 651] = -1.0, 2.0 ** -20
    steps = torch.arange(0, 128, device="cuda", dtype=torch.float32)
    x[250, :128], x[250, 0] = (steps + 0.5) / 16, 448.0   # scale 1: middles stay middles
    x[251, :128], x[251, 0] = torch.nextafter((steps + 0.5) / 16, steps + 9), 448.0
    check_quantized(x, block)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("block", [1, 128])
def test_quantize_rounds_each_division_once(block, dtype):
    """448 / a and a / 448 are the nearest fp32 values, which a rounded reciprocal times 448 (or a
    times a rounded 1 / 448) often is not; it decides values on a middle between two e4m3 ones."""
    gen = torch.Generator().manual_seed(40 + block)
    n = 4096 if block == 1 else 128 * 40
    x = torch.randn((n, 128 * 8), generator=gen).to(dtype)
    got = fs.fs_quantize(x.cuda(), block)
    top = x.double().abs().view(n // block, block, 8, 128).amax((1, 3))
    # 64 bits are more than twice 24 and 2: the second rounding changes nothing
    inverse, scale = (448.0 / top).float(), (top / 448.0).float()
    two = torch.full_like(inverse, 448.0) * (torch.ones_like(inverse) / top.float())
    assert bool((two != inverse).any())  # the inputs tell the two apart
    assert torch.equal(got.scale.cpu(), scale)
    wide = inverse.repeat_interleave(block, 0).repeat_interleave(128, 1)
    want = (x.float() * wide).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    same_bits(got.values, want, torch.uint8)


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("N,d,ld", [(2, 1, 4), (5, 3, 4), (130, 2, 4), (300, 4, 4), (3, 5, 8), (3, 9, 12)])
def test_quantize_of_very_narrow_rows(N, d, ld, block):
    """fp32 rows 16 bytes apart, up to the end of their buffer."""
    gen = torch.Generator().manual_seed(N)
    buf = torch.full(((N - 1) * ld + d,), float("nan"), device="cuda")
    x = buf.as_strided((N, d), (ld, 1))
    x.copy_(torch.randn((N, d), generator=gen))
    check_quantized(x, block)


def test_quantize_of_nothing():
    r = fs.fs_quantize(torch.zeros((0, 300), device="cuda"))
    assert r.values.shape == (0, 300) and r.scale.shape == (0, 3)


def check_product(A, a_scale, W, w_scale, dtype, out=None, **kw):
    got = fs.fs_matmul_fp8(A, a_scale, W, w_scale, out=out,
                           out_dtype=None if out is not None else dtype, **kw)
    want, bound = ref.matmul(A, a_scale, W, w_scale, dtype)
    assert got.dtype is dtype
    err = (got.cpu().double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound.clamp_min(1e-300)).max())
    return got


def operands(M, d, V, seed=0):
    x, _ = matrix(M, d, torch.bfloat16, seed=seed)
    w, _ = matrix(V, d, torch.bfloat16, seed=seed + 1, std=2.0 / d ** 0.5)
    a, b = fs.fs_quantize(x), fs.fs_quantize(w, 128)
    # scales that differ a lot from block to block
    gen = torch.Generator().manual_seed(seed)
    a.scale.mul_(torch.exp2(torch.randint(-3, 4, a.scale.shape, generator=gen)).cuda())
    b.scale.mul_(torch.exp2(torch.randint(-3, 4, b.scale.shape, generator=gen)).cuda())
    return a.values, a.scale, b.values, b.scale


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,d,V", [
    (1, 1, 1), (1, 128, 64), (4, 256, 4096), (3, 100, 130), (8, 129, 257), (17, 1000, 500),
    (64, 640, 1000), (127, 256, 300), (128, 384, 513),        # one tile of rows
    (129, 256, 300), (200, 130, 700), (256, 512, 1000), (257, 300, 255), (385, 200, 520),  # pairs
    (5, 256, 12000), (5, 256, 21000), (33, 130, 40000), (700, 128, 3000),  # wider units, waves
    (2, 5120, 100), (130, 2000, 130),
    (200, 130, 25000), (385, 200, 20001), (700, 128, 30000),  # CTA pairs, several rows of tiles
    (320, 256, 30000), (129, 2100, 45000), (300, 300, 10000)])  # single CTAs, several rows
def test_product(M, d, V, dtype):
    check_product(*operands(M, d, V, seed=M + d + V), dtype)


def test_product_is_what_the_values_say():
    """Whole numbers: every product and sum is exact, so is the result."""
    gen = torch.Generator().manual_seed(3)
    for M, d, V in ((7, 512, 300), (300, 640, 1000)):
        A = torch.randint(-8, 9, (M, d), generator=gen).float().cuda().to(torch.float8_e4m3fn)
        W = torch.randint(-8, 9, (V, d), generator=gen).float().cuda().to(torch.float8_e4m3fn)
        k = d // 128
        sa = torch.exp2(torch.randint(-2, 3, (M, k), generator=gen)).cuda()
        sw = torch.exp2(torch.randint(-2, 3, (-(-V // 128), k), generator=gen)).cuda()
        want = ref.widen(A, sa, 1) @ ref.widen(W, sw, 128).T
        got = fs.fs_matmul_fp8(A, sa, W, sw, out_dtype=torch.float32)
        assert torch.equal(got.cpu().double(), want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [1, 40, 129])
@pytest.mark.parametrize("ldo,shift", [(333, 0), (336, 8), (340, 1), (400, 4)])
def test_product_into_given_rows(M, ldo, shift, dtype):
    """Row strides and offsets of every alignment; nothing outside the rows is written."""
    d, V = 200, 333
    a, sa, w, sw = operands(M, d, V, seed=5)
    wide = torch.zeros((V, 1024), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    wide[:, 512:512 + d].copy_(w)  # a strided head
    out, buf = matrix(M, V, dtype, ld=ldo, shift=shift, seed=1)
    guard = buf.clone()
    scales = torch.zeros((M, 9), device="cuda")
    scales[:, :sa.shape[1]] = sa
    got = check_product(a, scales[:, :sa.shape[1]], wide[:, 512:512 + d], sw, dtype, out=out)
    assert got is out
    out.copy_(guard[shift:shift + M * ldo].view(M, ldo)[:, :V])
    assert torch.equal(buf, guard)


@pytest.mark.parametrize("V", [2000, 12000, 30000])
def test_rows_do_not_depend_on_the_batch(V):
    """A row's logits have the same bits alone, in a batch and in a pair's tile."""
    a, sa, w, sw = operands(700, 1000, V, seed=9)
    whole = fs.fs_matmul_fp8(a, sa, w, sw, out_dtype=torch.float32)
    for n in (1, 5, 64, 128, 129, 200, 320, 700):
        part = fs.fs_matmul_fp8(a[:n], sa[:n], w, sw, out_dtype=torch.float32)
        assert torch.equal(part, whole[:n])


def test_nan_and_infinity_stay_in_their_rows():
    a, sa, w, sw = operands(140, 512, 600, seed=11)
    want = fs.fs_matmul_fp8(a, sa, w, sw, out_dtype=torch.float32)
    a2, sa2, w2, sw2 = a.clone(), sa.clone(), w.clone(), sw.clone()
    a2.view(torch.uint8)[7, 300] = 0x7F
    sa2[9, 1] = float("inf")
    w2.view(torch.uint8)[450, 13] = 0xFF
    got = fs.fs_matmul_fp8(a2, sa2, w2, sw2, out_dtype=torch.float32)
    keep = torch.ones_like(want, dtype=torch.bool)
    keep[7], keep[9], keep[:, 450] = False, False, False
    assert torch.equal(got[keep], want[keep])
    assert not bool(got[7].isfinite().any() | got[9].isfinite().any() | got[:, 450].isfinite().any())


def test_product_of_nothing():
    a, sa, w, sw = operands(4, 256, 100)
    assert fs.fs_matmul_fp8(a[:0], sa[:0], w, sw).shape == (0, 100)


def test_refusals():
    a, sa, w, sw = operands(4, 256, 300)
    bad = [
        lambda: fs.fs_matmul_fp8(a, sa[:, :1], w, sw), lambda: fs.fs_matmul_fp8(a, sa, w, sw[:2]),
        lambda: fs.fs_matmul_fp8(a, sa.double(), w, sw), lambda: fs.fs_matmul_fp8(a, sa, w.float(), sw),
        lambda: fs.fs_matmul_fp8(a[:, :128], sa, w, sw), lambda: fs.fs_matmul_fp8(a.cpu(), sa, w, sw),
        lambda: fs.fs_matmul_fp8(a[:, 1:129], sa[:, :1], w[:, 1:129], sw[:, :1]),  # off 16 bytes
        lambda: fs.fs_matmul_fp8(a, sa, w, sw, out=torch.empty((4, 299), device="cuda")),
        lambda: fs.fs_matmul_fp8(a, sa, w, sw, out=torch.empty((4, 300), device="cuda").half()),
        lambda: fs.fs_quantize(torch.zeros((4, 8), device="cuda"), 64),
        lambda: fs.fs_quantize(torch.zeros((4, 8), device="cuda").t()),
        lambda: fs.fs_quantize(torch.zeros((4, 8), device="cuda"),
                               out=torch.zeros((4, 8), device="cuda")),
    ]
    for call in bad:
        with pytest.raises(fs.FsError) as e:
            call()
        assert e.value.status == fs.FS_ERR_INVALID_ARG


@pytest.mark.parametrize("M,V", [(6, 3000), (300, 3000), (200, 25000)])
def test_streams_graphs_and_overlap(M, V):
    """The same bits on another stream, in a replayed graph with new inputs, and behind the
    kernel that makes A with overlap_previous."""
    x, _ = matrix(M, 1000, torch.bfloat16, seed=21)
    w, _ = matrix(V, 1000, torch.bfloat16, seed=22)
    head = fs.fs_quantize(w, 128)
    first = fs.fs_quantize(x)
    want = fs.fs_matmul_fp8(*first, *head)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    q = fs.fs_quantize(x, stream=stream)
    got = fs.fs_matmul_fp8(*q, *head, stream=stream, overlap_previous=True)
    stream.synchronize()
    assert torch.equal(got, want)
    graph, xs = torch.cuda.CUDAGraph(), x.clone()
    with torch.cuda.graph(graph):
        q = fs.fs_quantize(xs)
        out = fs.fs_matmul_fp8(*q, *head, overlap_previous=True)
    for seed in range(3):
        xs.copy_(matrix(M, 1000, torch.bfloat16, seed=seed)[0])
        graph.replay()
        assert torch.equal(out, fs.fs_matmul_fp8(*fs.fs_quantize(xs), *head))
    for _ in range(20):  # call after call, overlapped
        q = fs.fs_quantize(x)
        assert torch.equal(fs.fs_matmul_fp8(*q, *head, overlap_previous=True), want)


def test_call_after_call():
    """Calls right behind one another that write what the next one reads: no call starts on
    what the one before has not finished."""
    a, sa, w, sw = operands(150, 640, 640, seed=17)
    x = a.float()
    want = []
    for _ in range(4):
        q = fs.fs_quantize(x)
        torch.cuda.synchronize()
        x = fs.fs_matmul_fp8(*q, w, sw, out_dtype=torch.float32)
        torch.cuda.synchronize()
        want.append(x)
    for _ in range(20):
        x = a.float()
        got = []
        for _ in range(4):
            x = fs.fs_matmul_fp8(*fs.fs_quantize(x), w, sw, out_dtype=torch.float32)
            got.append(x)
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_two_streams_at_once():
    cases = [operands(M, 1000, 25000, seed=M) for M in (20, 260)]
    want = [fs.fs_matmul_fp8(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [(fs.fs_matmul_fp8(*c, stream=s), w) for _ in range(5)
           for c, s, w in zip(cases, streams, want)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in got)


def test_offsets_past_32_bits():
    """A head, an output and quantised rows whose ends lie past 2^32 elements."""
    V, d, ld = 70000, 100, 1 << 16
    x, _ = matrix(V, d, torch.bfloat16, ld=104, seed=31)
    wide = torch.empty((V - 1) * ld + 112, dtype=torch.uint8, device="cuda")
    w = wide.view(torch.float8_e4m3fn).as_strided((V, d), (ld, 1))
    q = fs.fs_quantize(x, 128, out=w)
    small = fs.fs_quantize(x, 128)
    assert torch.equal(q.scale, small.scale)
    assert torch.equal(q.values.contiguous().view(torch.uint8),
                       small.values.contiguous().view(torch.uint8))
    a = fs.fs_quantize(matrix(3, d, torch.bfloat16, seed=32)[0])
    out = torch.empty(2 * (1 << 32) + V, dtype=torch.bfloat16, device="cuda")
    out = out.as_strided((3, V), (1 << 32, 1))
    got = fs.fs_matmul_fp8(*a, *q, out=out)
    assert torch.equal(got.contiguous(), fs.fs_matmul_fp8(*a, *small))
    rows = torch.as_strided(torch.empty((V - 1) * ld + d, dtype=torch.bfloat16, device="cuda"),
                            (V, d), (ld, 1))
    rows.copy_(x)
    assert torch.equal(fs.fs_quantize(rows).scale, fs.fs_quantize(x).scale)
