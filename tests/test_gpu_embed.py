"""The embedding lookup and its gradient on the GPU against 64-bit forms.

Lookup: one fp32 product and one rounding.  Gradient: a row named n times is a
sum of n exact terms in fp32, off by at most (n + 2) 2^-24 of the terms'
magnitudes (however it is split), times scale (one rounding more), plus the
rounding to the table's type."""
import pytest
import torch

import lm_head_gumbel_gb300 as fs
from gpu_cases import assert_no_device_error

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fs.load_library()
    yield
    assert_no_device_error()


def matrix(n, d, dtype, *, ld=None, shift=0, seed=0):
    """[n, d] normal values with row stride ld, `shift` elements into a buffer."""
    ld = ld or d
    gen = torch.Generator().manual_seed(seed)
    buf = torch.full((n * ld + shift + 16,), 5.0, dtype=dtype, device="cuda")
    view = buf[shift:shift + n * ld].view(n, ld)[:, :d]
    view.copy_(torch.randn((n, d), generator=gen).to(dtype))
    return view, buf


# (d, row stride, offset of the first element): rows on 16-byte boundaries, rows
# that end inside a vector, rows on odd addresses, several column segments.
ROWS = [(64, 64, 0), (1, 1, 0), (100, 104, 8), (100, 100, 0), (13, 21, 3), (257, 264, 0),
        (2048, 2048, 0), (1025, 1025, 1), (3000, 3008, 0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,ld,shift", ROWS)
def test_lookup(dtype, d, ld, shift):
    V, N = 300, 77
    E, _ = matrix(V, d, dtype, ld=ld, shift=shift, seed=d)
    gen = torch.Generator().manual_seed(1)
    ids = torch.randint(0, V, (N,), generator=gen).cuda()
    ids[5], ids[6], ids[7], ids[8] = -1, V, -(2**40), 2**40
    held = ((ids >= 0) & (ids < V)).unsqueeze(1)
    rows = torch.where(held, E[ids.clamp(0, V - 1)], torch.zeros((), dtype=dtype, device="cuda"))
    assert torch.equal(fs.fs_embed(ids, E), rows)
    out, buf = matrix(N, d, dtype, ld=ld, shift=shift, seed=2)
    guard = buf.clone()
    got = fs.fs_embed(ids, E, scale=1.7, out=out)
    want = rows.double() * torch.tensor(1.7, dtype=torch.float32).double().item()
    # fp32 product, then the table's type
    assert bool(((got.double() - want).abs() <= (ROUND[dtype] + U) * want.abs()).all())
    out.copy_(guard[shift:shift + N * ld].view(N, ld)[:, :d])
    assert torch.equal(buf, guard)  # nothing outside the rows was written


@pytest.mark.parametrize("N", [0, 1, 3, 5000])
def test_lookup_lengths_and_shards(N):
    E, _ = matrix(1000, 136, torch.bfloat16, seed=3)
    ids = torch.randint(0, 1000, (N,), generator=torch.Generator().manual_seed(N)).cuda()
    whole = fs.fs_embed(ids, E)
    assert torch.equal(whole, E[ids])
    parts = [fs.fs_embed(ids, E[a:b], vocab_offset=a) for a, b in ((0, 400), (400, 401),
                                                                   (401, 1000))]
    assert torch.equal(parts[0] + parts[1] + parts[2], whole)


def gradient_want(ids, dY, V, scale, offset=0, old=None):
    """dE and the bound of its error, in fp64."""
    ids = ids.cpu() - offset
    keep = (ids >= 0) & (ids < V)
    y = dY.cpu().double()[keep]
    s = torch.tensor(scale, dtype=torch.float32).double().item()
    total = torch.zeros((V, dY.shape[1]), dtype=torch.float64).index_add_(0, ids[keep], y)
    mag = torch.zeros_like(total).index_add_(0, ids[keep], y.abs())
    count = torch.zeros(V, dtype=torch.float64).index_add_(
        0, ids[keep], torch.ones(int(keep.sum()), dtype=torch.float64)).unsqueeze(1)
    total, mag = total * s, mag * abs(s)
    bound = (count + 4) * U * mag
    if old is not None:
        total = total + old.cpu().double()
        bound = bound + 2 * U * total.abs() * (count > 0)
    return total, bound, count > 0


def check_gradient(ids, dY, V, *, scale=1.0, out=None, accumulate=False, offset=0,
                   out_dtype=None):
    old = out.clone() if accumulate else None
    got = fs.fs_embed_grad(ids, dY, V, scale=scale, out=out, accumulate=accumulate,
                           vocab_offset=offset, out_dtype=out_dtype)
    want, bound, named = gradient_want(ids, dY, V, scale, offset, old)
    bound = bound + ROUND[got.dtype] * (want.abs() + bound)
    off = (got.cpu().double() - want).abs()
    rows = named.expand_as(off)
    assert bool((off[rows] <= bound[rows]).all()), float((off[rows] - bound[rows]).max())
    rest = old if accumulate else torch.zeros_like(got)
    assert torch.equal(got.cpu()[~rows], rest.cpu()[~rows])  # exactly
    return got


COMBOS = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
          (torch.float32, torch.float32)]


def some_ids(kind, N, V, seed=0):
    gen = torch.Generator().manual_seed(seed)
    if kind == "spread":
        ids = torch.randint(0, V, (N,), generator=gen)
    elif kind == "few":    # runs of one id over many blocks
        ids = torch.randint(0, 3, (N,), generator=gen) * (V // 3)
    elif kind == "one":
        ids = torch.full((N,), V - 1)
    elif kind == "sorted":
        ids = torch.arange(N) % V
    else:                  # "ragged": a hot id, padding, ids of other shards
        ids = torch.randint(0, V, (N,), generator=gen)
        ids[torch.rand(N, generator=gen) < 0.4] = V // 2
        ids[torch.rand(N, generator=gen) < 0.1] = -1
        ids[torch.rand(N, generator=gen) < 0.05] = V + 7
    return ids.cuda()


@pytest.mark.parametrize("ty,to", COMBOS)
@pytest.mark.parametrize("d,ld,shift", ROWS)
def test_gradient_rows(ty, to, d, ld, shift):
    V, N = 150, 333
    dY, _ = matrix(N, d, ty, ld=ld, shift=shift, seed=d)
    ids = some_ids("ragged", N, V)
    out, buf = matrix(V, d, to, ld=ld, shift=shift, seed=4)
    guard = buf.clone()
    check_gradient(ids, dY, V, scale=0.37, out=out)
    out.copy_(guard[shift:shift + V * ld].view(V, ld)[:, :d])
    assert torch.equal(buf, guard)
    check_gradient(ids, dY, V, scale=0.37, out=out, accumulate=True)


@pytest.mark.parametrize("kind", ["spread", "few", "one", "sorted", "ragged"])
@pytest.mark.parametrize("N", [1, 2, 31, 32, 33, 64, 500, 1024, 8191, 8192, 8193, 20011])
def test_gradient_lengths(kind, N):
    V, d = 700, 24
    dY, _ = matrix(N, d, torch.bfloat16, seed=N)
    ids = some_ids(kind, N, V, seed=N)
    check_gradient(ids, dY, V, out_dtype=torch.float32)
    old = torch.randn((V, d), generator=torch.Generator().manual_seed(9)).cuda()
    check_gradient(ids, dY, V, scale=-2.5, out=old, accumulate=True)


@pytest.mark.parametrize("V", [1, 2, 255, 511, 512, 513, 70000, 151936, 262143, 262144])
def test_gradient_vocabularies(V):
    """One to three radix passes; several ranges of rows to zero."""
    dY, _ = matrix(3000, 16, torch.bfloat16, seed=V)
    check_gradient(some_ids("ragged", 3000, V, seed=V), dY, V)


def test_gradient_of_no_ids():
    empty = torch.empty(0, dtype=torch.int64, device="cuda")
    dY = torch.empty((0, 40), dtype=torch.bfloat16, device="cuda")
    out = torch.full((90, 40), 2.0, dtype=torch.bfloat16, device="cuda")
    fs.fs_embed_grad(empty, dY, 90, out=out, accumulate=True)
    assert bool((out == 2.0).all())
    fs.fs_embed_grad(empty, dY, 90, out=out)
    assert bool((out == 0.0).all())
    ids = torch.full((50,), -1, dtype=torch.int64, device="cuda")  # none of them in the table
    check_gradient(ids, torch.ones((50, 40), dtype=torch.bfloat16, device="cuda"), 90)


def test_gradient_of_shards():
    ids = some_ids("spread", 4000, 1000, seed=5)
    dY, _ = matrix(4000, 72, torch.bfloat16, seed=5)
    whole = fs.fs_embed_grad(ids, dY, 1000, out_dtype=torch.float32)
    for a, b in ((0, 300), (300, 301), (301, 1000)):
        check_gradient(ids, dY, b - a, offset=a, out_dtype=torch.float32)
    assert whole.shape == (1000, 72)


def test_gradient_repeats_its_bits():
    """On other streams and in a replayed graph too, whatever the workspace holds."""
    N, V, d = 9000, 5000, 136
    ids = some_ids("ragged", N, V, seed=6)
    dY, _ = matrix(N, d, torch.float32, seed=6)
    want = fs.fs_embed_grad(ids, dY, V)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        got = fs.fs_embed_grad(ids, dY, V, stream=side)
        side.synchronize()
        assert torch.equal(got, want)
    ws = torch.empty(fs.fs_embed_grad_workspace_size(N, d), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fs.fs_embed_grad(ids, dY, V, out=out, workspace=ws)
    for _ in range(3):
        ws.fill_(255)
        out.fill_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_gradient_against_differences():
    """The loss <Y, D> is linear in E: its difference along a direction is the
    gradient's product with it."""
    E, _ = matrix(60, 32, torch.float32, seed=7)
    ids = some_ids("ragged", 200, 60, seed=7)
    D, _ = matrix(200, 32, torch.float32, seed=8)
    X, _ = matrix(60, 32, torch.float32, seed=9)
    dE = check_gradient(ids, D, 60, scale=1.25)
    _, bound, _ = gradient_want(ids, D, 60, 1.25)
    h = 0.5

    def loss(sign):
        Y = fs.fs_embed(ids, (E.double() + sign * h * X.double()).float(), scale=1.25)
        return (Y.double() * D.double()).sum().item()

    diff = (loss(1) - loss(-1)) / (2 * h)
    got = (dE.double() * X.double()).sum().item()
    # dE's own bound, and the roundings of E +- hX and of Y (3 u each way)
    size = (fs.fs_embed(ids, E.abs() + X.abs(), scale=1.25).double() * D.double().abs()).sum().item()
    tol = ((bound + U * dE.cpu().double().abs()) * X.cpu().double().abs()).sum().item() + 12 * U * size / (2 * h)
    assert abs(got - diff) <= tol


def test_binding_refusals():
    E, _ = matrix(50, 16, torch.bfloat16)
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    dY, _ = matrix(4, 16, torch.bfloat16)
    f32 = torch.zeros((4, 16), device="cuda")
    bad = [
        lambda: fs.fs_embed(ids.int(), E), lambda: fs.fs_embed(ids.cpu(), E),
        lambda: fs.fs_embed(ids, E.half()), lambda: fs.fs_embed(ids, E.t()),
        lambda: fs.fs_embed(ids.view(2, 2), E), lambda: fs.fs_embed(ids, E, out=f32),
        lambda: fs.fs_embed(ids, E, vocab_offset=-4),
        lambda: fs.fs_embed_grad(ids[:3], dY, 50), lambda: fs.fs_embed_grad(ids, dY, 0),
        lambda: fs.fs_embed_grad(ids, dY, 50, accumulate=True),
        lambda: fs.fs_embed_grad(ids, f32, 50, out=torch.zeros_like(E)),
        lambda: fs.fs_embed_grad(ids, dY, 50, out=E[:49]),
        lambda: fs.fs_embed_grad(ids, dY, 50,
                                 workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
    ]
    for call in bad:
        with pytest.raises(fs.FsError):
            call()


# --------------------------------------------------------------------------- sizes at which the work is cut differently
@pytest.mark.parametrize("ty,to", COMBOS)
@pytest.mark.parametrize("N,V,d", [(1023, 3000, 100), (1024, 3000, 65), (1025, 3000, 100),
                                   (4099, 70000, 40), (8192, 300, 136), (8193, 300, 136),
                                   (33000, 40000, 24)])
def test_gradient_of_every_path(ty, to, N, V, d):
    """One kernel, the cluster's shared memory, the cluster through L2; all rows
    written or some added to; hot ids over several runs."""
    dY, _ = matrix(N, d, ty, ld=(d + 7) // 8 * 8, seed=N)
    for kind in ("ragged", "few"):
        ids = some_ids(kind, N, V, seed=N)
        check_gradient(ids, dY, V, scale=0.5, out_dtype=to)
        old, _ = matrix(V, d, to, ld=(d + 7) // 8 * 8, seed=3)
        check_gradient(ids, dY, V, scale=0.5, out=old, accumulate=True)


@pytest.mark.parametrize("N", [2049, 5000, 5001, 12000, 12001, 20000, 20001])
def test_gradient_run_lengths(N):
    dY, _ = matrix(N, 40, torch.bfloat16, seed=N)
    for kind in ("ragged", "few"):
        ids = some_ids(kind, N, 5000, seed=N)
        check_gradient(ids, dY, 5000, out_dtype=torch.float32)
        old, _ = matrix(5000, 40, torch.bfloat16, seed=3)
        check_gradient(ids, dY, 5000, scale=2.0, out=old, accumulate=True)


def test_dense_gradient_in_a_graph_on_a_side_stream():
    """The zeroing runs beside the sort; what follows on the stream sees both done."""
    for N in (700, 5000, 20000):
        ids = some_ids("ragged", N, 30000, seed=N)
        dY, _ = matrix(N, 64, torch.bfloat16, seed=N)
        want = fs.fs_embed_grad(ids, dY, 30000)
        ws = torch.empty(fs.fs_embed_grad_workspace_size(N, 64), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(want)
        copy = torch.empty_like(want)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            for _ in range(20):
                out.fill_(7.0)
                fs.fs_embed_grad(ids, dY, 30000, out=out, workspace=ws)
                copy.copy_(out)
                assert torch.equal(copy, want)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out.fill_(7.0)
                fs.fs_embed_grad(ids, dY, 30000, out=out, workspace=ws)
                copy.copy_(out)
        for _ in range(20):
            copy.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(copy, want)


# --------------------------------------------------------------------------- offsets past 32 bits
def test_tables_past_32_bits():
    """Lookup and gradients (of one, a few thousand and more ids) of a table, and of
    an output, of more than 2^32 elements.  Whole numbers: every sum is exact."""
    V, d, ld = 70000, 24, 1 << 16
    table = torch.as_strided(torch.zeros((V - 1) * ld + d, dtype=torch.bfloat16, device="cuda"),
                             (V, d), (ld, 1))
    rows = torch.arange(V, device="cuda").unsqueeze(1)
    table.copy_((rows + torch.arange(d, device="cuda")) % 251 - 125)
    ids = torch.tensor([V - 1, 0, V - 2, 65536, -1, V], device="cuda")
    want = torch.zeros(6, d, dtype=torch.bfloat16, device="cuda")
    want[:4] = table[ids[:4]]
    assert torch.equal(fs.fs_embed(ids, table), want)
    out = torch.as_strided(torch.empty(5 * (1 << 30) + d, dtype=torch.bfloat16, device="cuda"),
                           (6, d), (1 << 30, 1))
    assert torch.equal(fs.fs_embed(ids, table, out=out), want)
    del out
    gen = torch.Generator(device="cuda").manual_seed(5)
    for N in (1000, 5000, 20000):
        ids = torch.randint(0, V, (N,), generator=gen, device="cuda")
        ids[:4] = torch.tensor([V - 1, 0, V - 2, 65536], device="cuda")
        dY = torch.randint(-8, 9, (N, d), generator=gen, device="cuda").bfloat16()
        sums = torch.zeros(V, d, device="cuda").index_add_(0, ids, dY.float())
        assert float(sums.abs().max()) <= 256
        dE = torch.as_strided(torch.full(((V - 1) * ld + d,), 3.0, dtype=torch.bfloat16,
                                         device="cuda"), (V, d), (ld, 1))
        fs.fs_embed_grad(ids, dY, V, out=dE)
        assert torch.equal(dE.float(), sums)
        assert float(dE.as_strided((V - 1, 8), (ld, 1), d).min()) == 3.0  # between the rows
        fs.fs_embed_grad(ids, dY, V, out=dE, accumulate=True)
        assert torch.equal(dE.float(), 2 * sums)
        del dE


@pytest.mark.parametrize("ty,to", COMBOS)
@pytest.mark.parametrize("d,ld", [(1, 1), (5, 5), (7, 8), (31, 33), (33, 33), (255, 255), (256, 257),
                                  (263, 263), (300, 301), (513, 515)])
def test_gradient_of_unaligned_rows(ty, to, d, ld):
    """Rows that do not start on 16-byte boundaries, of dY or of the table."""
    N, V = 2500, 600
    for kind in ("ragged", "few"):
        ids = some_ids(kind, N, V, seed=d)
        for dY_ld, out_ld in ((ld, ld), ((d + 7) // 8 * 8, ld), (ld, (d + 7) // 8 * 8)):
            dY, _ = matrix(N, d, ty, ld=dY_ld, seed=d)
            old, buf = matrix(V, d, to, ld=out_ld, seed=3)
            check_gradient(ids, dY, V, scale=0.5, out=old, accumulate=True)
            old, buf = matrix(V, d, to, ld=out_ld, seed=3)
            check_gradient(ids, dY, V, out=old)
            assert bool((buf[V * out_ld:] == 5.0).all())  # behind the last row
            assert bool((buf[:V * out_ld].view(V, out_ld)[:, d:] == 5.0).all())  # between rows


def test_workspaces_of_two_streams():
    """Gradients on two streams, neither waited for, with workspaces made inside."""
    V, N, d = 3000, 6000, 256
    cases = []
    for seed in (40, 41):
        dY, _ = matrix(N, d, torch.bfloat16, seed=seed)
        cases.append((some_ids("spread", N, V, seed).cuda(), dY))
    want = [fs.fs_embed_grad(ids, dY, V, out_dtype=torch.float32) for ids, dY in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(4):
        for (ids, dY), stream, w in zip(cases, streams, want):
            got.append((fs.fs_embed_grad(ids, dY, V, out_dtype=torch.float32, stream=stream), w))
        scratch = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
                   for _ in range(4)]  # the current stream's allocations meanwhile
    torch.cuda.synchronize()
    del scratch
    assert all(torch.equal(g, w) for g, w in got)
    owner = {seg["stream"] for g, _ in got[:1] for seg in torch.cuda.memory_snapshot()
             if seg["address"] <= g.data_ptr() < seg["address"] + seg["total_size"]}
    assert owner == {streams[0].cuda_stream}


@pytest.mark.parametrize("N", [1025, 1032, 2049, 8191, 8192])
def test_cluster_sort_call_after_call(N):
    """Sorts in one cluster's shared memory, right behind one another: CTAs that get
    their first pairs while others of the cluster have only just started."""
    V, d = 700, 8
    ids = some_ids("ragged", N, V, seed=N)
    dY, _ = matrix(N, d, torch.float32, seed=N)
    want = check_gradient(ids, dY, V)
    got = [fs.fs_embed_grad(ids, dY, V) for _ in range(50)]
    assert all(torch.equal(g, want) for g in got)
