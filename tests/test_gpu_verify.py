"""Probabilities from logits and the verification of drafted tokens on the GPU against
the forms of speculate_ref, and the operators of speculative decoding together."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import lm_head_gumbel_gb300 as fs
import speculate_ref as ref
from gpu_cases import assert_no_device_error
from oracle.merge import chi_square_gof

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float32]
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fs.load_library()
    yield
    assert_no_device_error()


def logits(N, V, dtype, *, ld=None, shift=0, seed=0, std=4.0):
    ld = ld or V
    gen = torch.Generator().manual_seed(seed)
    buf = torch.full((N * ld + shift + 16,), 5.0, dtype=dtype, device="cuda")
    view = buf[shift:shift + N * ld].view(N, ld)[:, :V]
    view.copy_((torch.randn((N, V), generator=gen) * std).to(dtype))
    return view, buf


def pack(allow):
    N, V = allow.shape
    n = (V + 31) // 32
    bits = torch.zeros((N, n * 32), dtype=torch.int64)
    bits[:, :V] = allow
    words = (bits.view(N, n, 32) << torch.arange(32)).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32).cuda()


def check_probs(x, T=None, mask=None, dtype=torch.float32, out=None):
    want, bound = ref.probs(x, T, mask, dtype)
    got = fs.fs_probs(x, temperature=T, vocab_mask=mask, out=out,
                      out_dtype=None if out is not None else dtype)
    assert got.dtype is dtype
    g = got.cpu().double()
    err = (g - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    assert bool((g[want == 0] <= 2.0 ** -126).all())
    return got


@pytest.mark.parametrize("ti", TYPES)
@pytest.mark.parametrize("to", TYPES)
@pytest.mark.parametrize("N,V,ld,shift", [
    (1, 1, 1, 0), (2, 31, 31, 0), (3, 33, 40, 8), (5, 1000, 1001, 1), (7, 4096, 4096, 0),
    (300, 513, 520, 0), (2, 50001, 50001, 3), (1, 151936, 151936, 0), (3, 262144, 262144, 0)])
def test_probs(N, V, ld, shift, ti, to):
    x, _ = logits(N, V, ti, ld=ld, shift=shift, seed=N + V)
    check_probs(x, dtype=to)
    gen = torch.Generator().manual_seed(V)
    T = (torch.rand(N, generator=gen) + 0.5).cuda()
    mask = pack(torch.rand((N, V), generator=gen) < 0.7)
    check_probs(x, T, mask, to)
    out, buf = logits(N, V, to, ld=ld + 3, shift=shift, seed=1)
    guard = buf.clone()
    assert check_probs(x, T, mask, to, out=out) is out
    out.copy_(guard[shift:shift + N * (ld + 3)].view(N, ld + 3)[:, :V])
    assert torch.equal(buf, guard)


@pytest.mark.parametrize("ti", TYPES)
@pytest.mark.parametrize("V,ld", [
    (8193, 8200), (16384, 16384), (16385, 16392), (33001, 33008), (49153, 49160), (100002, 100008),
    (131072, 131072), (131073, 131080), (170001, 170001), (262145, 262152)])
def test_probs_of_every_number_of_ctas(V, ld, ti):
    """Rows held by 1 to 16 CTAs and longer ones, whose last CTA has few elements or none, and
    whose ends do not fill 16 bytes."""
    x, _ = logits(2, V, ti, ld=ld, seed=V)
    x[0, V - 1] = 25.0
    gen = torch.Generator().manual_seed(V)
    check_probs(x, dtype=ti)
    check_probs(x, torch.tensor([0.7, 0.0]).cuda(), pack(torch.rand((2, V), generator=gen) < 0.5))


@pytest.mark.parametrize("ti", TYPES)
@pytest.mark.parametrize("N,V,ld", [(2000, 515, 520), (1300, 2051, 2056), (700, 4099, 4099),
                                    (130, 50003, 50008)])
def test_probs_of_more_rows_than_fit(N, V, ld, ti):
    """Clusters that take several rows, sampled and greedy ones, with their own masks."""
    x, _ = logits(N, V, ti, ld=ld, seed=N)
    gen = torch.Generator().manual_seed(N)
    T = torch.rand(N, generator=gen) + 0.5
    T[torch.rand(N, generator=gen) < 0.3] = 0.0
    allow = torch.rand((N, V), generator=gen) < 0.6
    allow[5], allow[N - 1, 1:] = False, False
    x[7] = -float("inf")
    mask = pack(allow)
    got = check_probs(x, T.cuda(), mask, ti)
    for _ in range(5):
        assert torch.equal(fs.fs_probs(x, temperature=T.cuda(), vocab_mask=mask, out_dtype=ti), got)
    for n in (0, 5, 7, N // 2, N - 1):  # a row's bits do not depend on the others
        one = fs.fs_probs(x[n:n + 1], temperature=T[n:n + 1].cuda(),
                          vocab_mask=mask[n:n + 1].contiguous(), out_dtype=ti)
        assert torch.equal(one, got[n:n + 1])


def test_probs_behind_the_kernel_that_makes_the_logits():
    """Call after call in place, then verification of what the last one made: none starts on
    what the one before has not finished."""
    z, _ = logits(40, 30000, torch.float32, seed=23)
    ids = torch.zeros((40, 0), dtype=torch.int64, device="cuda")
    u = torch.rand((40, 1), generator=torch.Generator().manual_seed(1)).cuda()

    def chain(sync):
        x = z.clone()
        for _ in range(4):
            x *= 3.0
            fs.fs_probs(x, out=x)
            sync()
        return x, fs.fs_verify(x.unsqueeze(1), ids, u).ids

    want, drawn = chain(torch.cuda.synchronize)
    for _ in range(20):
        x, got = chain(lambda: None)
        assert torch.equal(x, want) and torch.equal(got, drawn)


@pytest.mark.parametrize("ti", TYPES)
@pytest.mark.parametrize("V", [5, 1000, 70001])
def test_probs_of_greedy_rows(V, ti):
    """All on the lowest id of the largest allowed logit, whichever way T says greedy."""
    gen = torch.Generator().manual_seed(V)
    x = torch.randint(-3, 4, (6, V), generator=gen).to(ti).cuda()  # many equal largest
    x[4, 0] = float("nan")
    x[5, V - 1] = float("inf")
    T = torch.tensor([0.0, -1.0, float("nan"), float("inf"), 0.0, -float("inf")]).cuda()
    got = check_probs(x, T)
    assert bool((got.sum(1) == 1).all()) and bool((got.amax(1) == 1).all())
    allow = torch.rand((6, V), generator=gen) < 0.5
    allow[0] = False
    got = check_probs(x, T, pack(allow))
    assert float(got[0].sum()) == 0.0


def test_probs_of_rows_with_nothing_nan_or_infinities():
    V = 3000
    x, _ = logits(8, V, torch.float32, seed=3)
    allow = torch.ones((8, V), dtype=torch.bool)
    allow[0] = False                      # nothing allowed
    x[1] = -float("inf")                  # allowed, all -inf
    x[2, 5:] = -float("inf")              # a few left
    allow[3, 100:200] = False             # NaN and infinities at masked ids
    x[3, 100], x[3, 150], x[3, 199] = float("nan"), float("inf"), -float("inf")
    x[4, 7], x[5, 2999] = float("nan"), float("inf")
    x[6] = 1e30                           # far beyond what exp takes
    x[6, 17] = torch.nextafter(x[6, 17], x[6, 17] * 2)
    x[7] = torch.where(torch.arange(V, device="cuda") % 2 == 0, 3.4e38, -3.4e38)
    mask = pack(allow)
    keep = [0, 1, 2, 3, 6, 7]
    check_probs(x[keep], None, mask[keep].contiguous())
    got = fs.fs_probs(x, vocab_mask=mask)
    assert bool(got[4].isnan().all()) and bool(got[5].isnan().all())
    masked = allow.clone()
    masked[4, 50:60] = False
    got = fs.fs_probs(x, vocab_mask=pack(masked))
    assert bool((got[4, 50:60] == 0).all()) and bool(got[4, 60:].isnan().all())


@pytest.mark.parametrize("T", [1e-3, 2.0 ** -126, 1e-45, 0.03, 7.0, 1e6, 3e38])
def test_probs_temperatures(T):
    """From nearly greedy to nearly uniform."""
    x, _ = logits(3, 5000, torch.float32, seed=8)
    x[1].mul_(0.01)
    check_probs(x, torch.full((3,), T, device="cuda"))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [3000, 70000, 262145, 300000])
def test_probs_of_the_largest_logits_and_temperatures(V, dtype):
    """Logits whose difference is past the largest number, at temperatures that make it an
    ordinary one; and at ones that do not."""
    gen = torch.Generator().manual_seed(V)
    x = ((torch.rand((4, V), generator=gen) * 2 - 1) * 3.3e38).to(dtype).cuda()
    x[3, ::3] = -float("inf")
    check_probs(x, torch.tensor([1e38, 3e37, 1.0, 2e38]).cuda(), dtype=torch.float32)


def test_probs_far_below_the_largest():
    """Probabilities down to 2^-126 as exactly as the large ones."""
    x = torch.linspace(-87.0, 0.0, 4096, device="cuda").repeat(2, 1)
    x[1] += 30.0
    want, _ = ref.probs(x, None, None, torch.float32)
    got = fs.fs_probs(x).cpu().double()
    normal = want > 2.0 ** -125
    assert float(((got - want).abs() / want)[normal].max()) <= 2 * (2.0 ** -22 + 2.0 ** -23) + 107 * ref.U


@pytest.mark.parametrize("dtype", TYPES)
def test_probs_in_place(dtype):
    for N, V in ((3, 1000), (200, 4096), (2, 200000)):
        x, _ = logits(N, V, dtype, seed=V)
        T = torch.full((N,), 0.9, device="cuda")
        T[0] = 0.0
        want = fs.fs_probs(x, temperature=T, out_dtype=dtype)
        assert torch.equal(fs.fs_probs(x, temperature=T, out=x), want)


def test_probs_refusals():
    x = torch.zeros((4, 100), device="cuda")
    bad = [
        lambda: fs.fs_probs(x.half()), lambda: fs.fs_probs(x[0]), lambda: fs.fs_probs(x.t()),
        lambda: fs.fs_probs(x, temperature=torch.ones(3, device="cuda")),
        lambda: fs.fs_probs(x, temperature=torch.ones(4)),
        lambda: fs.fs_probs(x, vocab_mask=torch.ones((4, 3), dtype=torch.int32, device="cuda")),
        lambda: fs.fs_probs(x, vocab_mask=torch.ones((1, 4), dtype=torch.int32, device="cuda").expand(4, 4)),
        lambda: fs.fs_probs(x, out=torch.zeros((4, 99), device="cuda")),
        lambda: fs.fs_probs(x.expand(4, 4, 100)[0].as_strided((4, 100), (0, 1))),
    ]
    for call in bad:
        with pytest.raises(fs.FsError) as e:
            call()
        assert e.value.status == fs.FS_ERR_INVALID_ARG
    assert fs.fs_probs(x[:0]).shape == (0, 100)


def test_probs_of_very_many_rows():
    """More rows than 16 CTAs each would leave 32 bits for."""
    N = 2 ** 27 + 3
    x = torch.zeros((N, 1), dtype=torch.bfloat16, device="cuda")
    x[::5] = -float("inf")
    got = fs.fs_probs(x, out=x)
    assert bool((got[::5] == 0).all()) and int((got == 1).sum()) == N - (N + 4) // 5


# --------------------------------------------------------------------------- verification
def problem(B, K, V, dtype, *, seed=0, near=0.5, std=3.0, ragged=False, q=True, ld=None):
    gen = torch.Generator().manual_seed(seed)
    z = torch.randn((B, K + 1, V), generator=gen) * std
    zq = z[:, :K] + torch.randn((B, K, V), generator=gen) * near
    ld = ld or V
    p = torch.zeros((B, K + 1, ld), dtype=dtype)
    p[..., :V] = torch.softmax(z, -1)
    qs = torch.zeros((B, K, ld), dtype=dtype)
    qs[..., :V] = torch.softmax(zq, -1)
    ids = (zq + -torch.log(-torch.log(torch.rand((B, K, V), generator=gen).clamp(1e-9, 1 - 1e-7)))
           ).argmax(-1) if q else zq.argmax(-1)
    if ragged:
        length = torch.randint(0, K + 1, (B, 1), generator=gen)
        ids[torch.arange(K) >= length] = -1
    u = torch.rand((B, K + 1), generator=gen)
    return (p.cuda()[..., :V], ids.cuda(), u.cuda(), qs.cuda()[..., :V] if q else None)


def check_verify(p, ids, u, q=None, **kw):
    want = ref.verify(p, ids, u, q)
    got = fs.fs_verify(p, ids, u, q, **kw)
    assert torch.equal(got.accepted.cpu(), want[1])
    assert torch.equal(got.ids.cpu(), want[0])
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("q", [True, False])
@pytest.mark.parametrize("B,K,V,ld", [
    (1, 0, 1, 1), (3, 0, 50, 56), (2, 1, 7, 7), (5, 4, 1000, 1000), (1, 4, 151936, 151936),
    (9, 3, 4096, 4096), (2, 2, 262144, 262144), (64, 5, 1027, 1027), (400, 2, 300, 304),
    (2, 40, 2049, 2056), (3, 64, 33, 33), (1, 1024, 17, 17)])
def test_verify(B, K, V, ld, q, dtype):
    check_verify(*problem(B, K, V, dtype, q=q, ld=ld, seed=B + K + V))
    check_verify(*problem(B, K, V, dtype, q=q, ld=ld, seed=B + K + V + 1, ragged=True, std=6.0))


def test_verify_borders():
    """Sums that u hits exactly: the next id with a weight is drawn; accepted are drafts
    with u q < p, not those with u q = p."""
    p = torch.tensor([0.25, 0.0, 0.25, 0.0, 0.0, 0.5, 0.0]).cuda()
    u = torch.tensor([0.0, 0.2499, 0.25, 0.4999, 0.5, 0.75, 1 - 2.0 ** -24]).cuda()
    rows = p.expand(7, 1, 7)
    ids = torch.zeros((7, 0), dtype=torch.int64, device="cuda")
    got = check_verify(rows, ids, u.unsqueeze(1))
    assert got.ids[:, 0].tolist() == [0, 0, 2, 2, 5, 5, 5]
    q = torch.tensor([0.5, 0.0, 0.25, 0.0, 0.125, 0.125, 0.0]).cuda()
    ids = torch.tensor([[0], [0], [2], [2], [4], [1], [6], [5]]).cuda()
    u = torch.tensor([[0.5, 0.9], [0.4999, 0.9], [0.9999, 0.1], [0.0, 0.1], [0.0, 0.3], [0.0, 0.0],
                      [0.5, 0.5], [0.9999, 0.5]]).cuda()
    two = p.expand(8, 2, 7)
    got = check_verify(two, ids, u, q.expand(8, 1, 7))
    assert got.accepted.tolist() == [0, 1, 1, 1, 0, 0, 0, 1]
    assert got.ids[0].tolist() == [5, -1]  # only id 5 has p > q


def test_verify_numbers_outside():
    """u outside [0, 1) and NaN; ids at and past V and below 0; negative, infinite and NaN
    weights; rows without any weight; probabilities that are not normalised."""
    inf, nan = float("inf"), float("nan")
    p, ids, u, q = problem(12, 2, 500, torch.float32, seed=4)
    u[0], u[1], u[2] = nan, 1.0, -3.0
    u[3, 2], u[4, 2] = inf, -inf
    ids[5, 0], ids[6, 0], ids[7, 1] = 500, 2 ** 40, -(2 ** 40)
    p[8, :, 10:40], p[8, :, 50], p[8, :, 60] = -1.0, nan, inf
    q[9, :, :20], q[9, :, 30] = nan, inf
    p[10] = 0.0
    p[11] *= 1e20
    q[11] *= 1e20
    check_verify(p, ids, u, q)
    check_verify(p, ids, u)
    p[10] = nan
    got = check_verify(p, ids, u, q)
    assert got.ids[10, 0] == -1


def test_verify_falls_back_to_the_target():
    """A rejected draft where no p exceeds its q: the draw is from p."""
    p = torch.softmax(torch.randn((1, 1, 3000)), -1).cuda().expand(4, 3, 3000).contiguous()
    q = p[:, :2] * 1.5
    ids = torch.randint(0, 3000, (4, 2)).cuda()
    u = torch.full((4, 3), 0.99, device="cuda")
    u[:, 2] = torch.tensor([0.0, 0.3, 0.6, 0.95])
    got = check_verify(p, ids, u, q)
    assert got.accepted.tolist() == [0] * 4 and bool((got.ids[:, 0] >= 0).all())


def test_verify_reads_no_other_rows():
    """NaN in every row but the one that counts, and in q behind an acceptance."""
    p, ids, u, q = problem(40, 4, 1000, torch.float32, seed=6)
    want = check_verify(p, ids, u, q)
    x = ids.clamp_min(0).unsqueeze(2)
    dirty, dirty_q = torch.full_like(p, float("nan")), torch.full_like(q, float("nan"))
    rows = torch.arange(40, device="cuda")
    dirty[:, :4].scatter_(2, x, p[:, :4].gather(2, x))
    dirty_q.scatter_(2, x, q.gather(2, x))
    n = want.accepted
    dirty[rows, n] = p[rows, n]
    rejected = n < 4
    dirty_q[rows[rejected], n[rejected]] = q[rows[rejected], n[rejected]]
    got = fs.fs_verify(dirty, ids, u, dirty_q)
    assert torch.equal(got.ids, want.ids) and torch.equal(got.accepted, n)


def test_verify_strides_and_given_outputs():
    """Position-major probabilities, a shared row, drafts and numbers inside wider tensors."""
    p, ids, u, q = problem(6, 3, 700, torch.float32, seed=7)
    want = fs.fs_verify(p, ids, u, q)
    pt = p.transpose(0, 1).contiguous().transpose(0, 1)
    qt = q.transpose(0, 1).contiguous().transpose(0, 1)
    wide_ids = torch.full((6, 9), 3, device="cuda")
    wide_ids[:, 2:5] = ids
    wide_u = torch.zeros((6, 11), device="cuda")
    wide_u[:, 5:9] = u
    out = torch.full((6, 8), 77, device="cuda")
    accepted = torch.full((6,), 77, device="cuda")
    got = fs.fs_verify(pt, wide_ids[:, 2:5], wide_u[:, 5:9], qt, out_ids=out[:, 1:5],
                       out_accepted=accepted)
    assert torch.equal(out[:, 1:5], want.ids) and torch.equal(accepted, want.accepted)
    assert bool((out[:, 0] == 77).all()) and bool((out[:, 5:] == 77).all())
    assert got.accepted is accepted
    shared = p[:1, :1].expand(6, 4, 700)
    check_verify(shared, ids, u, q)


@pytest.mark.parametrize("B", [1, 2, 5, 20, 60, 150, 160])
def test_a_sequence_does_not_depend_on_the_batch(B):
    p, ids, u, q = problem(160, 2, 20000, torch.bfloat16, seed=9)
    whole = fs.fs_verify(p, ids, u, q)
    part = fs.fs_verify(p[:B], ids[:B], u[:B], q[:B])
    assert torch.equal(part.ids, whole.ids[:B])
    if B == 60:
        check_verify(p[:B], ids[:B], u[:B], q[:B])


def test_verify_refusals():
    p, ids, u, q = problem(3, 2, 50, torch.float32)
    bad = [
        lambda: fs.fs_verify(p.half(), ids, u, q), lambda: fs.fs_verify(p, ids, u, q.bfloat16()),
        lambda: fs.fs_verify(p, ids[:, :1], u, q), lambda: fs.fs_verify(p, ids, u[:, :2], q),
        lambda: fs.fs_verify(p, ids.int(), u, q), lambda: fs.fs_verify(p, ids, u.double(), q),
        lambda: fs.fs_verify(p, ids, u, q[:, :, :49]), lambda: fs.fs_verify(p[0], ids, u, q),
        lambda: fs.fs_verify(p, ids.cpu(), u, q), lambda: fs.fs_verify(p[:, :0], ids[:, :0], u),
        lambda: fs.fs_verify(p, ids, u, q, out_ids=torch.zeros((3, 2), dtype=torch.int64, device="cuda")),
        lambda: fs.fs_verify(p.transpose(1, 2), ids, u),
    ]
    for call in bad:
        with pytest.raises(fs.FsError) as e:
            call()
        assert e.value.status == fs.FS_ERR_INVALID_ARG
    r = fs.fs_verify(p[:0], ids[:0], u[:0], q[:0])
    assert r.ids.shape == (0, 3) and r.accepted.shape == (0,)


@pytest.mark.parametrize("with_q", [True, False])
def test_verified_tokens_are_the_targets(with_q):
    """First tokens of many sequences follow p whatever the drafter says, and second ones
    behind an acceptance follow the second row (chi-square)."""
    n, V = 20000, 24
    gen = torch.Generator().manual_seed(12)
    z = torch.randn((2, V), generator=gen)
    p = torch.softmax(z, -1).cuda()
    q = torch.softmax(z[:1] * 0.5 + torch.randn((1, V), generator=gen), -1).cuda()
    u = torch.rand((n, 3), generator=gen).cuda()
    if with_q:  # the drafter draws with a verification of nothing
        draft = fs.fs_verify(q.expand(n, 1, V), torch.zeros((n, 0), dtype=torch.int64, device="cuda"),
                             u[:, 2:].contiguous()).ids
        qs = q.expand(n, 1, V)
    else:
        draft, qs = torch.full((n, 1), int(p[0].argmax()), device="cuda"), None
    r = fs.fs_verify(p.expand(n, 2, V), draft, u[:, :2].contiguous(), qs)
    first = np.bincount(r.ids[:, 0].cpu().numpy(), minlength=V)
    assert chi_square_gof(first, p[0].double().cpu().numpy())[2] > 1e-4
    second = r.ids[r.accepted == 1, 1].cpu().numpy()
    assert len(second) > 2000
    assert chi_square_gof(np.bincount(second, minlength=V), p[1].double().cpu().numpy())[2] > 1e-4
    share = float(r.accepted.double().mean())
    want = float(torch.minimum(p[0], q[0]).sum()) if with_q else float(p[0].max())
    assert abs(share - want) < 5 * math.sqrt(0.25 / n)


def test_verify_streams_and_graphs():
    p, ids, u, q = problem(30, 3, 5000, torch.float32, seed=14)
    want = fs.fs_verify(p, ids, u, q)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = fs.fs_verify(p, ids, u, q, stream=stream)
    stream.synchronize()
    assert torch.equal(got.ids, want.ids)
    graph, us = torch.cuda.CUDAGraph(), u.clone()
    with torch.cuda.graph(graph):
        out = fs.fs_verify(p, ids, us, q)
    for seed in range(3):
        us.copy_(torch.rand((30, 4), generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        again = fs.fs_verify(p, ids, us, q)
        assert torch.equal(out.ids, again.ids) and torch.equal(out.accepted, again.accepted)
    for _ in range(50):
        assert torch.equal(fs.fs_verify(p, ids, u, q).ids, want.ids)


def test_offsets_past_32_bits():
    """Probabilities, their rows and logits that end past 2^32 elements."""
    B, K, V, ld = 3, 2, 1000, 1 << 30
    p, ids, u, q = problem(B, K, V, torch.bfloat16, seed=15)
    far = torch.empty((B * (K + 1) - 1) * ld + V, dtype=torch.bfloat16, device="cuda")
    far_p = far.as_strided((B, K + 1, V), (ld * (K + 1), ld, 1))
    far_p.copy_(p)
    want = check_verify(p, ids, u, q)
    assert torch.equal(fs.fs_verify(far_p, ids, u, q).ids, want.ids)
    assert torch.equal(fs.fs_verify(p, ids, u, far_p[:, :K]).ids,
                       fs.fs_verify(p, ids, u, p[:, :K]).ids)
    x = far.as_strided((B * (K + 1), V), (ld, 1))
    x.copy_(logits(B * (K + 1), V, torch.bfloat16, seed=16)[0])
    near = fs.fs_probs(x.contiguous(), out_dtype=torch.bfloat16)
    assert torch.equal(fs.fs_probs(x, out=x).contiguous(), near)


def test_a_very_long_row():
    """More elements than segments of 1024 hold: segments grow."""
    V = 1_300_001
    gen = torch.Generator(device="cuda").manual_seed(17)
    z = torch.randn((2, 2, V), generator=gen, device="cuda")
    p = fs.fs_probs(z.view(4, V)).unflatten(0, (2, 2))
    q = fs.fs_probs(z[:, 0] * 1.01).unflatten(0, (2, 1))
    ids = torch.tensor([[5], [V - 1]], device="cuda")
    for u in ([0.999, 0.3], [0.0, 0.9999], [1.0, 0.00001]):
        check_verify(p, ids, torch.tensor([u, u], device="cuda"), q)
    x = z.view(4, V)[:, :V]
    check_probs(x)


@pytest.mark.parametrize("shift", [0, 1])  # 16 bytes at a time, element by element
def test_sums_of_the_longest_segments(shift):
    """2^29 weights, of which every lane adds 16384: half of the row such that a plain gathering of
    what those lose is off by 2^-36.8 of them, half of it equal.  Uniform numbers whose target lies
    2^-44 to 2^-41 of the total from a border: the sums are held to 2^-45."""
    half, terms = 2 ** 28, 16384
    gen = torch.Generator().manual_seed(197)
    odd = torch.randint(0, 2 ** 23, (terms,), generator=gen) * 2 + 1
    down = torch.randint(0, 13, (terms,), generator=gen)
    units = odd << (12 - down)                                # of 2^-36
    lane = (odd.double() * 2.0 ** -24 * torch.exp2(-down.double())).float().cuda()
    buf = torch.empty(2 * half + shift, device="cuda")
    p = buf[shift:]
    p[:half] = lane.view(-1, 1, 4).expand(-1, 32, 4).reshape(-1).repeat(half // (32 * terms))
    p[half:] = 2.0 ** -4
    first, step = half // terms * int(units.sum()), 2 ** 32   # the half's sum, an equal weight
    total = first + half * step
    # target - first = (k total - first 2^24) / 2^24 for u = k 2^-24, in steps of 2^56 / 2^24
    k = np.arange(int(0.6 * 2 ** 24), int(0.98 * 2 ** 24), dtype=np.uint64)
    word = (1 << 64) - 1
    behind = (k * np.uint64(total & word) - np.uint64((first << 24) & word)) & np.uint64(2 ** 56 - 1)
    off = np.minimum(behind, np.uint64(2 ** 56) - behind).astype(np.float64) / 2 ** 24 / total
    k = k[(off > 2.0 ** -44) & (off < 2.0 ** -41)]
    k = k[::max(1, len(k) // 120)]
    want = [half + ((int(i) * total - (first << 24)) >> 56) for i in k]
    assert len(k) > 100
    u = torch.from_numpy(k.astype(np.float64) * 2.0 ** -24).float().cuda().unsqueeze(1)
    ids = torch.zeros((len(k), 0), dtype=torch.int64, device="cuda")
    got = fs.fs_verify(p.expand(len(k), 1, 2 * half), ids, u).ids[:, 0].tolist()
    assert got == want


@pytest.mark.parametrize("dtype", TYPES)
def test_long_rows_whatever_their_alignment(dtype):
    """Segments of 2048 and 4096 elements, as whole and element by element: the same ids."""
    for V in (1_300_001, 2_500_000):
        gen = torch.Generator(device="cuda").manual_seed(V)
        buf = torch.rand(V + 1, generator=gen, device="cuda").to(dtype)
        u = torch.rand((40, 1), generator=gen, device="cuda")
        ids = torch.zeros((40, 0), dtype=torch.int64, device="cuda")
        rows = [buf[:V].clone(), torch.cat([buf[:1], buf[:V]])[1:]]
        one, two = (fs.fs_verify(r.expand(40, 1, V), ids, u).ids for r in rows)
        assert torch.equal(one, two)
        sums = rows[0].double().cumsum(0)
        want = torch.searchsorted(sums, u[:, 0].double() * sums[-1], right=True)
        assert torch.equal(one[:, 0], want)


@pytest.mark.parametrize("call", [
    "fs.fs_quantize(x).scale", "fs.fs_matmul_fp8(*fs.fs_quantize(x), *fs.fs_quantize(w, 128))",
    "fs.fs_probs(w)", "fs.fs_verify(p, ids, u).ids"])
def test_first_calls_of_a_process_in_a_captured_graph(call):
    code = f"""
import sys
sys.path.insert(0, {ROOT!r})
import torch, lm_head_gumbel_gb300 as fs
gen = torch.Generator(device="cuda").manual_seed(1)
x = torch.randn((40, 30000), generator=gen, device="cuda")
w = torch.randn((300, 30000), generator=gen, device="cuda")
p = torch.rand((2, 3, 160000), generator=gen, device="cuda") * 1e-5
ids = torch.randint(0, 1000, (2, 2), generator=gen, device="cuda")
u = torch.rand((2, 3), generator=gen, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = {call}
graph.replay()
torch.cuda.synchronize()
assert torch.equal(out, {call})
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


# --------------------------------------------------------------------------- together
def test_a_step_of_speculative_decoding():
    """An 8-bit drafter's head proposes, the target's head scores, verification keeps: each
    operator against its own form on what the one before gave, in a captured graph too."""
    B, K, d, V = 6, 3, 200, 1500
    gen = torch.Generator().manual_seed(18)
    W = (torch.randn((V, d), generator=gen) * 0.2).bfloat16().cuda()
    head = fs.fs_quantize(W, 128)
    table = (torch.randn((V, d), generator=gen)).bfloat16().cuda()
    T = torch.tensor([1.0, 0.8, 0.0, 1.3, 0.6, 1.0]).cuda()
    u = torch.rand((2 * K + 1, B), generator=gen).cuda()
    start = torch.randint(0, V, (B,), generator=gen).cuda()
    none = torch.zeros((B, 0), dtype=torch.int64, device="cuda")

    def step():
        ids, q, x = [], [], start
        for i in range(K):
            logits = fs.fs_matmul_fp8(*fs.fs_quantize(fs.fs_embed(x, table)), *head,
                                      out_dtype=torch.float32, overlap_previous=True)
            row = fs.fs_probs(logits, temperature=T)
            x = fs.fs_verify(row.unsqueeze(1), none, u[i].unsqueeze(1)).ids[:, 0]
            q.append(row)
            ids.append(x)
        ids, q = torch.stack(ids, 1), torch.stack(q, 1)
        tokens = torch.cat([start.unsqueeze(1), ids], 1)
        H = fs.fs_embed(tokens.view(-1), table)
        p = fs.fs_probs((H.float() @ W.float().T), temperature=T.repeat_interleave(K + 1))
        p = p.unflatten(0, (B, K + 1))
        return q, ids, p, fs.fs_verify(p, ids, u[K:].T.contiguous(), q)

    q, ids, p, r = step()
    want = ref.verify(p, ids, u[K:].T, q)
    assert torch.equal(r.ids.cpu(), want[0]) and torch.equal(r.accepted.cpu(), want[1])
    # the drafter's rows, from the definition
    prev = torch.cat([start.unsqueeze(1), ids[:, :-1]], 1)
    A, sa = ref.quantize(table.cpu()[prev.cpu().view(-1)], 1)
    wv, ws = ref.quantize(W, 128)
    l, _ = ref.matmul(A, sa, wv, ws, torch.float32)
    want_q, _ = ref.probs(l, T.repeat_interleave(K), None, torch.float32)
    assert float((q.cpu().double().view(-1, V) - want_q).abs().max()) < 1e-4
    assert bool((r.accepted[2] == K) | (p[2, int(r.accepted[2])].max() == 1))  # a greedy sequence
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        _, ids2, _, r2 = step()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ids2, ids) and torch.equal(r2.ids, r.ids)


@pytest.mark.parametrize("q", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
def test_greedy_drafts_verify_as_greedy_decoding(dtype, q):
    """At T = 0 the accepted drafts are the leading ones that are the target's likeliest ids, and
    the token behind them is that id too: what greedy decoding of the target alone gives."""
    B, K, V = 64, 4, 3001
    gen = torch.Generator().manual_seed(41)
    target = torch.randint(-20, 21, (B, K + 1, V), generator=gen).float()  # equal largest ones too
    drafter = target[:, :K].clone()
    wrong = torch.rand((B, K), generator=gen) < 0.3
    drafter[wrong] = torch.randint(-20, 21, (int(wrong.sum()), V), generator=gen).float()
    zero = torch.zeros(B * (K + 1), device="cuda")
    p = fs.fs_probs(target.view(-1, V).to(dtype).cuda(), temperature=zero, out_dtype=dtype)
    qs = fs.fs_probs(drafter.view(-1, V).to(dtype).cuda(), temperature=zero[:B * K], out_dtype=dtype)
    none = torch.zeros((B * K, 0), dtype=torch.int64, device="cuda")
    u = torch.rand((B * K, 1), generator=gen).cuda()
    ids = fs.fs_verify(qs.unsqueeze(1), none, u).ids.view(B, K)
    lowest = torch.arange(V, 0, -1)
    likeliest = (torch.where(target == target.amax(-1, keepdim=True), lowest, 0)).argmax(-1)
    assert torch.equal(ids.cpu(), torch.where(
        drafter == drafter.amax(-1, keepdim=True), lowest, 0).argmax(-1))
    u = torch.rand((B, K + 1), generator=gen).cuda()
    r = fs.fs_verify(p.view(B, K + 1, V), ids, u, qs.view(B, K, V) if q else None)
    n = (ids.cpu() == likeliest[:, :K]).long().cumprod(1).sum(1)
    assert 0 < int((n == K).sum()) < B and int((n == 0).sum()) > 0
    assert torch.equal(r.accepted.cpu(), n)
    at = torch.arange(K + 1)
    assert torch.equal(r.ids.cpu(), torch.where(at <= n.unsqueeze(1), likeliest, -1))
