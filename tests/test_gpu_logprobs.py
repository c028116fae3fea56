"""Token log-probabilities, entropy, alternatives and their gradient on the GPU
against 64-bit forms, within the bounds derived in vocab_ref.py; alternatives'
ids are compared exactly."""
import math

import pytest
import torch

import lm_head_gumbel_gb300 as fs
from lm_head_gumbel_gb300 import workloads as wl
import vocab_ref as ref
from gpu_cases import assert_no_device_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fs.load_library()
    yield
    assert_no_device_error()


def padded(t):
    """The same matrix with rows at a stride of 8 elements more than needed."""
    n, d = t.shape
    out = torch.full((n, (d + 7) // 8 * 8 + 8), 7.0, dtype=t.dtype, device=t.device)
    out[:, :d] = t
    return out[:, :d]


def problem(B, d, V, *, T=None, mask_frac=0.0, seed=0):
    H = padded(wl.make_hidden(B, d, seed=10 + seed, device="cuda"))
    W = padded(wl.make_weights(d, V, seed=20 + seed, device="cuda"))
    gen = torch.Generator().manual_seed(30 + seed)
    tokens = torch.randint(0, V, (B,), generator=gen)
    temp = None
    if T == "rows":
        temp = torch.rand(B, generator=gen) + 0.5
        temp[::3] = 0.0  # greedy rows are scored at T = 1
        temp = temp.cuda()
    elif T is not None:
        temp = torch.full((B,), float(T), device="cuda")
    mask = wl.make_mask(B, V, mask_frac, seed=40 + seed, device="cuda") if mask_frac else None
    return dict(H=H, W=W, tokens=tokens.cuda(), temperature=temp, vocab_mask=mask)


def near(got, want, bound, what):
    got, want = got.detach().cpu().double(), want.double()
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), what
    off = (got - want).abs()[~inf]
    assert not torch.isnan(off).any(), what
    bound = bound if not torch.is_tensor(bound) else bound[~inf]
    assert bool((off <= bound).all()), (what, float(off.max()), float((off / bound).max()))


def check_forward(p, K, **kw):
    r = fs.fs_logprobs(p["H"], p["W"], p["tokens"], K, temperature=p["temperature"],
                       vocab_mask=p["vocab_mask"], **kw)
    w = ref.forward(p["H"], p["W"], p["tokens"], K, p["temperature"], p["vocab_mask"],
                    kw.get("vocab_offset", 0))
    near(r.lse, w["lse"], w["e_lse"], "lse")
    near(r.entropy, w["entropy"], w["e_entropy"], "entropy")
    near(r.logp, w["logp"], w["e_lse"] + 2 * ref.U * w["logp"].abs(), "logp")
    if K:
        assert torch.equal(r.topk_idx.cpu(), w["topk_idx"])
        near(r.topk_logp, w["topk_logp"], w["e_lse"] + 2 * ref.U * w["topk_logp"].abs(),
             "topk_logp")
    return r, w


# One row to several launches; one vocabulary block to several per worker; k
# slices, tiles, 16-byte vectors and mask words that end early.
SHAPES = [(1, 8, 1), (1, 64, 100), (2, 3, 33), (3, 100, 257), (5, 320, 1000), (64, 256, 4096),
          (128, 72, 513), (129, 64, 300), (257, 129, 511), (300, 264, 1003), (700, 72, 2001),
          (1300, 64, 600), (4, 128, 40001), (140, 64, 20011)]


@pytest.mark.parametrize("B,d,V", SHAPES)
@pytest.mark.parametrize("K", [0, 3, 20])
def test_forward(B, d, V, K):
    check_forward(problem(B, d, V, T="rows", seed=B + V + K), K)


@pytest.mark.parametrize("B,d,V", [(5, 64, 1000), (130, 64, 700)])
@pytest.mark.parametrize("K", [1, 2, 4, 5, 16, 19])
def test_every_list_capacity(B, d, V, K):
    check_forward(problem(B, d, V, T=0.7, seed=K), K)


@pytest.mark.parametrize("B,d,V", [(3, 100, 257), (128, 72, 513), (300, 264, 1003)])
@pytest.mark.parametrize("frac", [0.05, 0.97])
def test_masks(B, d, V, frac):
    p = problem(B, d, V, T="rows", mask_frac=frac, seed=V)
    p["vocab_mask"][0] = 0                      # a row that allows nothing
    p["vocab_mask"][1] = 0
    p["vocab_mask"][1, 2] = 1 << 5              # a row that allows one id
    p["tokens"][1] = 69
    r, w = check_forward(p, 20)
    assert r.lse[0].item() == -math.inf and r.entropy[0].item() == 0.0
    assert r.logp[0].item() == -math.inf and bool((r.topk_idx[0] == -1).all())
    assert r.entropy[1].item() == 0.0 and r.topk_idx[1, 0].item() == 69
    assert abs(r.logp[1].item()) <= w["e_lse"]


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, 3e38])
def test_values_behind_the_mask_change_nothing(bad):
    p = problem(6, 96, 700, mask_frac=0.1, seed=5)
    gone = torch.tensor([0, 31, 32, 255, 256, 699], device="cuda")
    for v in gone.tolist():
        word = ~torch.tensor(1 << (v % 32), dtype=torch.int64).to(torch.int32)
        p["vocab_mask"][:, v // 32] &= word.cuda()
    want = fs.fs_logprobs(p["H"], p["W"], p["tokens"], 20, vocab_mask=p["vocab_mask"])
    p["W"][gone] = bad
    got = fs.fs_logprobs(p["H"], p["W"], p["tokens"], 20, vocab_mask=p["vocab_mask"])
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_non_finite_logits_of_allowed_ids():
    p = problem(4, 64, 500, seed=6)
    p["H"][1, 3] = math.nan
    p["W"][77] = -math.inf
    p["H"][:, :] = p["H"].abs()      # every logit of id 77 is -inf, but row 1's (NaN)
    p["tokens"][:] = torch.tensor([77, 5, 6, 7], device="cuda")
    r = fs.fs_logprobs(p["H"], p["W"], p["tokens"], 5)
    assert bool(torch.isnan(r.lse[1])) and bool(torch.isnan(r.entropy[1]))
    assert bool(torch.isnan(r.logp[1]))
    ok = [0, 2, 3]
    assert bool(torch.isfinite(r.lse[ok]).all()) and bool(torch.isfinite(r.entropy[ok]).all())
    assert r.logp[0].item() == -math.inf
    assert not bool((r.topk_idx[ok] == 77).any())
    p["W"][78] = math.inf            # and one of +inf
    r = fs.fs_logprobs(p["H"], p["W"], p["tokens"], 5)
    assert bool(torch.isnan(r.lse).all()) and bool(torch.isnan(r.topk_logp[ok]).all())
    assert bool((r.topk_idx[ok, 0] == 78).all())


def test_special_tokens_and_shards():
    """-1: no token.  A vocabulary in three shards: lse and alternatives join to
    the whole call's, and a token's log-probability is its shard's."""
    p = problem(9, 128, 1500, T=0.8, seed=8)
    p["tokens"][2] = -1
    p["tokens"][3] = -100
    whole, _ = check_forward(p, 8)
    assert whole.logp[2].item() == 0.0 and whole.logp[3].item() == 0.0
    parts, lo = [], 0
    for hi in (512, 611, 1500):
        q = dict(p, W=p["W"][lo:hi])
        parts.append(check_forward(q, 8, vocab_offset=lo)[0])
        lo = hi
    lse = torch.logsumexp(torch.stack([r.lse.double() for r in parts]), 0)
    assert bool(((lse - whole.lse).abs() < 1e-5).all())
    logp = torch.stack([r.logp.double() + r.lse - lse for r in parts]).max(0).values
    named = p["tokens"] >= 0
    assert bool(((logp - whole.logp).abs()[named] < 1e-5).all())
    ids = torch.cat([r.topk_idx for r in parts], 1)
    val = torch.cat([r.topk_logp.double() + (r.lse - lse).unsqueeze(1) for r in parts], 1)
    at = val.sort(dim=1, descending=True, stable=True).indices[:, :8]
    assert torch.equal(ids.gather(1, at), whole.topk_idx)
    r = fs.fs_logprobs(p["H"], p["W"], torch.full_like(p["tokens"], 1500))
    assert bool((r.logp == -math.inf).all())


def test_ties_go_to_the_lower_id():
    """Equal logits everywhere, and copies of the best row in other tiles."""
    p = problem(130, 64, 5000, seed=9)
    zero = torch.zeros_like(p["H"])
    r = fs.fs_logprobs(zero, p["W"], p["tokens"], 20)
    assert torch.equal(r.topk_idx.cpu(), torch.arange(20).expand(130, 20))
    near(r.entropy, torch.full((130,), math.log(5000.0), dtype=torch.float64), 1e-4, "entropy")
    W = p["W"]
    W[:] = W * 0.25
    best = 2 * p["H"][7].clone()
    at = torch.arange(130, 4990, 37)          # 132 equal rows, best for row 7
    W[at.cuda()] = best
    r = fs.fs_logprobs(p["H"], W, p["tokens"], 20)
    assert torch.equal(r.topk_idx[7].cpu(), at[:20])
    one = fs.fs_logprobs(p["H"][7:8], W, p["tokens"][7:8], 20)  # the single-CTA kernel
    assert torch.equal(one.topk_idx[0].cpu(), at[:20])


def test_near_ties_rank_by_exact_logit():
    """24 ids whose logits differ by less than fp32 resolves at their size: in
    64 bits the order is known by construction."""
    d, V = 512, 3000
    gen = torch.Generator().manual_seed(3)
    h = torch.ones(1, d)
    W = (torch.randn((V, d), generator=gen) * 0.01).bfloat16()
    ids = torch.randperm(V, generator=gen)[:24]
    for j, v in enumerate(ids.tolist()):
        W[v] = 8.0                            # the logit is 4096 but for
        W[v, 100] = 8.0 + 0.0625 * (j % 2)    # coarse steps
        W[v, 7] = 2.0 ** -16 * (24 - j)       # and steps of 2^-16, an ulp of 4088 being 2^-12
    H = h.bfloat16().cuda()
    tokens = torch.zeros(1, dtype=torch.int64, device="cuda")
    r = fs.fs_logprobs(H, W.cuda(), tokens, 20)
    l = W.double().sum(1)
    want = sorted(range(V), key=lambda v: (-l[v].item(), v))[:20]
    assert r.topk_idx[0].tolist() == want
    assert len(set(l[ids].float().tolist())) < 24


def test_same_results_on_other_streams_in_graphs_and_overlapped():
    p = problem(200, 128, 3000, T="rows", mask_frac=0.05, seed=11)
    args = dict(temperature=p["temperature"], vocab_mask=p["vocab_mask"])
    want = fs.fs_logprobs(p["H"], p["W"], p["tokens"], 10, **args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = fs.fs_logprobs(p["H"], p["W"], p["tokens"], 10, **args)
    again = fs.fs_logprobs(p["H"], p["W"], p["tokens"], 10, stream=side, **args)
    side.synchronize()
    for r in (got, again):
        assert all(torch.equal(a, b) for a, b in zip(r, want))
    # H written by the kernel before, on the same stream
    for rows in (200, 64):
        w2 = fs.fs_logprobs(p["H"][:rows], p["W"], p["tokens"][:rows], 10,
                            temperature=p["temperature"][:rows], vocab_mask=p["vocab_mask"][:rows])
        for _ in range(5):
            H2 = torch.empty_like(p["H"][:rows])
            H2.copy_(p["H"][:rows])
            r = fs.fs_logprobs(H2, p["W"], p["tokens"][:rows], 10, overlap_previous=True,
                               temperature=p["temperature"][:rows],
                               vocab_mask=p["vocab_mask"][:rows])
            assert all(torch.equal(a, b) for a, b in zip(r, w2))
    ws = torch.empty(fs.fs_logprobs_workspace_size(200, 3000, 10), dtype=torch.uint8,
                     device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = fs.fs_logprobs(p["H"], p["W"], p["tokens"], 10, workspace=ws, **args)
    for _ in range(3):
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_rows_do_not_depend_on_the_batch():
    """Alternatives of a row are the same alone, in a batch and in a large one."""
    p = problem(600, 256, 9000, seed=12)
    big = fs.fs_logprobs(p["H"], p["W"], p["tokens"], 20)
    for rows in (1, 100, 300):
        r = fs.fs_logprobs(p["H"][:rows], p["W"], p["tokens"][:rows], 20)
        assert torch.equal(r.topk_idx, big.topk_idx[:rows])


def test_logp_agrees_with_the_sampler():
    """The token that greedy sampling picks is the first alternative."""
    p = problem(33, 256, 5000, seed=13)
    ids = fs.fs_sample(p["H"], p["W"], temperature=torch.zeros(33, device="cuda"))
    r = fs.fs_logprobs(p["H"], p["W"], ids, 2)
    gap = (r.topk_logp[:, 0] - r.topk_logp[:, 1]) > 1e-2
    assert int(gap.sum()) > 20
    assert torch.equal(r.topk_idx[gap, 0], ids[gap])
    assert torch.equal(r.logp[gap], r.topk_logp[gap, 0])


# --------------------------------------------------------------------------- gradient
def upstream(B, entropy, seed):
    gen = torch.Generator().manual_seed(50 + seed)
    a = torch.randn(B, generator=gen).cuda()
    e = torch.randn(B, generator=gen).cuda() if entropy else None
    return a, e


def check_gradient(p, a, e, **kw):
    f = fs.fs_logprobs(p["H"], p["W"], p["tokens"], temperature=p["temperature"],
                       vocab_mask=p["vocab_mask"])
    dH, dW = fs.fs_logprobs_grad(p["H"], p["W"], p["tokens"], f.lse, a,
                                 entropy=f.entropy if e is not None else None, grad_entropy=e,
                                 temperature=p["temperature"], vocab_mask=p["vocab_mask"], **kw)
    wH, bH, wW, bW, G = ref.gradient(p["H"], p["W"], p["tokens"], a, e, p["temperature"],
                                     p["vocab_mask"])
    if dH is not None:
        near(dH, wH, bH, "dH")
    if dW is not None:
        near(dW, wW, bW, "dW")
    return dH, dW, wH, bH, wW, bW


@pytest.mark.parametrize("B,d,V", SHAPES)
@pytest.mark.parametrize("entropy", [False, True])
def test_gradient(B, d, V, entropy):
    p = problem(B, d, V, T="rows", seed=B + V)
    check_gradient(p, *upstream(B, entropy, V))


@pytest.mark.parametrize("B,d,V", [(3, 100, 257), (128, 72, 513), (300, 264, 1003)])
def test_gradient_with_masks(B, d, V):
    p = problem(B, d, V, T="rows", mask_frac=0.3, seed=V)
    p["vocab_mask"][0] = 0
    p["vocab_mask"][1] = 0
    p["vocab_mask"][1, 2] = 1 << 5
    p["tokens"][1] = 69
    p["tokens"][2] = -1
    dH, dW, *_ = check_gradient(p, *upstream(B, True, V))
    assert bool((dH[0] == 0).all())


def test_gradient_against_differences():
    """Along a random direction, the 64-bit loss's central difference."""
    p = problem(7, 40, 300, T=0.9, mask_frac=0.1, seed=14)
    a, e = upstream(7, True, 14)
    dH, dW, wH, bH, wW, bW = check_gradient(p, a, e)
    gen = torch.Generator().manual_seed(15)
    H, W = p["H"].cpu().double(), p["W"].cpu().double()
    held = ref.forward(H, W, p["tokens"], 0, p["temperature"], p["vocab_mask"])["held"]

    def loss(Hx, Wx):
        f = ref.forward(Hx, Wx, p["tokens"], 0, p["temperature"], p["vocab_mask"])
        lp = torch.where(held, f["logp"], 0.0)
        return float((a.cpu().double() * lp).sum() + (e.cpu().double() * f["entropy"]).sum())

    h = 1e-5
    for which, (g, bound) in enumerate(((dH, bH), (dW, bW))):
        D = torch.randn(g.shape, generator=gen, dtype=torch.float64)
        step = [(D * h, 0.0), (0.0, D * h)][which]
        diff = (loss(H + step[0], W + step[1]) - loss(H - step[0], W - step[1])) / (2 * h)
        got = float((g.cpu().double() * D).sum())
        # the elementwise bounds, and the difference's own error (h^2, 1e-16/h)
        assert abs(got - diff) <= float((bound * D.abs()).sum()) + 1e-6 * abs(diff) + 1e-8


def test_gradient_of_shards_adds_up():
    p = problem(6, 72, 900, T=0.8, seed=16)
    a, e = upstream(6, True, 16)
    f = fs.fs_logprobs(p["H"], p["W"], p["tokens"], temperature=p["temperature"])
    wH, bH, wW, bW, _ = ref.gradient(p["H"], p["W"], p["tokens"], a, e, p["temperature"])
    total = torch.zeros(6, 72, dtype=torch.float64)
    rounding = torch.zeros(6, 72, dtype=torch.float64)
    lo = 0
    for hi in (128, 131, 900):
        dH, dW = fs.fs_logprobs_grad(p["H"], p["W"][lo:hi], p["tokens"], f.lse, a,
                                     entropy=f.entropy, grad_entropy=e,
                                     temperature=p["temperature"], vocab_offset=lo)
        near(dW, wW[lo:hi], bW[lo:hi], "dW")
        total += dH.cpu().double()
        rounding += dH.cpu().double().abs() * ref.BF16 * 2  # each shard's own result
        lo = hi
    assert bool(((total - wH).abs() <= bH + rounding).all())


def test_gradient_parts_and_given_outputs():
    """dH or dW alone, into given strided outputs, leave everything else alone."""
    p = problem(70, 100, 1000, seed=17)
    a, _ = upstream(70, False, 17)
    dH, dW, *_ = check_gradient(p, a, None)
    bufH = torch.full((72, 112), 3.0, dtype=torch.bfloat16, device="cuda")
    bufW = torch.full((1002, 112), 3.0, dtype=torch.bfloat16, device="cuda")
    f = fs.fs_logprobs(p["H"], p["W"], p["tokens"])
    r = fs.fs_logprobs_grad(p["H"], p["W"], p["tokens"], f.lse, a, out_dH=bufH[:70, :100],
                            need_dW=False)
    assert r[1] is None and torch.equal(bufH[:70, :100], dH)
    r = fs.fs_logprobs_grad(p["H"], p["W"], p["tokens"], f.lse, a, out_dW=bufW[:1000, :100],
                            need_dH=False)
    assert r[0] is None and torch.equal(bufW[:1000, :100], dW)
    for buf, n in ((bufH, 70), (bufW, 1000)):
        assert bool((buf[n:] == 3.0).all()) and bool((buf[:, 100:] == 3.0).all())


def test_gradient_in_a_graph_and_on_a_stream():
    p = problem(300, 136, 2000, T="rows", seed=18)
    a, e = upstream(300, True, 18)
    f = fs.fs_logprobs(p["H"], p["W"], p["tokens"], temperature=p["temperature"])
    call = dict(entropy=f.entropy, grad_entropy=e, temperature=p["temperature"])
    want = fs.fs_logprobs_grad(p["H"], p["W"], p["tokens"], f.lse, a, **call)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = fs.fs_logprobs_grad(p["H"], p["W"], p["tokens"], f.lse, a, stream=side, **call)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    ws = torch.empty(fs.fs_logprobs_grad_workspace_size(300, 136, 2000), dtype=torch.uint8,
                     device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fs.fs_logprobs_grad(p["H"], p["W"], p["tokens"], f.lse, a, workspace=ws, **call)
    for _ in range(3):
        ws.fill_(255)  # NaN in bf16: nothing unwritten is read
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_binding_refusals():
    p = problem(4, 64, 500, seed=19)
    f = fs.fs_logprobs(p["H"], p["W"], p["tokens"])
    bad = [
        lambda: fs.fs_logprobs(p["H"].float(), p["W"], p["tokens"]),
        lambda: fs.fs_logprobs(p["H"], p["W"][:, :32], p["tokens"]),
        lambda: fs.fs_logprobs(p["H"], p["W"], p["tokens"][:3]),
        lambda: fs.fs_logprobs(p["H"], p["W"], p["tokens"].int()),
        lambda: fs.fs_logprobs(p["H"], p["W"], p["tokens"].cpu()),
        lambda: fs.fs_logprobs(p["H"], p["W"], p["tokens"], 21),
        lambda: fs.fs_logprobs(p["H"], p["W"], p["tokens"], temperature=torch.ones(4).cuda().double()),
        lambda: fs.fs_logprobs(p["H"], p["W"], p["tokens"],
                               vocab_mask=torch.zeros((4, 15), dtype=torch.int32, device="cuda")),
        lambda: fs.fs_logprobs(p["H"], p["W"], p["tokens"], 4,
                               out_topk_idx=torch.zeros((4, 5), dtype=torch.int64, device="cuda")),
        lambda: fs.fs_logprobs(p["H"], p["W"], p["tokens"],
                               workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
        lambda: fs.fs_logprobs_grad(p["H"], p["W"], p["tokens"], f.lse, f.lse, grad_entropy=f.lse),
        lambda: fs.fs_logprobs_grad(p["H"], p["W"], p["tokens"], f.lse, f.lse, need_dH=False,
                                    need_dW=False),
        lambda: fs.fs_logprobs_grad(p["H"], p["W"], p["tokens"], f.lse.double(), f.lse),
        lambda: fs.fs_logprobs_grad(p["H"], p["W"], p["tokens"], f.lse, f.lse,
                                    out_dH=torch.empty((4, 65), dtype=torch.bfloat16, device="cuda")),
    ]
    for call in bad:
        with pytest.raises(fs.FsError):
            call()


# --------------------------------------------------------------------------- sizes at which the work is cut differently
@pytest.mark.parametrize("B,V", [(3, 9728), (3, 9729), (70, 19456), (70, 19457), (128, 38912),
                                 (5, 39000), (129, 40000)])
@pytest.mark.parametrize("K", [0, 5])
def test_unit_widths(B, V, K):
    """Units of 64, 128 and 256 ids, one per CTA and more; ragged k slices in a stage."""
    check_forward(problem(B, 200, V, T="rows", mask_frac=0.02, seed=V + B), K)


@pytest.mark.parametrize("K", [8, 12, 13, 20])
def test_more_list_capacities(K):
    check_forward(problem(6, 128, 45000, T=0.9, seed=60 + K), K)
    check_forward(problem(150, 64, 5000, T=0.9, seed=61 + K), K)


@pytest.mark.parametrize("B", [127, 128, 129, 256, 257, 1280, 1281, 1537])
def test_rows_per_launch(B):
    check_forward(problem(B, 32, 300, T="rows", seed=B), 3)


@pytest.mark.parametrize("B,d,V", [(9, 2492, 300), (2, 8, 5000), (260, 40, 3000), (130, 520, 129),
                                   (16, 72, 19457), (6, 1200, 1940), (130, 260, 4096),
                                   (300, 520, 2000), (60, 300, 11137), (128, 264, 5281)])
def test_gradient_splits(B, d, V):
    """dH with and without splits, singles and pairs, narrow and wide units."""
    p = problem(B, d, V, T="rows", mask_frac=0.02, seed=B + d)
    check_gradient(p, *upstream(B, True, V))


def test_log_probabilities_are_at_most_zero():
    """Rows whose mass is on one token, by 20 to 200 units of logit."""
    p = problem(64, 64, 3000, seed=70)
    p["W"][:64] = (p["H"] * torch.linspace(0.3, 3.0, 64, device="cuda").unsqueeze(1)).bfloat16()
    p["tokens"][:] = torch.arange(64, device="cuda")
    r, _ = check_forward(p, 4)
    assert bool((r.logp <= 0).all()) and bool((r.topk_logp <= 0).all())
    assert bool((r.logp[-1] > -1e-6).all())


def test_few_rows_at_low_temperature():
    """What the accumulator's truncation would show in: one row, a long k, T = 0.5.
    The bound is fp32's own for sums of this length, not vocab_ref's (16 products
    cut off at a time): 4 u sqrt(d/16) of the logits' size, and 4 u of lse's."""
    p = problem(3, 4096, 20000, T=0.5, seed=71)
    r = fs.fs_logprobs(p["H"], p["W"], p["tokens"], 20, temperature=p["temperature"])
    w = ref.forward(p["H"], p["W"], p["tokens"], 20, p["temperature"])
    size = float((w["topk_logp"] + w["lse"].unsqueeze(1)).abs().max())
    bound = 4 * ref.U * math.sqrt(4096 / 16) * size + 4 * ref.U * float(w["lse"].abs().max())
    near(r.lse, w["lse"], bound, "lse")
    near(r.topk_logp, w["topk_logp"], bound + 2 * ref.U * w["topk_logp"].abs(), "topk_logp")


@pytest.mark.parametrize("B,d,V,tokens", [
    (2, 520, 2000, "one"), (60, 516, 2000, "one"), (128, 520, 700, "few"), (200, 520, 2000, "few"),
    (300, 1000, 500, "rows"), (5, 520, 20000, "one"), (700, 520, 3000, "rows"),
    (150, 520, 40000, "one"), (1500, 264, 700, "few"), (1100, 272, 900, "rows")])
def test_gradient_has_no_rounding_bias_at_the_token(B, d, V, tokens):
    """Upstream gradients that bf16 rounds the furthest, all the same way: the
    rounding of the results (u = 2^-8 at most, either way) averages out along a
    row, one of the token's factor would not.  Small logits, so that the token's
    term is nearly all of its rows; "few" and "one": many rows share a token."""
    p = problem(B, d, V, seed=B + V)
    p["H"].mul_(1 / 64)
    n = {"one": 1, "few": 3, "rows": V}[tokens]
    gen = torch.Generator().manual_seed(B)
    p["tokens"] = (torch.randint(0, n, (B,), generator=gen) * 37 % V).cuda()
    p["vocab_mask"] = None
    f = fs.fs_logprobs(p["H"], p["W"], p["tokens"])
    # G at the token, a (1 - P), close to 1 + 2^-8: half a step above 1.
    a = (1 + 2.0 ** -8 - 2.0 ** -14) / (1 - f.logp.exp())
    dH, dW, wH, _, wW, _ = check_gradient(p, a, None)
    held = torch.unique(p["tokens"]).cpu()
    for got, want in ((dH.cpu().double(), wH), (dW.cpu().double()[held], wW[held])):
        bias = ((got - want) * want).sum(1) / (want * want).sum(1)
        # 8 deviations of a mean of d roundings (weights want^2: 3 d^-1 for normal
        # values), and the other ids' elements of G, a/V each: 2^-8 / sqrt(V) a row.
        limit = 8 * 2.0 ** -8 / math.sqrt(3) * math.sqrt(3 / d) + 2 * 2.0 ** -8 / math.sqrt(V)
        assert limit < 2.0 ** -8 * 0.6
        assert float(bias.abs().max()) < limit


# --------------------------------------------------------------------------- offsets past 32 bits
def far_apart(t, ld):
    """The same matrix with rows at stride ld (what lies between is never touched)."""
    out = torch.empty((t.shape[0] - 1) * ld + t.shape[1], dtype=t.dtype, device=t.device)
    out = torch.as_strided(out, t.shape, (ld, 1))
    out.copy_(t)
    return out


def test_row_strides_past_32_bits():
    """H and W, and dH and dW, of more than 2^32 elements from first to last."""
    for B, V, ldh, ldw in ((4, 40000, 64, 1 << 17), (300, 700, 1 << 24, 64)):
        p = problem(B, 64, V, seed=80)
        p["H"], p["W"] = far_apart(p["H"], ldh), far_apart(p["W"], ldw)
        p["tokens"][-1] = V - 1
        check_forward(p, 3)
        out_dH = far_apart(torch.zeros_like(p["H"]), ldh)
        out_dW = far_apart(torch.zeros_like(p["W"]), ldw)
        check_gradient(p, *upstream(B, True, V), out_dH=out_dH, out_dW=out_dW)
        del p, out_dH, out_dW
        torch.cuda.empty_cache()


def test_gradient_whose_logits_pass_32_bits():
    """B V > 2^32; dH and dW compared at the first, some and the last rows."""
    B, d, V = 33000, 32, 131200
    gen = torch.Generator(device="cuda").manual_seed(81)
    H = torch.randn(B, d, generator=gen, device="cuda").bfloat16()
    W = (torch.randn(V, d, generator=gen, device="cuda") * 0.3).bfloat16()
    t = torch.randint(0, V, (B,), generator=gen, device="cuda")
    t[-1], t[-2] = V - 1, 0
    a = torch.randn(B, generator=gen, device="cuda")
    f = fs.fs_logprobs(H, W, t)
    dH, dW = fs.fs_logprobs_grad(H, W, t, f.lse, a)
    rows = torch.cat([torch.randint(0, B, (6,), generator=gen, device="cuda"),
                      torch.tensor([0, B - 2, B - 1], device="cuda")])
    ids = torch.cat([torch.randint(0, V, (6,), generator=gen, device="cuda"),
                     torch.tensor([0, V - 2, V - 1], device="cuda"), t[rows]])
    Hd, Wd = H.double(), W.double()
    l = Hd[rows] @ Wd.T
    lse = torch.logsumexp(l, 1)
    # Bounds as in vocab_ref, from these rows' and ids' own magnitudes.
    e_l = (d / 16 + 1) * 2.0 ** -23 * float((Hd.abs() @ Wd.abs().max(0).values).max())
    e_lse = (e_l + 4 * ref.U * float(l.abs().max()) / math.log(2) + 2.0 ** -22
             + (700 + V / 64) * ref.U + 4 * ref.U * float(lse.abs().max()))
    near(f.lse[rows], lse.cpu(), e_lse, "lse")

    def compare(got, p, hot, scale, other, terms, what):
        G, mag = scale * (hot - p), scale.abs() * (hot + p)
        want = G @ other
        dG = (ref.BF16 * G.abs() + mag * (4 * e_lse + 8 * ref.U)) * (1 + ref.BF16)
        bound = dG @ other.abs() + (terms / 16 + 64) * 2.0 ** -23 * (G.abs() @ other.abs())
        near(got, want.cpu(), (bound * (1 + ref.BF16) + ref.BF16 * want.abs()).cpu(), what)

    hot = torch.zeros_like(l).scatter_(1, t[rows].unsqueeze(1), 1.0)
    compare(dH[rows], (l - lse.unsqueeze(1)).exp(), hot, a[rows].double().unsqueeze(1), Wd, V, "dH")
    p = (Wd[ids] @ Hd.T - f.lse.double()).exp()  # lse's own error is in the bound
    hot = (ids.unsqueeze(1) == t.unsqueeze(0)).double()
    compare(dW[ids], p, hot, a.double(), Hd, B, "dW")


# --------------------------------------------------------------------------- masks' row strides
def test_masks_whose_rows_overlap_are_refused():
    """One row of allow-bits expanded to all rows, and rows closer than their words:
    the library has no stride for the first and must not make one up."""
    B, V = 4, 500
    p = problem(B, 64, V, mask_frac=0.1, seed=90)
    words = p["vocab_mask"].shape[1]
    flat = p["vocab_mask"].reshape(-1)
    f = fs.fs_logprobs(p["H"], p["W"], p["tokens"])
    for mask in (p["vocab_mask"][:1].expand(B, -1),
                 torch.as_strided(flat, (B, words), (words - 1, 1))):
        with pytest.raises(fs.FsError):
            fs.fs_logprobs(p["H"], p["W"], p["tokens"], vocab_mask=mask)
        with pytest.raises(fs.FsError):
            fs.fs_logprobs_grad(p["H"], p["W"], p["tokens"], f.lse, f.lse, vocab_mask=mask)


def test_masks_of_other_row_strides():
    """Rows further apart than their words, rows wider than the vocabulary needs, a
    single row out of an expanded mask: the same results."""
    B, V = 5, 500
    p = problem(B, 64, V, T="rows", mask_frac=0.3, seed=91)
    want, _ = check_forward(p, 4)
    mask = p["vocab_mask"]
    wide = torch.full((B, mask.shape[1] + 7), -1, dtype=torch.int32, device="cuda")
    wide[:, :mask.shape[1]] = mask
    for m in (wide, wide[:, :mask.shape[1]], wide[:, :mask.shape[1] + 3]):
        got = fs.fs_logprobs(p["H"], p["W"], p["tokens"], 4, temperature=p["temperature"],
                             vocab_mask=m)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    one = fs.fs_logprobs(p["H"][:1], p["W"], p["tokens"][:1], 4, temperature=p["temperature"][:1],
                         vocab_mask=mask[:1].expand(3, -1)[:1])
    first = fs.fs_logprobs(p["H"][:1], p["W"], p["tokens"][:1], 4,
                           temperature=p["temperature"][:1], vocab_mask=mask[:1])
    assert all(torch.equal(a, b) for a, b in zip(one, first))


# --------------------------------------------------------------------------- memory of the stream's own
def pool_of(t):
    """The stream whose blocks of the caching allocator `t` lies in."""
    at = t.data_ptr()
    for segment in torch.cuda.memory_snapshot():
        if segment["address"] <= at < segment["address"] + segment["total_size"]:
            return segment["stream"]
    raise AssertionError("not the allocator's")


def test_results_and_workspaces_belong_to_the_given_stream():
    """Results lie in the given stream's blocks, whether it is given as a stream, a
    handle or 0; the workspace does too: nothing is taken from the current
    stream's blocks, where it could be handed out again while the kernels run."""
    p = problem(200, 128, 3000, seed=92)
    side = torch.cuda.Stream()
    f = fs.fs_logprobs(p["H"], p["W"], p["tokens"])
    torch.cuda.synchronize()
    for stream, owner in ((side, side.cuda_stream), (side.cuda_stream, side.cuda_stream), (0, 0)):
        r = fs.fs_logprobs(p["H"], p["W"], p["tokens"], 3, stream=stream)
        g = fs.fs_logprobs_grad(p["H"], p["W"], p["tokens"], f.lse, f.lse, stream=stream)
        torch.cuda.synchronize()
        assert [pool_of(t) for t in (*r, *g)] == [owner] * 7
    with torch.cuda.stream(side):  # the current stream is another than the given one
        r = fs.fs_logprobs(p["H"], p["W"], p["tokens"], 3, stream=0)
        torch.cuda.synchronize()
        assert torch.cuda.current_stream() == side and pool_of(r.lse) == 0
    # The workspace, freed on return, left its block to the given stream.
    need = fs.fs_logprobs_grad_workspace_size(200, 128, 3000)
    fresh = torch.cuda.Stream()
    g = fs.fs_logprobs_grad(p["H"], p["W"], p["tokens"], f.lse, f.lse, stream=fresh)
    torch.cuda.synchronize()
    sizes = [segment["total_size"] for segment in torch.cuda.memory_snapshot()
             if segment["stream"] == fresh.cuda_stream]
    assert sum(sizes) >= need + 2 * (g[0].numel() + g[1].numel())


def test_two_streams_at_once():
    """Calls on two streams, none waited for, their workspaces made inside: each as alone."""
    p = problem(300, 512, 40000, T="rows", seed=93)
    q = problem(96, 512, 40000, T="rows", seed=94)
    a, e = upstream(300, True, 93)
    call = lambda x, **kw: fs.fs_logprobs(x["H"], x["W"], x["tokens"], 10,
                                          temperature=x["temperature"], **kw)
    f = call(p)
    grad = lambda **kw: fs.fs_logprobs_grad(p["H"], p["W"], p["tokens"], f.lse, a,
                                            entropy=f.entropy, grad_entropy=e,
                                            temperature=p["temperature"], **kw)
    want = [tuple(call(p)), tuple(call(q)), grad()]
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(4):
        got.append([tuple(call(p, stream=one)), tuple(call(q, stream=two)), grad(stream=one)])
        scratch = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
                   for _ in range(8)]  # the current stream's allocations meanwhile
    torch.cuda.synchronize()
    del scratch
    for r in got:
        for x, y in zip(r, want):
            assert all(torch.equal(s, t) for s, t in zip(x, y))


@pytest.mark.parametrize("B", [7, 8, 17, 24, 25, 41, 48, 49, 57, 65])
def test_box_heights_of_narrow_units(B):
    """Units of 64 ids with every slice of every stage in use: short boxes of H."""
    check_forward(problem(B, 2120, 1500, T="rows", seed=100 + B), 5)
    check_forward(problem(B, 1100, 9000, T="rows", seed=101 + B), 0)


@pytest.mark.parametrize("K", [1, 2, 4, 5, 12, 20])
@pytest.mark.parametrize("B,V,at", [
    (1, 300, "one thread"), (1, 300, "spread"), (20, 15000, "spread"), (1, 45000, "spread"),
    (3, 90000, "far"), (150, 3000, "spread"), (150, 60000, "far")])
def test_alternatives_close_together(B, V, at, K):
    """30 logits 2^-9 apart at 4096, where fp32 has 2^-11: all within 2^-16 of their
    size.  Sums of two exact terms, so tensor-core sums are exact and the order known:
    the highest ids are the best.  "far": in the units that a worker visits later."""
    d = 72
    W = torch.zeros((V, d))
    gen = torch.Generator().manual_seed(B + V + K)
    W[:, 0] = torch.randn(V, generator=gen) * 50
    ids = {"one thread": torch.arange(30), "spread": torch.randperm(V, generator=gen)[:30].sort().values,
           "far": V - 30 * 61 + torch.arange(30) * 61}[at]
    W[ids, 0] = 4096.0
    W[ids, 40] = torch.arange(30) / 512.0
    H = torch.zeros((B, d))
    H[:, 0] = 1.0
    H[:, 40] = 1.0
    tokens = ids[torch.arange(B) % 30].cuda()
    p = dict(H=H.bfloat16().cuda(), W=W.bfloat16().cuda(), tokens=tokens, temperature=None,
             vocab_mask=None)
    r, _ = check_forward(p, K)
    assert torch.equal(r.topk_idx.cpu(), ids.flip(0)[:K].expand(B, K))


@pytest.mark.parametrize("K", [1, 5, 20])
@pytest.mark.parametrize("B,V", [(8, 20000), (8, 60000), (140, 20000)])
def test_alternatives_beside_a_common_offset(B, V, K):
    """Logits of 60 and a deviation of 0.03, as a common direction of H and W leaves
    them: neighbours in rank are several fp32 steps of the sum apart, and closer than
    2^-16 of it.  (Seeds without 5 ids within 1e-6 of 60 of the K-th, checked here.)"""
    d = 64
    gen = torch.Generator().manual_seed(2)
    W = torch.randn((V, d), generator=gen) * 0.004
    W[:, 0] = 60.0
    H = torch.randn((B, d), generator=gen)
    H[:, 0] = 1.0
    p = dict(H=H.bfloat16().cuda(), W=W.bfloat16().cuda(), temperature=None, vocab_mask=None,
             tokens=torch.randint(0, V, (B,), generator=gen).cuda())
    l = (p["H"].double() @ p["W"].double().T).sort(dim=1, descending=True).values
    near_kth = (l - l[:, K - 1:K]).abs() < 2 * 60e-6
    assert int(near_kth.sum(1).max()) <= 5
    check_forward(p, K)


def decided_rows(kind, B, d, V, seed):
    """Rows that one id decides, 60 units of x or more ahead of the next, whose logits are
    not what the tensor core's mean cut-off expects: "few" non-zeros in H (sums are exact
    on the way), partial sums 100 times the logit that "cancel", "dense" ones."""
    gen = torch.Generator().manual_seed(seed)
    W = torch.randn((V, d), generator=gen) / math.sqrt(d)
    H = torch.randn((B, d), generator=gen)
    best = torch.randperm(V, generator=gen)[:B]
    if kind == "few":
        H.zero_()
        H[torch.arange(B), torch.arange(B) * 7 % d] = 256.0
        W = (W * math.sqrt(d)).clamp_(max=5.0)
        W[best, torch.arange(B) * 7 % d] = 7.8125          # 2000, the others at most 1280
    elif kind == "cancel":
        half = d // 2
        sign = torch.randint(0, 2, (B, half), generator=gen) * 2.0 - 1.0
        W[:, half:] = W[:, :half]
        W += 4.0
        H = H.abs()
        H[:, :half] *= 1.0 + 0.9 * sign
        H[:, half:] = -H[:, :half]
        W[best, half:] -= 0.5 * sign                       # ahead by 0.45 sum |H|
    else:
        W[best] += (H * 0.1)                               # ahead by |H|^2 / 10
    return H.bfloat16().cuda(), W.bfloat16().cuda(), best


@pytest.mark.parametrize("kind", ["few", "cancel", "dense"])
@pytest.mark.parametrize("B,V,K", [(3, 3000, 0), (3, 3000, 5), (3, 50000, 0), (3, 50000, 20),
                                   (140, 3000, 0), (140, 3000, 5)])
def test_rows_that_one_id_decides(kind, B, V, K):
    """lse is the id's logit, summed exactly: off by the rounding of its result, 2 u.  A
    log-probability is a difference of two exact logits over T, each operation off by u
    of its result; the log-sum of one term of 1 is 0 but for the others' e^-60."""
    d = 4096
    H, W, best = decided_rows(kind, B, d, V, seed=110 + B + V)
    tokens = best.clone()
    tokens[1::2] = (tokens[1::2] + 17) % V
    T = torch.full((B,), 0.5)
    T[::3] = 1.0
    p = dict(H=H, W=W, tokens=tokens.cuda(), temperature=T.cuda(), vocab_mask=None)
    r = fs.fs_logprobs(H, W, p["tokens"], K, temperature=p["temperature"])
    w = ref.forward(H, W, p["tokens"], K, p["temperature"])
    x = (H.double() @ W.double().T).cpu() / T.double().unsqueeze(1)
    first = x.topk(2, dim=1).values
    assert float((first[:, 0] - first[:, 1]).min()) > 60.0
    near(r.lse, w["lse"], 2 * ref.U * w["lse"].abs() + 2 * ref.U, "lse")
    near(r.logp, w["logp"], 6 * ref.U * w["logp"].abs() + 2 * ref.U, "logp")
    near(r.entropy, w["entropy"], 2.0 ** -22, "entropy")
    assert bool((r.logp.cpu()[tokens == best] >= -2 * ref.U).all())
    if K:
        assert torch.equal(r.topk_idx[:, 0].cpu(), best)
        near(r.topk_logp[:, 0], w["topk_logp"][:, 0], 2 * ref.U, "topk_logp")


@pytest.mark.parametrize("kind", ["few", "dense"])
@pytest.mark.parametrize("B,V", [(3, 3000), (20, 50000), (140, 3000)])
def test_gradient_of_likely_tokens(kind, B, V):
    """Tokens of probability 1 - e^-4 or more: G there is a (1 - P), a small difference, of
    an exact logit and lse: off by the rounding of lse, u |lse| of P, and a few u.  The
    others' logits are the tensor core's: their probabilities off by its cut-off, 1.55e-8
    per 16 products and twice that for one id, u |lse|, and bf16."""
    d = 4096
    H, W, best = decided_rows(kind, B, d, V, seed=120 + B + V)
    free = torch.ones(V, dtype=torch.bool).index_fill(0, best, False)
    second = free.nonzero().squeeze(1)[:B]
    if kind == "few":
        W[second.cuda(), (torch.arange(B) * 7 % d).cuda()] = 7.78125  # 1992 to 2000
    else:
        W[second.cuda()] = (W[best.cuda()].float() * 0.985).bfloat16()
    gen = torch.Generator().manual_seed(B)
    a = torch.randn(B, generator=gen)
    f = fs.fs_logprobs(H, W, best.cuda())
    dH, dW = fs.fs_logprobs_grad(H, W, best.cuda(), f.lse, a.cuda())
    Hd, Wd = H.cpu().double(), W.cpu().double()
    x = Hd @ Wd.T
    lse = torch.logsumexp(x, 1, keepdim=True)
    p = (x - lse).exp()
    at = best.unsqueeze(1)
    assert float(p.gather(1, at).min()) > 1 - math.exp(-4)
    rest = p.scatter(1, at, 0.0)
    G = -a.double().unsqueeze(1) * rest
    G.scatter_(1, at, a.double().unsqueeze(1) * rest.sum(1, keepdim=True))
    e_lse = 2 * ref.U * lse.abs()
    dG = a.double().abs().unsqueeze(1) * rest * (
        ref.BF16 + e_lse + 3 * 1.55e-8 * (d / 16) * x.abs() + 8 * ref.U) * (1 + ref.BF16)
    dG.scatter_(1, at, a.double().abs().unsqueeze(1) * (e_lse + 8 * ref.U))
    sums = (V / 16 + 64) * 2.0 ** -23
    wH, wW = G @ Wd, G.T @ Hd
    bH = dG @ Wd.abs() + sums * (G.abs() @ Wd.abs())
    bW = dG.T @ Hd.abs() + sums * (G.abs().T @ Hd.abs())
    near(dH, wH, bH * (1 + ref.BF16) + ref.BF16 * wH.abs() + 1e-38, "dH")
    near(dW, wW, bW * (1 + ref.BF16) + ref.BF16 * wW.abs() + 1e-38, "dW")


@pytest.mark.parametrize("B", [4, 140])
@pytest.mark.parametrize("K", [3, 20])
def test_rows_of_nan(B, K):
    """No id of a row whose logits are all NaN can be listed; what is returned for it is
    NaN, as in a row with one NaN and fewer ids than places."""
    p = problem(B, 64, 500, mask_frac=0.1, seed=130)
    p["H"][1] = math.nan
    p["vocab_mask"][2] = 0
    p["vocab_mask"][2, 1] = 3 << 8          # ids 40 and 41
    p["W"][40] = math.nan
    p["vocab_mask"][0, 1] &= ~(1 << 8)      # masked in rows 0 and 3
    p["vocab_mask"][3:, 1] &= ~(1 << 8)
    p["vocab_mask"][3] = 0                  # a row that allows nothing is not NaN
    r = fs.fs_logprobs(p["H"], p["W"], p["tokens"], K, vocab_mask=p["vocab_mask"])
    for b in (1, 2):
        assert bool(torch.isnan(r.lse[b])) and bool(torch.isnan(r.entropy[b]))
        assert bool(torch.isnan(r.topk_logp[b]).all())
    assert bool((r.topk_idx[1] == -1).all())
    assert r.topk_idx[2].tolist() == [41] + [-1] * (K - 1)
    assert r.lse[3].item() == -math.inf
    assert bool((r.topk_logp[3] == -math.inf).all()) and bool((r.topk_idx[3] == -1).all())
    assert bool(torch.isfinite(r.topk_logp[0]).all()) and not bool((r.topk_idx[0] == 40).any())


@pytest.mark.parametrize("B,d,V", [(16, 520, 3000), (140, 264, 2000)])
@pytest.mark.parametrize("share", [0.5, 0.9, 0.99])
def test_gradient_of_rows_that_another_id_holds(B, d, V, share):
    """Row b's mass is on id b, its token is another: G there is -a p, rounded to bf16 as
    every element but the token's, which the elementwise bounds hold."""
    p = problem(B, d, V, seed=140 + B)
    H, W = p["H"].double(), p["W"].double()
    rows = torch.arange(B, device="cuda")
    x = H @ W.T
    rise = torch.logsumexp(x, 1) + math.log(share / (1 - share)) - x[rows, rows]
    p["W"][:B] = (W[:B] + (rise / (H * H).sum(1)).unsqueeze(1) * H).bfloat16()
    p["tokens"] = p["tokens"] % (V - B) + B
    f = fs.fs_logprobs(p["H"], p["W"], p["tokens"], 1)
    assert torch.equal(f.topk_idx[:, 0], rows)
    assert float((f.topk_logp[:, 0].exp() - share).abs().max()) < 0.3 * share
    check_gradient(p, *upstream(B, True, B))


@pytest.mark.parametrize("B,d,V,K", [(2, 4096, 117000, 5), (2, 4096, 117000, 20), (2, 4096, 117000, 1),
                                     (2, 4032, 117000, 5)])
def test_long_units_of_few_rows(B, d, V, K):
    """Three units a CTA and more, of 64 k slices, where lists begin without a sort."""
    p = problem(B, d, V, T=0.7, seed=150 + K)
    p["W"][V - 40 * 37::37] = p["W"][5]  # equal rows in units visited late
    check_forward(p, K)


@pytest.mark.parametrize("T", [1e-5, 1e-7, 1e-12, 1e-30, 2e-38, 1e-40])
@pytest.mark.parametrize("B,K", [(3, 0), (3, 5), (140, 0), (140, 20)])
def test_temperatures_near_zero(B, K, T):
    """As some write greedy decoding: the largest logit has all the mass however small T
    is, also below what the logits' own rounding amounts to in units of T."""
    d, V = 1024, 3000
    H, W, best = decided_rows("dense", B, d, V, seed=160 + B)
    tokens = best.clone()
    tokens[1::2] = (tokens[1::2] + 17) % V
    temp = torch.full((B,), T)
    r = fs.fs_logprobs(H, W, tokens.cuda(), K, temperature=temp.cuda())
    t = temp.double().clamp_min(2.0 ** -126)
    x = (H.double() @ W.double().T).cpu()
    top = x.gather(1, best.unsqueeze(1)).squeeze(1)
    lse = (top / t).float().double()               # +inf where fp32 ends
    near(r.lse, lse, 4 * ref.U * lse.abs(), "lse")
    want = ((x.gather(1, tokens.unsqueeze(1)).squeeze(1) - top) / t).float().double()
    near(r.logp, want, 6 * ref.U * want.abs(), "logp")
    assert bool((r.entropy == 0).all())
    if K:
        assert torch.equal(r.topk_idx[:, 0].cpu(), best) and bool((r.topk_logp[:, 0] == 0).all())


@pytest.mark.parametrize("T", [0.3, 1e-2, 1e-4, 1e-7, 1e-20])
@pytest.mark.parametrize("B", [3, 140])
def test_gradient_at_temperatures_near_zero(B, T):
    """Rows that an id other than the token holds: dH = (a/T) (W[token] - P W[id]), P = 1.
    P is at least exp(-off), off what the tensor core cuts off (3 times its mean at most, as
    in test_gradient_of_likely_tokens) and lse's rounding, in units of T, and at most 1.  So
    dH lies between the two ends, but for G's rounding, u = 2^-8 of P, the result's, 2^-8 of
    the larger end, and the fp32 sums' (a few 2^-23 of the two terms)."""
    d, V = 1024, 3000
    H, W, best = decided_rows("dense", B, d, V, seed=170 + B)
    tokens = torch.ones(V, dtype=torch.bool).index_fill(0, best, False).nonzero().squeeze(1)[:B]
    temp = torch.full((B,), T).cuda()
    a = torch.randn(B, generator=torch.Generator().manual_seed(B))
    f = fs.fs_logprobs(H, W, tokens.cuda(), temperature=temp)
    dH, dW = fs.fs_logprobs_grad(H, W, tokens.cuda(), f.lse, a.cuda(), temperature=temp)
    assert bool(torch.isfinite(dH).all()) and bool(torch.isfinite(dW).all())
    t = temp.cpu().double()
    x = ((H.double() @ W.double().T).cpu() / t.unsqueeze(1)).max(1).values
    low = torch.exp(-(3 * 1.55e-8 * (d / 16) + 2 * ref.U) * x - 8 * ref.U).unsqueeze(1)
    scale = (a.double() / t).unsqueeze(1)
    named, held = scale * W[tokens.cuda()].cpu().double(), scale * W[best.cuda()].cpu().double()
    ends = torch.stack([named - held, named - low * held])
    slack = (ref.BF16 * held.abs() + ref.BF16 * (1 + ref.BF16) * ends.abs().max(0).values
             + (V / 16 + 64) * 2.0 ** -23 * (named.abs() + held.abs()) + 1e-38)
    got = dH.cpu().double()
    assert bool((got >= ends.min(0).values - slack).all())
    assert bool((got <= ends.max(0).values + slack).all())
