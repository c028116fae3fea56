"""Cases of the operators at the vocabulary ends of a model: token log-probabilities with
entropy and top alternatives, their gradient, the embedding lookup and its gradient.

``run`` computes them in plain torch operations; with ``own`` set it calls the library.
Sizes are the LM heads of the benchmark's workloads and ragged ones between them."""
import math

import torch

own = False

HEADS = [(256, 4096), (2048, 151936), (4096, 151936), (4096, 128256), (5120, 262144)]


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # One decode step of one sequence: the sampled token and 20 alternatives.
        dict(name="logprobs_step", op="logprobs", B=1, d=4096, V=151936, K=20, mask=False,
             rows_t=False),
        # A full decode batch under per-row vocabulary masks and temperatures.
        dict(name="logprobs_masked", op="logprobs", B=128, d=4096, V=128256, K=5, mask=True,
             rows_t=True),
        # The tokens of a long prompt, scored with 5 alternatives each.
        dict(name="logprobs_prompt", op="logprobs", B=1000, d=4096, V=151936, K=5, mask=False,
             rows_t=False),
        # A toy head's training step: launch latency.
        dict(name="grad_tiny", op="logprobs_grad", B=4, d=256, V=4096, mask=False, rows_t=False,
             entropy=True),
        # A short sequence's likelihood gradient on the d=2048 head.
        dict(name="grad_short", op="logprobs_grad", B=96, d=2048, V=151936, mask=False,
             rows_t=False, entropy=False),
        # A policy-gradient step over 1024 sampled tokens with an entropy bonus.
        dict(name="grad_policy", op="logprobs_grad", B=1024, d=4096, V=151936, mask=False,
             rows_t=True, entropy=True),
        # The sampled ids of a decode batch on their way back in.
        dict(name="embed_step", op="embed", N=64, d=4096, V=151936, dtype="bf16", scaled=False,
             pad=False),
        # A padded ragged batch through a 32-bit table.
        dict(name="embed_ragged", op="embed", N=4099, d=2048, V=151936, dtype="fp32", scaled=True,
             pad=True),
        # A long prompt batch on the large vocabulary, scaled by sqrt(d).
        dict(name="embed_prompt", op="embed", N=16384, d=5120, V=262144, dtype="bf16",
             scaled=True, pad=False),
        # A toy table's whole gradient.
        dict(name="embed_grad_tiny", op="embed_grad", N=512, d=256, V=4096, dtype="fp32",
             out="fp32", accumulate=False, pad=False),
        # A ragged micro-batch added into the 32-bit gradient of a tied table.
        dict(name="embed_grad_tied", op="embed_grad", N=4099, d=2048, V=151936, dtype="bf16",
             out="fp32", accumulate=True, pad=True),
        # A training batch's whole gradient, untouched rows zeroed.
        dict(name="embed_grad_batch", op="embed_grad", N=32768, d=4096, V=151936, dtype="bf16",
             out="bf16", accumulate=False, pad=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs_grad", "embed", "embed_grad"])
    if rng.random() < 0.4:
        d, V = rng.choice(HEADS)
    else:  # odd sizes: rows that end inside a tile, in both directions
        d, V = _log_int(rng, 64, 5120), _log_int(rng, 1000, 262144)
    if op in ("logprobs", "logprobs_grad"):
        B = _log_int(rng, 1, 1024)
        B = max(1, min(B, (1000 * 4096 * 151936) // (d * V)))
        c = dict(op=op, B=B, d=d, V=V, mask=rng.random() < 0.3, rows_t=rng.random() < 0.5)
        if op == "logprobs":
            c["K"] = rng.choice([0, 1, 4, 5, 11, 20])
        else:
            c["entropy"] = rng.random() < 0.5
        return c
    dtype = rng.choice(["bf16", "fp32"])
    if op == "embed":
        N = max(1, min(_log_int(rng, 1, 32768), 16384 * 5120 // d // (2 if dtype == "fp32" else 1)))
        return dict(op=op, N=N, d=d, V=V, dtype=dtype, scaled=rng.random() < 0.5,
                    pad=rng.random() < 0.5)
    N = _log_int(rng, 1, 32768)
    out = rng.choice(["bf16", "fp32"]) if dtype == "bf16" else "fp32"
    # The dense gradient is no larger than the listed batch's.
    most = 4096 * (151936 + 32768) * 2
    size = d * (V * (4 if out == "fp32" else 2) + N * (4 if dtype == "fp32" else 2))
    if size > most:
        V = max(1000, int(V * most / size))
        N = max(1, int(N * most / size))
    return dict(op=op, N=N, d=d, V=V, dtype=dtype, out=out, accumulate=rng.random() < 0.4,
                pad=rng.random() < 0.5)


# --------------------------------------------------------------------------- inputs
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _rows(n, d, std, gen, dtype):
    """[n, d] normal values, rows starting at multiples of 8 elements."""
    ld = (d + 7) // 8 * 8
    out = torch.empty((n, ld), dtype=dtype, device="cuda")
    step = max(1, (1 << 27) // ld)
    for i in range(0, n, step):
        out[i:i + step] = torch.randn((min(step, n - i), ld), generator=gen, device="cuda") * std
    return out[:, :d]


def _token_ids(N, V, pad, gen):
    """Ids of a 1/rank law over a shuffled vocabulary; with `pad`, one in eight is -1."""
    u = torch.rand(N, generator=gen, device="cuda", dtype=torch.float64)
    rank = ((V + 1.0) ** u).floor().long().sub(1).clamp(0, V - 1)
    ids = torch.randperm(V, generator=gen, device="cuda")[rank]
    if pad:
        ids[torch.rand(N, generator=gen, device="cuda") < 0.125] = -1
    return ids


def _pack(allow):
    """[B, V] truth values as [B, ceil(V/32)] words, bit v % 32 of word v // 32."""
    B, V = allow.shape
    n = (V + 31) // 32
    bits = torch.zeros((B, n * 32), dtype=torch.int64, device="cuda")
    bits[:, :V] = allow
    words = (bits.view(B, n, 32) << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def _allow(words, V):
    bits = (words.unsqueeze(-1) >> torch.arange(32, dtype=torch.int32, device="cuda")) & 1
    return bits.reshape(words.shape[0], -1)[:, :V].bool()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    d, V = case["d"], case["V"]
    if case["op"] in ("logprobs", "logprobs_grad"):
        B = case["B"]
        s["H"] = _rows(B, d, 1.0, gen, torch.bfloat16)
        s["W"] = _rows(V, d, 2.0 / math.sqrt(d), gen, torch.bfloat16)
        s["T"] = None
        if case["rows_t"]:  # as the decode workload: U[0.5, 1.5], one row in ten greedy
            s["T"] = torch.rand(B, generator=gen, device="cuda") + 0.5
            s["T"][torch.rand(B, generator=gen, device="cuda") < 0.1] = 0.0
        s["mask"] = None
        if case["mask"]:
            s["mask"] = _pack(torch.rand((B, V), generator=gen, device="cuda") >= 0.05)
        # Plausible tokens: of 32 random ids per row, one drawn by its probability among them.
        some = torch.randint(0, V, (B, 32), generator=gen, device="cuda")
        l = (s["W"][some].float() * s["H"].float().unsqueeze(1)).sum(-1)
        u = torch.rand(l.shape, generator=gen, device="cuda").clamp_min(1e-9)
        s["tokens"] = some.gather(1, (l - (-u.log()).log()).argmax(1, keepdim=True)).squeeze(1)
        if case["op"] == "logprobs_grad":
            f = _plain_logprobs(s, 0)
            s["lse"], s["ent"] = f["lse"], f["entropy"]
            s["a"] = torch.randn(B, generator=gen, device="cuda") / B
            s["e"] = None
            if case["entropy"]:
                s["e"] = (torch.randn(B, generator=gen, device="cuda") * 0.1 + 1.0) * (0.01 / B)
        return s
    N = case["N"]
    s["ids"] = _token_ids(N, V, case["pad"], gen)
    t = _TYPES[case["dtype"]]
    if case["op"] == "embed":
        s["E"] = _rows(V, d, 2.0 / math.sqrt(d), gen, t)
        s["scale"] = math.sqrt(d) if case["scaled"] else 1.0
    else:
        s["dY"] = _rows(N, d, 1.0 / math.sqrt(d), gen, t)
        s["scale"] = math.sqrt(d)
        s["dE"] = None
        if case["accumulate"]:  # what the head's gradient left there
            s["dE"] = _rows(V, d, 0.1, gen, _TYPES[case["out"]])
    return s


# --------------------------------------------------------------------------- plain forms
def _temperature(T, B):
    if T is None:
        return torch.ones(B, device="cuda")
    return torch.where((T > 0) & torch.isfinite(T), T, torch.ones_like(T))


def _plain_scaled(s):
    """l' [B, V] in 32 bits, -inf at masked ids, and the temperatures."""
    T = _temperature(s["T"], s["H"].shape[0])
    x = (s["H"].float() @ s["W"].float().T) / T.unsqueeze(1)
    if s["mask"] is not None:
        x = x.masked_fill(~_allow(s["mask"], x.shape[1]), -math.inf)
    return x, T


def _plain_logprobs(s, K):
    x, T = _plain_scaled(s)
    B, V = x.shape
    top = x.max(1, keepdim=True).values
    e = (x - top).exp()
    lse = (top + e.sum(1, keepdim=True).log()).squeeze(1)
    lp = x - lse.unsqueeze(1)
    entropy = -(torch.where(e > 0, lp, 0.0) * lp.exp()).sum(1)
    logp = lp.gather(1, s["tokens"].unsqueeze(1)).squeeze(1)
    out = dict(logp=logp, entropy=entropy, lse=lse)
    if K:
        # Neighbours in rank are often closer than 32-bit sums of d products tell apart: the
        # nearest candidates are summed again in 64 bits, then ranked.
        n = min(V, K + 12)
        cand = x.topk(n, 1).indices.sort(dim=1).values
        l = torch.cat([(s["W"][c].double() * h.double().unsqueeze(1)).sum(-1)
                       for c, h in zip(cand.split(256), s["H"].split(256))])
        l = torch.where(x.gather(1, cand) > -math.inf, l, -math.inf)
        l, at = l.sort(dim=1, descending=True, stable=True)
        l, idx = l[:, :K], cand.gather(1, at)[:, :K]
        out["topk_idx"] = torch.where(l > -math.inf, idx, -1)
        out["topk_logp"] = (l / T.double().unsqueeze(1) - lse.double().unsqueeze(1)).float()
    return out


def _plain_grad(s):
    x, T = _plain_scaled(s)
    lp = x - s["lse"].unsqueeze(1)
    p = lp.exp()
    at = s["tokens"].unsqueeze(1)
    a = torch.where(x.gather(1, at).squeeze(1) > -math.inf, s["a"], 0.0)
    g = -a.unsqueeze(1) * p
    g.scatter_add_(1, at, a.unsqueeze(1))
    if s["e"] is not None:
        lp = torch.where(p > 0, lp, 0.0)
        g -= s["e"].unsqueeze(1) * p * (lp + s["ent"].unsqueeze(1))
    g /= T.unsqueeze(1)
    dH = (g @ s["W"].float()).to(torch.bfloat16)
    dW = (g.T @ s["H"].float()).to(torch.bfloat16)
    return dict(dH=dH, dW=dW)


def _plain_embed(s):
    ids = s["ids"]
    y = s["E"][ids.clamp_min(0)].float() * s["scale"]
    return torch.where((ids >= 0).unsqueeze(1), y, 0.0).to(s["E"].dtype)


def _plain_embed_grad(s):
    ids, dY = s["ids"], s["dY"]
    keep = (ids >= 0).unsqueeze(1)
    rows = torch.where(keep, dY.float() * s["scale"], 0.0)
    if s["accumulate"]:
        if s["dE"].dtype == torch.float32:
            return s["dE"].index_add_(0, ids.clamp_min(0), rows)
        wide = s["dE"].float().index_add_(0, ids.clamp_min(0), rows)
        return s["dE"].copy_(wide)
    dE = torch.zeros((s["V"], dY.shape[1]), device="cuda")
    return dE.index_add_(0, ids.clamp_min(0), rows).to(_TYPES[s["out"]])


# --------------------------------------------------------------------------- one pass
def run(state):
    s, op = state, state["op"]
    if not own:
        return {"logprobs": lambda: _plain_logprobs(s, s["K"]), "logprobs_grad": lambda: _plain_grad(s),
                "embed": lambda: _plain_embed(s), "embed_grad": lambda: _plain_embed_grad(s)}[op]()
    import lm_head_gumbel_gb300 as fs
    if op == "logprobs":
        r = fs.fs_logprobs(s["H"], s["W"], s["tokens"], s["K"], temperature=s["T"],
                           vocab_mask=s["mask"])
        out = dict(logp=r.logp, entropy=r.entropy, lse=r.lse)
        if s["K"]:
            out["topk_idx"], out["topk_logp"] = r.topk_idx, r.topk_logp
        return out
    if op == "logprobs_grad":
        dH, dW = fs.fs_logprobs_grad(s["H"], s["W"], s["tokens"], s["lse"], s["a"],
                                     entropy=s["ent"] if s["e"] is not None else None,
                                     grad_entropy=s["e"], temperature=s["T"],
                                     vocab_mask=s["mask"])
        return dict(dH=dH, dW=dW)
    if op == "embed":
        return fs.fs_embed(s["ids"], s["E"], scale=s["scale"])
    return fs.fs_embed_grad(s["ids"], s["dY"], s["V"], scale=s["scale"], out=s["dE"],
                            out_dtype=_TYPES[s["out"]], accumulate=s["accumulate"])


# --------------------------------------------------------------------------- what a pass needs
def _touched(N, V, pad):
    """Expected number of different rows that N ids of _token_ids' law name."""
    n = N * (0.875 if pad else 1.0)
    r = torch.arange(V, dtype=torch.float64)
    p = ((r + 2) / (r + 1)).log() / math.log(V + 1.0)
    return float((1 - (1 - p) ** n).sum())


def work(case):
    d, V = case["d"], case["V"]
    if case["op"] in ("logprobs", "logprobs_grad"):
        B = case["B"]
        small = 8 * B + (4 * B if case["rows_t"] else 0)
        small += B * ((V + 31) // 32) * 4 if case["mask"] else 0
        ins = 2 * (V + B) * d + small
        if case["op"] == "logprobs":
            return dict(bytes=ins + 12 * B + 12 * B * case["K"], flops=2.0 * B * V * d)
        ins += 8 * B + (8 * B if case["entropy"] else 0)
        return dict(bytes=ins + 2 * (V + B) * d, flops=6.0 * B * V * d)
    N = case["N"]
    es = 2 if case["dtype"] == "bf16" else 4
    rows = _touched(N, V, case["pad"])
    if case["op"] == "embed":
        return dict(bytes=rows * d * es + N * d * es + 8 * N, flops=float(N * d))
    kept = N * (0.875 if case["pad"] else 1.0)
    eo = 2 if case["out"] == "bf16" else 4
    out = 2 * rows * d * eo if case["accumulate"] else V * d * eo
    return dict(bytes=kept * d * es + 8 * N + out, flops=float(N * d))


# --------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "embed":
        ids = s["ids"]
        y = torch.zeros((ids.numel(), case["d"]), dtype=torch.float64, device="cuda")
        y[ids >= 0] = s["E"][ids[ids >= 0]].double() * s["scale"]
        return y
    if case["op"] == "embed_grad":
        ids, order = s["ids"].sort(stable=True)
        dE = torch.zeros((case["V"], case["d"]), dtype=torch.float64, device="cuda")
        if s["accumulate"]:
            dE += s["dE"]
        order, ids = order[ids >= 0], ids[ids >= 0]
        return dE.index_put_((ids,), s["dY"][order].double() * s["scale"], accumulate=True)
    B, V = case["B"], case["V"]
    T = torch.ones(B, dtype=torch.float64, device="cuda")
    if s["T"] is not None:
        T = torch.where(s["T"] > 0, s["T"], 1.0).double()
    W = s["W"].double()
    parts = []
    for b in range(0, B, 256):
        at = slice(b, min(B, b + 256))
        h = s["H"][at].double()
        l = h @ W.T
        if s["mask"] is not None:
            l[~_allow(s["mask"][at], V)] = -math.inf
        lp = torch.log_softmax(l / T[at, None], 1)
        p = lp.exp()
        plogp = torch.special.xlogy(p, p)
        tok = s["tokens"][at]
        if case["op"] == "logprobs":
            o = dict(logp=lp.gather(1, tok[:, None])[:, 0], entropy=-plogp.sum(1),
                     lse=torch.logsumexp(l / T[at, None], 1))
            if case["K"]:
                best, idx = l.sort(dim=1, descending=True, stable=True)
                best, idx = best[:, :case["K"]], idx[:, :case["K"]]
                o["topk_idx"] = torch.where(best > -math.inf, idx, -1)
                o["topk_logp"] = best / T[at, None] - o["lse"][:, None]
            parts.append(o)
            continue
        a = torch.where(lp.gather(1, tok[:, None])[:, 0] > -math.inf, s["a"][at].double(), 0.0)
        g = torch.nn.functional.one_hot(tok, V).double() - p
        g *= a[:, None]
        if s["e"] is not None:
            g -= s["e"][at].double()[:, None] * (plogp - p * plogp.sum(1, keepdim=True))
        g /= T[at, None]
        parts.append((g @ W, g.T @ h))
    if case["op"] == "logprobs":
        return {k: torch.cat([o[k] for o in parts]) for k in parts[0]}
    return dict(dH=torch.cat([o[0] for o in parts]), dW=sum(o[1] for o in parts))
