"""Cases of the operators of speculative decoding at the LM head: quantisation to 8-bit floating
point with a scale for each block of 128, the product of such matrices, probabilities from
logits, and the verification of drafted tokens.

``run`` computes them in plain torch operations; with ``own`` set it calls the library.
Sizes are the LM heads of the benchmark's workloads and ragged ones between them."""
import math

import torch

own = False

HEADS = [(256, 4096), (2048, 151936), (4096, 151936), (4096, 128256), (5120, 262144)]


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # A decode batch's hidden states on their way into the 8-bit head.
        dict(name="quantize_step", op="quantize", N=64, d=4096, block=1, dtype="bf16"),
        # A long prompt batch's.
        dict(name="quantize_prompt", op="quantize", N=16384, d=5120, block=1, dtype="bf16"),
        # An LM head, when the model is loaded.
        dict(name="quantize_head", op="quantize", N=151936, d=4096, block=128, dtype="bf16"),
        # A toy head's logits: launch latency.
        dict(name="matmul_tiny", op="matmul", M=4, d=256, V=4096, out="fp32"),
        # One token's logits in single-sequence decoding.
        dict(name="matmul_step", op="matmul", M=1, d=4096, V=151936, out="fp32"),
        # 64 sequences with 4 drafted tokens each: the target's logits at every position.
        dict(name="matmul_drafts", op="matmul", M=320, d=4096, V=128256, out="bf16"),
        # A prompt's logits on the same head as the decode step.
        dict(name="matmul_prompt", op="matmul", M=1000, d=4096, V=151936, out="bf16"),
        # One sequence's target probabilities over 5 positions.
        dict(name="probs_step", op="probs", N=5, V=151936, dtype="fp32", out="fp32", mask=False,
             rows_t=False),
        # A batch's, under vocabulary masks and temperatures, from 16-bit logits.
        dict(name="probs_batch", op="probs", N=320, V=128256, dtype="bf16", out="fp32", mask=True,
             rows_t=True),
        # One sequence with 4 drafted tokens.
        dict(name="verify_one", op="verify", B=1, K=4, V=151936, dtype="fp32", q=True,
             ragged=False),
        # A batch with drafts of different lengths from a deterministic drafter (an n-gram table).
        dict(name="verify_ngram", op="verify", B=64, K=6, V=128256, dtype="bf16", q=False,
             ragged=True),
        # A large batch on the large vocabulary.
        dict(name="verify_batch", op="verify", B=256, K=4, V=262144, dtype="fp32", q=True,
             ragged=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "probs", "verify"])
    if rng.random() < 0.4:
        d, V = rng.choice(HEADS)
    else:  # odd sizes: rows that end inside a block, in both directions
        d, V = _log_int(rng, 64, 5120), _log_int(rng, 1000, 262144)
    if op == "quantize":
        block = rng.choice([1, 128])
        dtype = rng.choice(["bf16", "fp32"])
        N = _log_int(rng, 1, 16384) if block == 1 else V
        most = 151936 * 4096 // (2 if dtype == "fp32" else 1)
        return dict(op=op, N=max(1, min(N, most // d)), d=d, block=block, dtype=dtype)
    if op == "matmul":
        M = max(1, min(_log_int(rng, 1, 1024), (1000 * 4096 * 151936) // (d * V)))
        return dict(op=op, M=M, d=d, V=V, out=rng.choice(["bf16", "fp32"]))
    if op == "probs":
        N = max(1, min(_log_int(rng, 1, 1024), 320 * 262144 // V))
        return dict(op=op, N=N, V=V, dtype=rng.choice(["bf16", "fp32"]),
                    out=rng.choice(["bf16", "fp32"]), mask=rng.random() < 0.3,
                    rows_t=rng.random() < 0.5)
    K = rng.randint(0, 8)
    B = max(1, min(_log_int(rng, 1, 256), 256 * 9 * 262144 // ((2 * K + 1) * V)))
    return dict(op=op, B=B, K=K, V=V, dtype=rng.choice(["bf16", "fp32"]), q=rng.random() < 0.7,
                ragged=rng.random() < 0.3)


# --------------------------------------------------------------------------- inputs
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _empty(n, d, dtype, multiple=8):
    """[n, d] whose rows start at multiples of `multiple` elements."""
    ld = (d + multiple - 1) // multiple * multiple
    return torch.empty((n, ld), dtype=dtype, device="cuda")[:, :d]


def _rows(n, d, std, gen, dtype):
    out = _empty(n, d, dtype)
    step = max(1, (1 << 27) // d)
    for i in range(0, n, step):
        out[i:i + step] = torch.randn((min(step, n - i), d), generator=gen, device="cuda") * std
    return out


def _pack(allow):
    """[N, V] truth values as [N, ceil(V/32)] words, bit v % 32 of word v // 32."""
    N, V = allow.shape
    n = (V + 31) // 32
    bits = torch.zeros((N, n * 32), dtype=torch.int64, device="cuda")
    bits[:, :V] = allow
    words = (bits.view(N, n, 32) << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def _allow(words, V):
    bits = (words.unsqueeze(-1) >> torch.arange(32, dtype=torch.int32, device="cuda")) & 1
    return bits.reshape(words.shape[0], -1)[:, :V].bool()


def _quantized_rows(n, d, std, block, gen):
    """Normal rows in 8 bits with their scales, rows on 16-byte boundaries."""
    q = _empty(n, d, torch.float8_e4m3fn, 16)
    scale = torch.empty(((n + block - 1) // block, (d + 127) // 128), device="cuda")
    step = max(1, (1 << 27) // d // 128) * 128
    for i in range(0, n, step):
        x = torch.randn((min(step, n - i), d), generator=gen, device="cuda") * std
        v, s = _plain_quantize(x.bfloat16(), block)
        q[i:i + step] = v
        scale[i // block:i // block + s.shape[0]] = s
    return q, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "quantize":
        std = 1.0 if case["block"] == 1 else 2.0 / math.sqrt(case["d"])
        s["x"] = _rows(case["N"], case["d"], std, gen, _TYPES[case["dtype"]])
        return s
    V = case["V"]
    if case["op"] == "matmul":
        d = case["d"]
        s["A"], s["a_scale"] = _quantized_rows(case["M"], d, 1.0, 1, gen)
        s["W"], s["w_scale"] = _quantized_rows(V, d, 2.0 / math.sqrt(d), 128, gen)
        return s
    if case["op"] == "probs":
        N = case["N"]
        s["logits"] = _rows(N, V, 3.0, gen, _TYPES[case["dtype"]])
        s["T"] = s["mask"] = None
        if case["rows_t"]:  # as the decode workload: U[0.5, 1.5], one row in ten greedy
            s["T"] = torch.rand(N, generator=gen, device="cuda") + 0.5
            s["T"][torch.rand(N, generator=gen, device="cuda") < 0.1] = 0.0
        if case["mask"]:
            s["mask"] = _pack(torch.rand((N, V), generator=gen, device="cuda") >= 0.05)
        return s
    # The drafter's logits are the target's with noise; four in five of its tokens pass. A
    # deterministic drafter names the likeliest id of such logits, where the target is surer.
    B, K, t = case["B"], case["K"], _TYPES[case["dtype"]]
    p = _empty(B * (K + 1), V, t).unflatten(0, (B, K + 1))
    q = _empty(B * K, V, t).unflatten(0, (B, K)) if case["q"] else None
    ids = torch.empty((B, K), dtype=torch.int64, device="cuda")
    step = max(1, (1 << 27) // ((K + 1) * V))
    for b in range(0, B, step):
        n = min(step, B - b)
        z = torch.randn((n, K + 1, V), generator=gen, device="cuda") * (3.0 if case["q"] else 6.0)
        p[b:b + n] = torch.softmax(z, -1)
        z = z[:, :K] + torch.randn((n, K, V), generator=gen, device="cuda") * 0.5
        if case["q"]:
            q[b:b + n] = torch.softmax(z, -1)
            u = torch.rand((n, K, V), generator=gen, device="cuda").clamp_min(1e-30)
            z -= (-u.log()).clamp_min(1e-30).log()
        ids[b:b + n] = z.argmax(-1)
    if case["ragged"]:  # a draft ends at its first id below 0
        length = torch.randint(0, K + 1, (B, 1), generator=gen, device="cuda")
        ids[torch.arange(K, device="cuda") >= length] = -1
    s["p"], s["q_rows"], s["ids"] = p, q, ids
    s["u"] = torch.rand((B, K + 1), generator=gen, device="cuda")
    return s


# --------------------------------------------------------------------------- plain forms
def _blocks(x, block):
    """x [N, d] as [row blocks, block, column blocks, 128], 0 behind the ends."""
    N, d = x.shape
    n, k = (N + block - 1) // block, (d + 127) // 128
    if (n * block, k * 128) != (N, d):
        wide = torch.zeros((n * block, k * 128), dtype=x.dtype, device="cuda")
        wide[:N, :d] = x
        x = wide
    return x.reshape(n, block, k, 128)


def _plain_quantize(x, block):
    N, d = x.shape
    b = _blocks(x.float(), block)
    top = b.abs().amax((1, 3)).clamp_min(2.0 ** -100)
    b = b * (448.0 / top)[:, None, :, None]
    v = b.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    v = v.view(torch.uint8).reshape(b.shape[0] * block, -1)[:N, :d].view(torch.float8_e4m3fn)
    return v, top / 448.0


def _plain_wide(x, scale, block):
    """The values an 8-bit matrix stands for, in 32 bits."""
    b = _blocks(x.float(), block) * scale[:, None, :, None]
    return b.reshape(b.shape[0] * block, -1)[:x.shape[0], :x.shape[1]]


def _plain_matmul(s):
    out = _plain_wide(s["A"], s["a_scale"], 1) @ _plain_wide(s["W"], s["w_scale"], 128).T
    return out.to(_TYPES[s["out"]])


def _plain_probs(s):
    x = s["logits"].float()
    if s["mask"] is not None:
        x = x.masked_fill(~_allow(s["mask"], x.shape[1]), -math.inf)
    T, top = s["T"], x.max(1, keepdim=True).values
    x = x - top
    if T is not None:
        x = x / torch.where((T > 0) & torch.isfinite(T), T, 1.0).unsqueeze(1)
    p = x.exp()
    p = p / p.sum(1, keepdim=True)
    if T is not None:  # greedy rows: all on the lowest id of the largest logit
        at = torch.arange(x.shape[1], device="cuda")
        first = torch.where(x == 0, at, x.shape[1]).min(1, keepdim=True).values
        p = torch.where(((T > 0) & torch.isfinite(T)).unsqueeze(1), p, (at == first).float())
    return p.to(_TYPES[s["out"]])


def _plain_verify(s):
    p, q, ids, u = s["p"], s["q_rows"], s["ids"], s["u"]
    B, K = ids.shape
    rows = torch.arange(B, device="cuda")
    at = ids.clamp_min(0).unsqueeze(2)
    px = p[:, :K].gather(2, at).squeeze(2).double()
    qx = q.gather(2, at).squeeze(2).double() if q is not None else torch.ones_like(px)
    passes = (u[:, :K].double() * qx < px) & (ids >= 0)
    n = passes.long().cumprod(1).sum(1)
    w = p[rows, n].float()
    rejected = torch.zeros(B, dtype=torch.bool, device="cuda")
    if K:
        x = ids.gather(1, n.clamp_max(K - 1).unsqueeze(1)).squeeze(1)
        rejected = (n < K) & (x >= 0)
        if q is not None:
            less = q[rows, n.clamp_max(K - 1)].float()
        else:
            less = torch.zeros_like(w)
            less[rows, x.clamp_min(0)] = math.inf
        w = torch.where(rejected.unsqueeze(1), (w - less).clamp_min(0.0), w)
    total = w.double().cumsum(1)
    drawn = (total <= u[:, K:].double() * total[:, -1:]).sum(1)
    drafts = torch.cat([ids, torch.full((B, 1), -1, device="cuda")], 1)
    i = torch.arange(K + 1, device="cuda")
    out = torch.where(i < n.unsqueeze(1), drafts, -1)
    out[rows, n] = drawn
    return dict(ids=out, accepted=n)


# --------------------------------------------------------------------------- one pass
def run(state):
    s, op = state, state["op"]
    if not own:
        if op == "quantize":
            values, scale = _plain_quantize(s["x"], s["block"])
            return dict(values=values, scale=scale)
        return {"matmul": _plain_matmul, "probs": _plain_probs, "verify": _plain_verify}[op](s)
    import lm_head_gumbel_gb300 as fs
    if op == "quantize":
        r = fs.fs_quantize(s["x"], s["block"])
        return dict(values=r.values, scale=r.scale)
    if op == "matmul":
        return fs.fs_matmul_fp8(s["A"], s["a_scale"], s["W"], s["w_scale"],
                                out_dtype=_TYPES[s["out"]])
    if op == "probs":
        return fs.fs_probs(s["logits"], temperature=s["T"], vocab_mask=s["mask"],
                           out_dtype=_TYPES[s["out"]])
    r = fs.fs_verify(s["p"], s["ids"], s["u"], s["q_rows"])
    return dict(ids=r.ids, accepted=r.accepted)


# --------------------------------------------------------------------------- what a pass needs
def work(case):
    size = {"bf16": 2, "fp32": 4}
    if case["op"] == "quantize":
        N, d, block = case["N"], case["d"], case["block"]
        scales = -(-N // block) * -(-d // 128)
        return dict(bytes=N * d * (size[case["dtype"]] + 1) + 4 * scales, flops=2.0 * N * d)
    V = case["V"]
    if case["op"] == "matmul":
        M, d = case["M"], case["d"]
        scales = (M + -(-V // 128)) * -(-d // 128)
        return dict(bytes=(M + V) * d + 4 * scales + M * V * size[case["out"]],
                    flops=2.0 * M * V * d)
    if case["op"] == "probs":
        N = case["N"]
        rows = 4 * N * -(-V // 32) if case["mask"] else 0
        rows += 4 * N if case["rows_t"] else 0
        return dict(bytes=N * V * (size[case["dtype"]] + size[case["out"]]) + rows,
                    flops=3.0 * N * V)
    # One row of p a sequence and, where a draft is rejected (one token in five), one of q.
    B, K = case["B"], case["K"]
    rows = 1.0
    if case["q"]:
        kept = [0.8 ** k for k in range(K + 1)]
        rows += 1.0 - (sum(kept) / len(kept) if case["ragged"] else kept[-1])
    gathered = B * K * (8 + 4 + size[case["dtype"]] * (2 if case["q"] else 1)) + 4 * B
    return dict(bytes=B * rows * V * size[case["dtype"]] + gathered + 8 * B * (K + 2),
                flops=2.0 * B * V)


# --------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":  # values before their rounding to 8 bits
        x, block = s["x"].double(), case["block"]
        N, d = x.shape
        scale = torch.empty((-(-N // block), -(-d // 128)), dtype=torch.float64, device="cuda")
        for i in range(scale.shape[1]):
            part = x[:, 128 * i:128 * i + 128]
            top = part.abs().amax(1)
            top = torch.nn.functional.pad(top, (0, scale.shape[0] * block - N))
            scale[:, i] = top.view(-1, block).amax(1).clamp_min(2.0 ** -100) / 448.0
            part /= scale[:, i].repeat_interleave(block)[:N, None]
        return dict(values=x, scale=scale)
    if case["op"] == "matmul":
        if 2.0 * case["M"] * case["V"] * case["d"] > 8e12:
            return None
        A, W = s["A"].double(), s["W"].double()
        out = torch.zeros((case["M"], case["V"]), dtype=torch.float64, device="cuda")
        for i in range(s["a_scale"].shape[1]):
            k = slice(128 * i, 128 * i + 128)
            part = A[:, k] @ W[:, k].T
            part *= s["a_scale"][:, i, None].double()
            out += part * s["w_scale"][:, i].double().repeat_interleave(128)[:case["V"]]
        return out
    if case["op"] == "probs":
        out = torch.empty((case["N"], case["V"]), dtype=torch.float64, device="cuda")
        for n in range(case["N"]):
            x = s["logits"][n].double()
            if s["mask"] is not None:
                x[~_allow(s["mask"][n:n + 1], case["V"])[0]] = -math.inf
            T = 1.0 if s["T"] is None else float(s["T"][n])
            if T > 0:
                out[n] = torch.softmax(x / T, 0)
            else:
                out[n] = 0.0
                out[n, int((x == x.max()).nonzero()[0])] = 1.0
        return out
    B, K = case["B"], case["K"]
    ids, u = s["ids"].tolist(), s["u"].double()
    out = torch.full((B, K + 1), -1, dtype=torch.int64, device="cuda")
    accepted = torch.zeros(B, dtype=torch.int64, device="cuda")
    for b in range(B):
        n = 0
        while n < K and ids[b][n] >= 0:
            x = ids[b][n]
            qx = float(s["q_rows"][b, n, x]) if case["q"] else 1.0
            if not float(u[b, n]) * qx < float(s["p"][b, n, x]):
                break
            out[b, n] = x
            n += 1
        w = s["p"][b, n].double()
        if n < K and ids[b][n] >= 0:
            if case["q"]:
                w = torch.relu(w - s["q_rows"][b, n].double())
            else:
                w[ids[b][n]] = 0.0
        at = torch.cumsum(w, 0)
        out[b, n] = torch.searchsorted(at, u[b, K] * at[-1], right=True)
        accepted[b] = n
    return dict(ids=out, accepted=accepted)
