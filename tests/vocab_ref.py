"""64-bit forms of the vocabulary-end operators and the error bounds that the
GPU tests hold the kernels to.  u = 2^-24 is the fp32 rounding, 2^-8 the bf16
one (relative, to nearest).

Logits.  A product of two bf16 values is exact; the tensor core adds 16 of them
to the fp32 accumulator at a time, each step off by at most 2^-23 (truncation)
of the terms' magnitude, so a logit is within
    e_l = (d/16 + 1) 2^-23 max_{b,v} sum_k |H[b,k] W[v,k]|.
x = l/T in base 2 (one multiplication by a rounded factor) is within
    e_x = e_l/T + 4u |x|max.
Log-sum-exp.  Each exponential is within e_x + 2^-22 relative, a sum of 32 terms
and then of n chunks adds (32 + n) u; the joins of at most 304 parts as much
again for each.  With log and the last product:
    e_lse = e_x + (2^-22 + (700 + V/64) u) + 4u |lse|max.
Entropy = sum p (lse - x): each p is within 2 e_lse relative, each factor within
2 e_lse, and sum p |lse - x| = entropy <= log V:
    e_ent = 2 e_lse (log V + 1) + 8u log V.
Token and alternatives: their logits are summed to 2^-40, so only lse and the
rounding of the result remain: e_logp = e_lse + 2u |logp|.
"""
import math

import torch

U = 2.0 ** -24
BF16 = 2.0 ** -8


def temperatures(T, B):
    if T is None:
        return torch.ones(B, dtype=torch.float64)
    T = T.detach().cpu().double()
    return torch.where((T > 0) & torch.isfinite(T), T, torch.ones_like(T))


def allowed(mask, B, V):
    if mask is None:
        return torch.ones((B, V), dtype=torch.bool)
    m = mask.detach().cpu()
    bits = (m.unsqueeze(-1) >> torch.arange(32, dtype=torch.int32)) & 1
    return bits.reshape(B, -1)[:, :V].bool()


def forward(H, W, tokens, K, T=None, mask=None, vocab_offset=0):
    """logp, entropy, lse, topk ids and logp in fp64 on the CPU, and the bounds."""
    H, W = H.detach().cpu().double(), W.detach().cpu().double()
    (B, d), V = H.shape, W.shape[0]
    t = temperatures(T, B).unsqueeze(1)
    allow = allowed(mask, B, V)
    Wz = torch.where(allow.any(0).unsqueeze(1), W, 0.0)  # ids masked for every row: any value
    l = (H @ Wz.T).masked_fill(~allow, -math.inf)
    x = l / t
    lse = torch.logsumexp(x, 1)
    lp = x - lse.unsqueeze(1)
    p = lp.exp().masked_fill(~allow, 0.0)
    entropy = -(p * lp.masked_fill(~allow, 0.0)).sum(1).masked_fill(~allow.any(1), 0.0)
    out = dict(lse=lse, entropy=entropy, p=p.nan_to_num(0.0))
    out["lp"] = lp.masked_fill(~allow, 0.0)
    if tokens is not None:
        tok = tokens.detach().cpu()
        loc = tok - vocab_offset
        held = (tok >= 0) & (loc >= 0) & (loc < V)
        at = loc.clamp(0, V - 1).unsqueeze(1)
        held &= allow.gather(1, at).squeeze(1)
        logp = lp.gather(1, at).squeeze(1)
        out["logp"] = torch.where(held, logp, torch.where(tok < 0, 0.0, -math.inf))
        out["held"] = held
    if K:
        n = min(K, V)
        best, idx = l.sort(dim=1, descending=True, stable=True)
        best, idx = best[:, :n], idx[:, :n]
        none = best == -math.inf
        ids = torch.full((B, K), -1, dtype=torch.int64)
        val = torch.full((B, K), -math.inf, dtype=torch.float64)
        ids[:, :n] = torch.where(none, -1, idx + vocab_offset)
        val[:, :n] = torch.where(none, -math.inf, best / t - lse.unsqueeze(1))
        out["topk_idx"], out["topk_logp"] = ids, val
    some = allow.any(1)
    e_l = (d / 16 + 1) * 2.0 ** -23 * float((H.abs() @ Wz.abs().T).max())
    finite = x[allow] if bool(some.any()) else torch.zeros(1, dtype=torch.float64)
    tmin = float(t.min())
    e_x = e_l / tmin + 4 * U * float(finite.abs().max()) / math.log(2)
    lmax = float(lse[some].abs().max()) if bool(some.any()) else 0.0
    e_lse = e_x + 2.0 ** -22 + (700 + V / 64) * U + 4 * U * lmax
    out["e_x"], out["e_lse"] = e_x, e_lse
    out["e_entropy"] = 2 * e_lse * (math.log(V) + 1) + 8 * U * math.log(V + 1)
    return out


def gradient(H, W, tokens, a, e, T=None, mask=None, vocab_offset=0, whole=None):
    """dH, dW in fp64 and their elementwise bounds.

    The kernel's G is off by its rounding (2^-8 of G), by the probabilities'
    error (2 e_lse + 8u relative, on both of G's terms, whose magnitudes are
    added here without their cancellation) and, with an entropy term, by
    e_entropy of its factor; its sums over n terms by (n/16 + 64) 2^-23 of the
    terms' magnitudes (the splits' sums included), its result by 2^-8."""
    f = whole or forward(H, W, tokens, 0, T, mask, vocab_offset)
    (B, d), V = H.shape, W.shape[0]
    t = temperatures(T, B).unsqueeze(1)
    allow = allowed(mask, B, V)
    tok = tokens.detach().cpu()
    loc = tok - vocab_offset
    inside = (loc >= 0) & (loc < V) & (tok >= 0)
    a = a.detach().cpu().double()
    a = torch.where((tok < 0) | (inside & ~f["held"]), 0.0, a).unsqueeze(1)
    e = torch.zeros(B, dtype=torch.float64) if e is None else e.detach().cpu().double()
    e = e.unsqueeze(1)
    hot = torch.zeros((B, V), dtype=torch.float64)
    rows = inside & f["held"]
    hot[rows, loc[rows]] = 1.0
    p, lp, ent = f["p"], f["lp"], f["entropy"].unsqueeze(1)
    G = (a * (hot - p) - e * p * (lp + ent)) / t
    mag = (a.abs() * (hot + p) + e.abs() * p * (lp.abs() + ent)) / t
    G, mag = G.masked_fill(~allow, 0.0), mag.masked_fill(~allow, 0.0)
    none = (f["lse"] == -math.inf).unsqueeze(1)
    G, mag = G.masked_fill(none, 0.0), mag.masked_fill(none, 0.0)
    Hd, Wd = H.detach().cpu().double(), W.detach().cpu().double()
    dH, dW = G @ Wd, G.T @ Hd
    # error of G, elementwise
    dG = BF16 * G.abs() + mag * (2 * f["e_lse"] + 8 * U) + e.abs() * p / t * f["e_entropy"]
    dG = dG * (1 + BF16)
    bH = dG @ Wd.abs() + (V / 16 + 64) * 2.0 ** -23 * (G.abs() @ Wd.abs())
    bW = dG.T @ Hd.abs() + (B / 16 + 64) * 2.0 ** -23 * (G.abs().T @ Hd.abs())
    tiny = 1e-38
    return (dH, bH * (1 + BF16) + BF16 * dH.abs() + tiny,
            dW, bW * (1 + BF16) + BF16 * dW.abs() + tiny, G)
