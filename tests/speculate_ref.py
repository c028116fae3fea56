"""Plain forms of the speculative-decoding operators on the CPU and the error bounds
that the GPU tests hold the kernels to.  u = 2^-24 is the fp32 rounding, 2^-8 the bf16
one (relative, to nearest).

Quantisation is defined in fp32, operation by operation, and compared bit by bit.

Product.  Products of e4m3 values are exact.  The tensor core adds 32 of them to the
accumulator at a time, each step off by at most 2^-23 (truncation) of the terms'
magnitude; 4 steps a block.  The scales' product is off by u, each of the n blocks'
additions by u of the magnitudes added so far:
    e = (4 2^-23 + (n + 2) u) sum |a_scale w_scale A W|.
Then the result's rounding.

Probabilities.  exp is within 2^-22 (the hardware's base-2 exponential, on an argument that is
off by at most 2^-24 in all) of itself; the sum's terms are positive, so it is within that and
its additions' (n + 32 of them in a chain at most, V / threads + 64) u; one reciprocal and
one product: 2 (2^-22 + 2^-23) + (V / 512 + 96 + 3) u, relative; plus 2^-126, below which exp
is 0.  Then the result's rounding (2^-133 in the subnormal bf16 range, half of its step).
"""
import math

import torch

U = 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def quantize(x, block):
    """values (bytes), scale."""
    x = x.detach().cpu().float()
    N, d = x.shape
    n, k = -(-N // block), -(-d // 128)
    b = torch.zeros((n * block, k * 128))
    b[:N, :d] = x
    b = b.view(n, block, k, 128)
    top = b.abs().amax((1, 3))
    top = torch.where(top < 2.0 ** -100, torch.tensor(2.0 ** -100), top)
    # (a number over a tensor is torch's reciprocal times that number: two roundings)
    y = b * (torch.full_like(top, 448.0) / top)[:, None, :, None]
    y = torch.where(y.abs() > 448.0, 448.0 * y.sign(), y)
    return y.reshape(n * block, k * 128)[:N, :d].to(torch.float8_e4m3fn), top / torch.full_like(top, 448.0)


def widen(values, scale, block):
    """What an 8-bit matrix stands for, in fp64."""
    v, s = values.detach().cpu().float().double(), scale.detach().cpu().double()
    N, d = v.shape
    s = s.repeat_interleave(block, 0)[:N].repeat_interleave(128, 1)[:, :d]
    return v * s


def matmul(A, a_scale, W, w_scale, dtype):
    """[M, V] in fp64 and its elementwise bound."""
    a, w = widen(A, a_scale, 1), widen(W, w_scale, 128)
    out, mag = a @ w.T, a.abs() @ w.abs().T
    e = (4 * 2.0 ** -23 + (a_scale.shape[1] + 2) * U) * mag
    return out, e * (1 + ROUND[dtype]) + ROUND[dtype] * out.abs()


def allowed(mask, N, V):
    if mask is None:
        return torch.ones((N, V), dtype=torch.bool)
    bits = (mask.detach().cpu().unsqueeze(-1) >> torch.arange(32, dtype=torch.int32)) & 1
    return bits.reshape(N, -1)[:, :V].bool()


def probs(logits, T, mask, dtype):
    """[N, V] in fp64 and its elementwise bound."""
    x = logits.detach().cpu().double()
    N, V = x.shape
    allow = allowed(mask, N, V)
    t = torch.ones(N) if T is None else T.detach().cpu()
    out = torch.zeros((N, V), dtype=torch.float64)
    for n in range(N):
        at = allow[n].nonzero().squeeze(1)
        l = x[n, at]
        if not (t[n] > 0 and math.isfinite(t[n])):
            l = torch.where(l.isnan(), -math.inf, l)
            if l.numel() and float(l.max()) > -math.inf:
                out[n, at[(l == l.max()).nonzero()[0]]] = 1.0
        elif l.numel() and not bool((l == -math.inf).all()):
            out[n, at] = torch.softmax(l / max(float(t[n]), 2.0 ** -126), 0)
    e = 2 * (2.0 ** -22 + 2.0 ** -23) + (V / 512 + 99) * U
    tiny = 2.0 ** -126 + (2.0 ** -133 if dtype is torch.bfloat16 else 2.0 ** -149)
    return out, (e * (1 + ROUND[dtype]) + ROUND[dtype]) * out.abs() + tiny


def verify(p, ids, u, q=None):
    """ids [B, K + 1] and accepted [B], token by token in fp64."""
    p, ids, u = p.detach().cpu(), ids.detach().cpu(), u.detach().cpu().double()
    q = None if q is None else q.detach().cpu()
    B, K, V = p.shape[0], p.shape[1] - 1, p.shape[2]
    u = torch.where(u > 0, u, 0.0).clamp_max(1 - 2.0 ** -24)
    out = torch.full((B, K + 1), -1, dtype=torch.int64)
    accepted = torch.zeros(B, dtype=torch.int64)

    def draw(w, at):
        w = torch.where((w > 0) & w.isfinite(), w, 0.0).double()
        sums = w.cumsum(0)
        if not float(sums[-1]) > 0:
            return -1
        return int((sums > at * sums[-1]).nonzero()[0])

    for b in range(B):
        n = 0
        while n < K:
            x = int(ids[b, n])
            if x < 0 or x >= V:
                break
            qx = 1.0 if q is None else float(q[b, n, x])
            if not float(u[b, n]) * qx < float(p[b, n, x]):
                break
            out[b, n] = x
            n += 1
        w, drawn = p[b, n].float(), -1
        if n < K and int(ids[b, n]) >= 0:
            if q is not None:
                r = w - q[b, n].float()
            else:
                r = w.clone()
                if int(ids[b, n]) < V:
                    r[int(ids[b, n])] = 0.0
            drawn = draw(r, u[b, K])
        out[b, n] = drawn if drawn >= 0 else draw(w, u[b, K])
        accepted[b] = n
    return out, accepted
