#!/usr/bin/env python
"""Policy-gradient training of a tiny next-token policy with a tied table.

The operators run as a training loop uses them: fs_embed looks the previous
token up, fs_sample draws the next one, fs_logprobs scores the draw,
fs_logprobs_grad turns rewards and an entropy bonus into gradients of the hidden
states and the head, and fs_embed_grad adds the lookup's gradient into the
head's, the two sharing one table.  The task: after token t, say (7 t + 3) mod V.

    python examples/policy_gradient.py --steps 300
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import lm_head_gumbel_gb300 as fs  # noqa: E402


def train(steps=300, V=64, d=64, B=1024, lr=0.004, bonus=0.03, seed=0, log=print):
    """Returns the mean reward of the first and of the last ten steps."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    table = torch.randn((V, d), generator=gen, device="cuda") / math.sqrt(d)  # fp32 masters
    mix = torch.eye(d, device="cuda")
    moments = [[torch.zeros_like(w), torch.zeros_like(w)] for w in (table, mix)]
    workspace = torch.zeros(fs.fs_workspace_size(B, V), dtype=torch.uint8, device="cuda")
    baseline, rewards = 0.0, []
    for step in range(steps):
        W = table.bfloat16()
        prev = torch.randint(0, V, (B,), generator=gen, device="cuda")
        X = fs.fs_embed(prev, W, scale=math.sqrt(d))
        H = (X.float() @ mix).bfloat16()
        token = fs.fs_sample(H, W, seed=seed, offset=step, workspace=workspace)
        score = fs.fs_logprobs(H, W, token, 3, overlap_previous=True)
        reward = (token == (7 * prev + 3) % V).float()
        # The loss: -(reward - baseline) logp - bonus entropy, averaged.
        dH, dW = fs.fs_logprobs_grad(H, W, token, score.lse, (baseline - reward) / B,
                                     entropy=score.entropy,
                                     grad_entropy=torch.full((B,), -bonus / B, device="cuda"))
        dX = (dH.float() @ mix.T).bfloat16()
        dmix = X.float().T @ dH.float()
        dtable = dW.float()
        fs.fs_embed_grad(prev, dX, V, scale=math.sqrt(d), out=dtable, accumulate=True)
        for w, g, (m, v) in zip((table, mix), (dtable, dmix), moments):  # Adam
            m.mul_(0.9).add_(g, alpha=0.1)
            v.mul_(0.99).addcmul_(g, g, value=0.01)
            at = step + 1
            w -= lr * (m / (1 - 0.9 ** at)) / ((v / (1 - 0.99 ** at)).sqrt() + 1e-8)
        mean = float(reward.mean())
        baseline = 0.9 * baseline + 0.1 * mean
        rewards.append(mean)
        if log and step % 50 == 0:
            best = score.topk_idx[0].tolist()
            log(f"step {step}: reward {mean:.3f}, entropy {float(score.entropy.mean()):.3f}, "
                f"after {int(prev[0])}: {int(token[0])} at {float(score.logp[0]):.2f}, best {best}")
    return sum(rewards[:10]) / 10, sum(rewards[-10:]) / 10


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--steps", type=int, default=300)
    first, last = train(ap.parse_args().steps)
    print(f"mean reward: first steps {first:.3f}, last steps {last:.3f}")
