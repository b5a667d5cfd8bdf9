"""Distilling a teacher's choices into a student's lm_head, step by step.

    python examples/distil_head.py [--tokens 4096] [--hidden 4096] [--vocab 128256] [--steps 5]

Every step: the frozen teacher's head, held in 8 bits, gives logits; their most likely
token and its log probability are what the student is taught; the student's head gives
the log probability of that token, the entropy and both gradients without forming its
own logits; AdamW with 8-bit states steps the head and a small adapter on the hidden
states. Hidden states and weights are random (no checkpoint is needed to see it run).
"""
from __future__ import annotations

import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from lm_head_jsd_gb300 import (AdamW, fp8_linear, fp8_quantize, fused_linear_logprobs,  # noqa: E402
                               logits_logprobs)


def run(tokens, hidden, vocab, steps, *, lr=2e-3, seed=0, device="cuda", log=print):
    """The mean log probability of the teacher's tokens before each step."""
    g = torch.Generator(device=device).manual_seed(seed)
    rand = lambda *shape, std=1.0: torch.randn(*shape, device=device, generator=g).mul_(std)  # noqa: E731
    x_t = rand(tokens, hidden).bfloat16()
    codes, scales = fp8_quantize(rand(vocab, hidden, std=3 / math.sqrt(hidden)))  # the teacher's head
    x_s = (x_t.float() + rand(tokens, hidden, std=0.3)).bfloat16()
    w = rand(vocab, hidden, std=1 / math.sqrt(hidden)).bfloat16().requires_grad_()
    gain = torch.ones(hidden, device=device, dtype=torch.bfloat16, requires_grad=True)
    opt = AdamW([w, gain], lr=lr, weight_decay=0.0, state_bits=8, master=True)
    seen = []
    for step in range(steps):
        began = time.perf_counter()
        teacher = logits_logprobs(fp8_linear(x_t, codes, scales), top_k=1)
        target = teacher.top_id[:, 0]
        weight = teacher.top_logp[:, 0].exp()  # the surer the teacher, the more it counts
        student = fused_linear_logprobs(x_s * gain, w, target)
        loss = -(weight * student.logp).sum() / weight.sum() - 1e-3 * student.entropy.mean()
        loss.backward()
        opt.step()
        w.grad = gain.grad = None
        seen.append(student.logp.mean().item())  # (waits for the step)
        log(f"step {step}: mean log p of the teacher's token {seen[-1]:8.4f}, "
            f"entropy {student.entropy.mean().item():7.4f}, {1e3 * (time.perf_counter() - began):7.2f} ms")
    return seen


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--vocab", type=int, default=128256)
    ap.add_argument("--steps", type=int, default=5)
    a = ap.parse_args()
    run(a.tokens, a.hidden, a.vocab, a.steps)


if __name__ == "__main__":
    main()
