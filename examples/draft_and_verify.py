"""Serving with drafted tokens: one frozen head for all requests, each with an adapter of its own.

    python examples/draft_and_verify.py [--requests 32] [--hidden 4096] [--vocab 128256] [--drafts 4] [--steps 5]

Every step: a drafter proposes up to --drafts tokens for each request (some requests fewer, some
greedy); the target's head, held in 8 bits with the requests' low-rank adapters on it, gives the
logits in front of and behind them; the drafted tokens are verified against both, and each request
moves on by the accepted ones and one more. Hidden states and weights are random, the drafter's
close to the target's (no checkpoint is needed to see it run).
"""
from __future__ import annotations

import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from lm_head_jsd_gb300 import fp8_linear, fp8_quantize, verify_drafts  # noqa: E402


def run(requests, hidden, vocab, drafts, steps, *, adapters=8, rank=16, seed=0, device="cuda", log=print):
    """The tokens of every request."""
    g = torch.Generator(device=device).manual_seed(seed)
    rand = lambda *shape, std=1.0: torch.randn(*shape, device=device, generator=g).mul_(std)  # noqa: E731
    number = lambda *shape: torch.rand(*shape, device=device, generator=g)  # noqa: E731
    head = fp8_quantize(rand(vocab, hidden, std=3 / math.sqrt(hidden)))
    a = rand(adapters, rank, hidden, std=1 / math.sqrt(hidden)).bfloat16()
    b = rand(adapters, vocab, rank, std=0.5 / math.sqrt(rank)).bfloat16()
    of = torch.randint(-1, adapters, (requests,), device=device, generator=g)  # -1: the plain head
    temperature = torch.where(number(requests) < 0.25, 0.0, 0.8)
    answers = [[] for _ in range(requests)]
    for step in range(steps):
        began = time.perf_counter()
        count = torch.randint(0, drafts + 1, (requests,), device=device, generator=g)
        offsets = torch.zeros(requests + 1, dtype=torch.int64, device=device)
        offsets[1:] = count.cumsum(0)
        n = int(offsets[-1])
        owner = torch.repeat_interleave(torch.arange(requests, device=device), count)  # of each drafted token
        # the states in front of every drafted token and behind the last one, request by request
        row_owner = torch.repeat_interleave(torch.arange(requests, device=device), count + 1)
        x = rand(n + requests, hidden).bfloat16()
        row = torch.arange(n, device=device) + owner
        x_draft = (x[row].float() + rand(n, hidden, std=0.15)).bfloat16()
        draft_logits = tokens = None
        if n:  # the drafter has the plain head
            draft_logits = fp8_linear(x_draft, *head)
            z = draft_logits.float() / temperature[owner].clamp_min(1e-3)[:, None]
            tokens = torch.where(temperature[owner] > 0, torch.multinomial(z.softmax(1), 1, generator=g)[:, 0], z.argmax(1))
        else:
            tokens = torch.zeros(0, dtype=torch.int64, device=device)
        logits = fp8_linear(x, *head, adapters=(a, b, of[row_owner].contiguous()))
        r = verify_drafts(logits, tokens, number(n), number(requests), draft_logits=draft_logits, offsets=offsets,
                          max_drafts=drafts, temperature=temperature)
        for answer, line, k in zip(answers, r.tokens.tolist(), r.accepted.tolist()):
            answer.extend(line[:k + 1])
        log(f"step {step}: {int(r.accepted.sum())} of {n} drafted tokens accepted (expected share "
            f"{r.accept_prob.mean().item() if n else 0.0:.3f} each), {1e3 * (time.perf_counter() - began):7.2f} ms")
    return answers


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=32)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--vocab", type=int, default=128256)
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--steps", type=int, default=5)
    a = ap.parse_args()
    run(a.requests, a.hidden, a.vocab, a.drafts, a.steps)


if __name__ == "__main__":
    main()
