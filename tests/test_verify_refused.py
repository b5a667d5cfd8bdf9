"""Verification of batches with requests that are refused as a whole: everything is written, and the other
requests' results are those of a batch without them."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def fl():
    from conftest import build_library

    build_library()
    import lm_head_jsd_gb300 as fl

    return fl


def _inputs(n, requests, v=300, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    zt = (torch.randn(n + requests, v, device="cuda", generator=g) * 2).to(BF)
    zd = (torch.randn(n, v, device="cuda", generator=g) * 2).to(BF)
    tok = torch.randint(0, v, (n,), device="cuda", generator=g)
    return zt, zd, tok, torch.rand(n, device="cuda", generator=g), torch.rand(requests, device="cuda", generator=g)


def _run(fl, x, offsets, max_drafts, t):
    """Through the C entry, into results that hold something else before; t: a number for each request."""
    zt, zd, tok, u, ud = x
    n, b, v = tok.numel(), ud.numel(), zt.shape[1]
    out = torch.full((b, max_drafts + 1), 77, dtype=torch.int64, device="cuda")
    acc, prob = torch.full((b,), 77, dtype=torch.int64, device="cuda"), torch.full((n,), 77.0, device="cuda")
    ws = torch.full((fl.fljsd_verify_workspace_bytes(b, n),), 0x7f, dtype=torch.uint8, device="cuda")
    off = None if offsets is None else torch.tensor(offsets, device="cuda")
    fl.fljsd_verify(b, n, v, max_drafts, "bf16", zt, v, zd, v, tok, u, ud, off, torch.tensor(t, device="cuda"), 1.0, out, acc, prob, ws)
    return out, acc, prob, ws[:4].view(torch.int32).item()


def _check(fl, x, offsets, max_drafts, t, valid):
    out, acc, prob, status = _run(fl, x, offsets, max_drafts, t)
    assert status == (0 if all(valid) else 1)
    want = torch.zeros_like(prob)
    zt, zd, tok, u, ud = x
    ends = offsets if offsets is not None else [max_drafts * i for i in range(len(valid) + 1)]
    for b, ok in enumerate(valid):
        if not ok:
            assert acc[b] == 0 and (out[b] == -1).all()
            continue
        s, e = ends[b], ends[b + 1]
        o, a, p, st = _run(fl, (zt[s + b:e + b + 1], zd[s:e], tok[s:e], u[s:e], ud[b:b + 1]), [0, e - s], max_drafts, t[b:b + 1])
        assert st == 0 and torch.equal(o[0], out[b]) and a[0] == acc[b]
        want[s:e] = p
    assert torch.equal(prob, want)


@pytest.mark.parametrize("ragged", [True, False], ids=["ragged", "even"])
@pytest.mark.parametrize("bad", [math.nan, -1.0, math.inf, 1e-40])
def test_temperatures(fl, bad, ragged):
    for at in range(4):
        t, valid = [1.0, 0.0, 0.7, 1.3], [True] * 4
        t[at], valid[at] = bad, False
        _check(fl, _inputs(12, 4), [0, 3, 6, 9, 12] if ragged else None, 3, t, valid)


# offsets of 12 drafted tokens, the requests that hold
OFFSETS = [([0, 3, 9, 12], [True, False, True]),  # more than there is room for
           ([0, 12, 12, 12], [False, True, True]), ([2, 4, 4, 11], [True, True, False]), ([3, 5, 7, 9], [True, True, True]),
           ([0, 2, 4, 13], [True, True, False]), ([0, 2, 4, 1 << 40], [True, True, False]), ([-2, 2, 4, 6], [False, True, True]),
           ([-(1 << 40), 2, 4, 6], [False, True, True])]
# the last request's fall, into those of the others too
LAST_FALLS = [([0, 2, 4, 3], [True, True, False]), ([0, 2, 4, 0], [True, True, False]), ([0, 3, 6, -1], [True, True, False]),
              ([1, 4, 7, -(1 << 40)], [True, True, False])]


@pytest.mark.parametrize("offsets,valid", OFFSETS, ids=str)
def test_offsets(fl, offsets, valid):
    _check(fl, _inputs(12, 3), offsets, 3, [1.0, 0.6, 0.0], valid)


@pytest.mark.parametrize("offsets,valid", LAST_FALLS, ids=str)
def test_offsets_that_fall_at_the_end(fl, offsets, valid):
    for _ in range(5):
        _check(fl, _inputs(12, 3), offsets, 3, [1.0, 0.6, 0.0], valid)


def test_a_long_buffer_of_refused_requests(fl):
    """More tokens than a launch has threads."""
    n = 300_000
    out, acc, prob, status = _run(fl, _inputs(n, 2, v=2), [0, n // 2, n], 1, [1.0, 1.0])
    assert status == 1 and not prob.any() and not acc.any() and (out == -1).all()


# From the first offsets that fall on nothing is taken: what comes then claims tokens and rows that others have too,
# at a temperature of its own.
FALLS = [([0, 2, 1, 3], 2), ([0, 5, 3, 6], 5), ([0, 5, 2, 4, 6, 8], 5), ([4, 8, 0, 3, 6, 9], 4), ([0, 3, 2, 6, 1, 12], 12),
         ([0, 1 << 40, 2, 4], 4), ([3, 0, 3, 6], 3), ([0, 4, 4, 3, 7, 7, 12], 4)]


@pytest.mark.parametrize("offsets,max_drafts", FALLS, ids=str)
def test_offsets_that_fall(fl, offsets, max_drafts):
    b = len(offsets) - 1
    fall = next(i for i in range(b) if offsets[i] > offsets[i + 1])
    valid = [i < fall and 0 <= offsets[i] <= offsets[i + 1] <= 12 and offsets[i + 1] - offsets[i] <= max_drafts for i in range(b)]
    for seed in range(5):
        _check(fl, _inputs(12, b, v=5000, seed=seed), offsets, max_drafts, [0.5 + 0.3 * i for i in range(b)], valid)


@pytest.mark.parametrize("fall", [0, 1, 255, 256, 700, 2999])
def test_offsets_that_fall_among_many(fl, fall):
    b, n = 3000, 6000
    x, t = _inputs(n, b, v=40), [0.5 + (i % 7) * 0.2 for i in range(b)]
    ends = [2 * i for i in range(b + 1)]
    out, acc, prob, status = _run(fl, x, ends, 2, t)
    assert status == 0
    o, a, p, status = _run(fl, x, ends[:fall + 1] + [e - 3 for e in ends[fall + 1:]], 2, t)
    assert status == 1 and torch.equal(o[:fall], out[:fall]) and torch.equal(a[:fall], acc[:fall]) and torch.equal(p[:2 * fall], prob[:2 * fall])
    assert (o[fall:] == -1).all() and not a[fall:].any() and not p[2 * fall:].any()
