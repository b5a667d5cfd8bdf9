"""Token log probabilities where the schedule changes: tiles narrower than 256 columns
and the last chunk of a plan, the products around 16 rows, rows with more candidates
than are ranked at once, and calls back to back over one workspace."""
import numpy as np
import pytest
import torch

import test_logprobs as base
from oracle import lp_rows_ref
from parity_util import f64

gpu = pytest.mark.gpu
IGN = base.IGN


# x of 128 KB and more gets tiles of as few columns as the rounds allow: 128 (one round),
# odd halves (104, 112, 120 columns a part), and 256; one CTA a tile and pairs
TILES = [(64, 1024, 5000), (100, 2048, 3001), (130, 1024, 30007), (200, 512, 40960),
         (333, 512, 40961), (300, 512, 20009), (700, 256, 26003), (65, 1032, 129)]


@gpu
@pytest.mark.parametrize("k", [0, 20])
@pytest.mark.parametrize("shape", TILES, ids=lambda s: "x".join(map(str, s)))
def test_tile_widths(shape, k):
    bt, h, v = shape
    x, w, y = base._inputs(bt, h, v, torch.bfloat16, 70 + bt, grid=True, ignored=0.1)
    w[v - 40:] = w[v - 40:] * 2  # the largest in the last, partial part
    _, _, r = base._fused(x, w, y, top_k=k, temperature=0.8)
    ref = lp_rows_ref(f64(x) @ f64(w).T, y.numpy(), top_k=k, temperature=0.8)
    base._check_rows(r, ref, base._logit_bound(x, w, 0.8), str(shape))


@gpu
@pytest.mark.parametrize("bt,c", [(333, 150), (300, 299), (40, 16)])
def test_last_chunk_of_a_plan(bt, c):
    # a last chunk of fewer rows runs the planned tiles; chunks of up to 16 rows are few
    # rows only where the whole call is
    x, w, y = base._inputs(bt, 1024, 9001, torch.bfloat16, 80 + bt, grid=True, ignored=0.1)
    run, _, r = base._fused(x, w, y, top_k=7, chunk_rows=c)
    assert run.plan.num_chunks == -(-bt // c)
    ref = lp_rows_ref(f64(x) @ f64(w).T, y.numpy(), top_k=7)
    base._check_rows(r, ref, base._logit_bound(x, w, 1.0), f"{bt} by {c}")


def _tied(bt, h, v, seed):
    """Products that are small integers: hundreds of equal logits a row."""
    g = torch.Generator().manual_seed(seed)
    x = torch.zeros(bt, h)
    x[torch.arange(bt)[:, None], torch.randint(0, h, (bt, 4), generator=g)] = 1.0
    w = torch.randint(-2, 3, (v, h), generator=g).float()
    return x.bfloat16(), w.bfloat16()


@gpu
@pytest.mark.parametrize("k", [5, 20, 32])
@pytest.mark.parametrize("bt,v", [(1, 1003), (16, 5000), (40, 1003), (300, 700), (1300, 515)])
def test_many_equal_candidates(bt, v, k):
    x, w = _tied(bt, 64, v, bt + k)
    z = f64(x) @ f64(w).T
    ref = lp_rows_ref(z, None, top_k=k)
    _, _, r = base._fused(x, w, None, top_k=k)
    base._check_rows(r, ref, base._logit_bound(x, w, 1.0), f"fused {bt}x{v}")


@gpu
@pytest.mark.parametrize("k", [5, 32])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("rows,v", [(3, 1003), (700, 1003), (3, 8200), (700, 8200), (2, 40)])
def test_many_equal_candidates_of_logits(rows, v, dtype, k):
    from lm_head_jsd_gb300 import logits_logprobs

    x, w = _tied(rows, 64, v, rows + k)
    z = torch.from_numpy(f64(x) @ f64(w).T).to(dtype)  # small integers: exact
    z[0, ::3] = -float("inf")
    z[rows - 1] = 2.0
    ref = lp_rows_ref(f64(z), None, top_k=k)
    r = logits_logprobs(z.cuda(), top_k=k)
    base._check_rows(r, ref, 0.0, f"logits {rows}x{v}")


@gpu
def test_few_rows_masked_and_infinite():
    # rows of the product for few rows: all equal, NaN, an infinity of either sign, one
    # token far above the rest, labels at the ends
    x, w, y = base._inputs(9, 64, 1000, torch.bfloat16, 90)
    w[:, 0] = w[:, 0].abs() + 0.01
    x[0] = 0
    x[1] = float("nan")
    x[2, 0] = float("inf")
    x[3, 0] = -float("inf")  # every logit -inf
    w[7, 1] = 60.0
    x[4, 1] = 60.0
    y[5], y[6], y[7], y[8] = 0, 999, IGN, 5
    _, _, r = base._fused(x, w, y, top_k=4)
    keep = [0, 4, 5, 6, 7, 8]
    ref = lp_rows_ref(f64(x[keep]) @ f64(w).T, y.numpy()[keep], top_k=4)
    base._check_rows([None if t is None else t[keep] for t in r], ref,
                     base._logit_bound(x[keep], w, 1.0), "few")
    assert torch.isnan(r.lse[1:3]).all()
    assert r.lse[3].item() == -float("inf") and r.entropy[3].item() == 0.0
    assert r.top_id[3].tolist() == [-1] * 4


@gpu
@pytest.mark.parametrize("bt", [3, 60, 333])
def test_back_to_back_over_one_workspace(bt):
    # every call's kernels follow the one before without a gap: results of calls with
    # other inputs and another plan's calls in between stay what they are alone
    from lm_head_jsd_gb300 import FusedLinearLogprobs, fp8_linear, fp8_quantize

    cases, alone = [], []
    for i in range(3):
        x, w, y = base._inputs(bt, 512, 20000, torch.bfloat16, 100 + i)
        x, w, y = x.cuda(), w.cuda(), y.cuda()
        q = fp8_quantize(w)
        cases.append((x, w, y, q))
    run = FusedLinearLogprobs(bt, 512, 20000, top_k=20)
    few = FusedLinearLogprobs(2, 512, 20000, top_k=3)
    for x, w, y, q in cases:
        torch.cuda.synchronize()
        alone.append((run.forward(x, w, y), few.forward(x[:2], w), fp8_linear(x[:2], *q)))
        torch.cuda.synchronize()
    for _ in range(10):
        got = [(run.forward(x, w, y), few.forward(x[:2], w), fp8_linear(x[:2], *q))
               for x, w, y, q in cases]
        for a, b in zip(alone, got):
            for p, q in zip((*a[0], *a[1], a[2]), (*b[0], *b[1], b[2])):
                assert p is None and q is None or torch.equal(p, q)


@gpu
@pytest.mark.parametrize("bt", [2, 200])
def test_captured_calls_follow_each_other(bt):
    from lm_head_jsd_gb300 import FusedLinearLogprobs, fp8_linear, fp8_quantize

    x, w, y = (t.cuda() for t in base._inputs(bt, 512, 9000, torch.bfloat16, 110))
    q = fp8_quantize(w)
    run = FusedLinearLogprobs(bt, 512, 9000, top_k=20)
    r = run.forward(x, w, y)
    o = torch.empty(bt, 9000, device="cuda", dtype=torch.bfloat16)
    fp8_linear(x, *q, out=o)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        for _ in range(3):
            run.forward(x, w, y, out=r)
            fp8_linear(x, *q, out=o)
    x2, _, y2 = (t.cuda() for t in base._inputs(bt, 512, 9000, torch.bfloat16, 111))
    x.copy_(x2)
    y.copy_(y2)
    g.replay()
    torch.cuda.synchronize()
    want, wo = run.forward(x2, w, y2), fp8_linear(x2, *q)
    assert all(torch.equal(a, b) for a, b in zip(r, want)) and torch.equal(o, wo)


@gpu
@pytest.mark.parametrize("bt,v", [(100, 20011), (333, 40960), (700, 9000)])
def test_alternatives_beside_a_kept_forward(bt, v):
    # the first columns' logits go out through the buffers that 2^t leaves by: neither
    # changes the other
    x, w, y = base._inputs(bt, 512, v, torch.bfloat16, 120 + bt, grid=True, ignored=0.1)
    a = torch.randn(bt, generator=torch.Generator().manual_seed(1)).cuda()
    run, args, r = base._fused(x, w, y, top_k=20, keep_for_backward=True)
    plain, _, r0 = base._fused(x, w, y, keep_for_backward=True)
    ref = lp_rows_ref(f64(x) @ f64(w).T, y.numpy(), top_k=20)
    base._check_rows(r, ref, base._logit_bound(x, w, 1.0), f"{bt}x{v}")
    assert torch.equal(r.logp, r0.logp) and torch.equal(r.entropy, r0.entropy)
    got, want = run.backward(*args, r, a, a), plain.backward(*args, r0, a, a)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
