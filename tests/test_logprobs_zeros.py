"""Alternatives that are zeros: logits equal to a threshold of zero are kept, and zeros of
either sign are equal."""
import math

import pytest
import torch

import test_logprobs as base
from oracle import lp_rows_ref
from parity_util import f64

gpu = pytest.mark.gpu


def _zeros_case(bt, h, v, zeros):
    """Logits that are all negative but for zeros at the given columns."""
    g = torch.Generator().manual_seed(bt + v)
    x = torch.rand(bt, h, generator=g) + 0.25
    w = -torch.rand(v, h, generator=g) - 0.25
    w[zeros] = 0.0
    return (x / h).bfloat16(), w.bfloat16()


# a vocabulary padded with rows of zeros, and zeros over the columns of many parts; one CTA
# a tile (a short contraction) and pairs, and up to 16 rows
@gpu
@pytest.mark.parametrize("keep", [False, True], ids=["forward", "kept"])
@pytest.mark.parametrize("k", [1, 2, 8, 32])
@pytest.mark.parametrize("where", ["padding", "spread"])
@pytest.mark.parametrize("bt,h", [(5, 64), (17, 64), (300, 256), (700, 768)])
def test_threshold_of_zero(bt, h, where, k, keep):
    v = 50304
    zeros = torch.arange(50257, v) if where == "padding" else torch.arange(42001, v, 37)
    x, w = _zeros_case(bt, h, v, zeros)
    _, _, r = base._fused(x, w, None, top_k=k, keep_for_backward=keep)
    assert torch.equal(r.top_id.cpu(), zeros[:k].expand(bt, k))
    lse = torch.logsumexp(x.cuda().double() @ w.cuda().double().T, 1)
    base._close(r.top_logp, (-lse)[:, None].expand(bt, k).cpu().numpy(),
                2 * base._logit_bound(x, w, 1.0), "log probabilities")


@gpu
def test_threshold_of_zero_where_one_part_holds_more_than_k():
    # the first 40000 columns are -1, all others equal
    bt, h, v = 17, 64, 50000
    x, w = torch.ones(bt, h), torch.zeros(v, h)
    w[:40000, 0] = -1.0
    for k in (1, 20):
        _, _, r = base._fused(x.bfloat16(), w.bfloat16(), None, top_k=k)
        assert torch.equal(r.top_id.cpu(), (40000 + torch.arange(k)).expand(bt, k))
        lse = math.log(40000 * math.exp(-1.0) + 10000)
        assert (r.top_logp.cpu() + lse).abs().max().item() <= base.EPS32 * lse


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("k", [1, 3, 32])
@pytest.mark.parametrize("rows,v", [(1, 5000), (2, 20011), (700, 9001)])
def test_zeros_of_either_sign_are_equal(rows, v, k, dtype):
    """The lower column first, whatever the signs: next to each other, in the same 256
    logits and in others."""
    from lm_head_jsd_gb300 import logits_logprobs

    z = -torch.rand(rows, v, generator=torch.Generator().manual_seed(v)) - 1.0
    at = torch.tensor([3, 4, 5, 200, 201, 1023, 1024, 2500, 4097, 4990, v - 2, v - 1])
    z[:, at] = 0.0
    z[:, at[::2]] = -0.0
    if rows > 1:
        z[1] = -z[1]  # the other zeros, below every other logit
        z[1, at[-4:]] *= -1.0
        z[1, 50:] = torch.where(z[1, 50:] == 0, z[1, 50:], -1.0)
    z = z.to(dtype)
    assert z[0, 3].signbit() and not z[0, 4].signbit()
    r = logits_logprobs(z.cuda(), top_k=k)
    base._check_rows(r, lp_rows_ref(f64(z), None, top_k=k), 0.0, f"{rows}x{v}")
