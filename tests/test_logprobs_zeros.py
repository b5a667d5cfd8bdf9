"""Alternatives whose k-th largest logit is a zero: logits equal to the threshold are kept."""
import math

import pytest
import torch

import test_logprobs as base

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
