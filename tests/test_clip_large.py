"""The norm of large finite gradients in tensors of many chunks a thread: their squares leave fp32's range
one by one, or only when they are added up."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24  # an fp32 rounding
BF = torch.bfloat16
# On either side of what is added in 64 bits (squares of 64 bytes that add up to 2^96), and where the squares of 64 bytes
# fit fp32 but not those of several chunks (2e18: of four in bf16, seven in fp32; 4e18: of two in fp32)
LARGE = [2e13, 7e13, 5e17, 1.3e18, 2e18, 4e18, 1e19]


@pytest.fixture(scope="module", autouse=True)
def fl():
    from conftest import build_library

    build_library()
    import lm_head_jsd_gb300 as fl

    return fl


def _large(dtype, value, n=60_000_001):
    """120 MB of bf16, 240 MB of fp32: at least three chunks of 16 KB to each of 16 CTAs on an SM."""
    g = torch.rand(n, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).add_(0.5).mul_(value)
    return g.to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("value", LARGE)
def test_norm(fl, value, dtype):
    x = _large(dtype, value)
    want = x.double().square().sum().sqrt().item()
    got = fl.grad_norm(x)
    # as for values near one: 16 roundings of 64 bytes' sum and one for each chunk of a thread, 7 at most, are 12 of the
    # root, whose own is one more; sums in 64 bits lose nothing to speak of
    assert abs(got.item() - want) <= 13 * U * want
    assert abs(fl.grad_norm([x[:7], x[7:]]).item() - want) <= 13 * U * want
    assert fl.grad_norm(x, norm_type=math.inf).item() == x.abs().max().item()


@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("value", [2e18, 4e18])
def test_clip(fl, value, dtype):
    x = _large(dtype, value)
    kept = x.clone()
    norm = fl.clip_grads(x, 1.0)
    assert abs(norm.item() - kept.double().square().sum().sqrt().item()) <= 13 * U * norm.item()
    f = float(np.float32(1.0) / (np.float32(norm.item()) + np.float32(1e-6)))
    assert torch.equal(x, (kept.float() * f).to(dtype)) and x.count_nonzero().item() == x.numel()


def test_clipped_step(fl):
    g = _large(BF, 2e18)
    want = g.double().square().sum().sqrt().item()
    a, b = (fl.AdamW([torch.zeros(g.numel(), dtype=BF, device="cuda")], lr=1e-2) for _ in range(2))
    a.step([g], max_norm=1.0)
    assert abs(a.grad_norm.item() - want) <= 13 * U * want
    f = np.float32(1.0) / (np.float32(a.grad_norm.item()) + np.float32(1e-6))
    b.step([g], grad_scale=torch.tensor(float(f), device="cuda"))
    assert torch.equal(a.params[0], b.params[0]) and torch.equal(a.exp_avg[0], b.exp_avg[0])
    assert a.exp_avg[0].count_nonzero().item() == g.numel()
