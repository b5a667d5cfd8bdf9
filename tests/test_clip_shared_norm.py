"""Two optimizers whose steps are clipped by one norm, as AdamW.step's documentation says it is done."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def fl():
    from conftest import build_library

    build_library()
    import lm_head_jsd_gb300 as fl

    return fl


def test_one_norm_for_two(fl):
    """Bit by bit the step of one optimizer for all of them; and of two dtypes."""
    g = torch.Generator("cuda").manual_seed(0)
    r = lambda n: torch.randn(n, device="cuda", generator=g)  # noqa: E731
    sizes, grads = (1000, 7, 4097), [r(n) for n in (1000, 7, 4097)]
    one, first, rest = (fl.AdamW([torch.ones(n, device="cuda") for n in s], lr=1e-2) for s in (sizes, sizes[:1], sizes[1:]))
    for scale in (1.0, 1e-4):  # longer than max_norm, and shorter
        now = [x * scale for x in grads]
        one.step(now, max_norm=0.5)
        norm = fl.grad_norm(now)
        assert torch.equal(norm, one.grad_norm)
        factor = (0.5 / (norm + 1e-6)).clamp(max=1)
        assert (factor.item() < 1) == (scale == 1.0)
        first.step(now[:1], grad_scale=factor)
        rest.step(now[1:], grad_scale=factor)
        assert all(torch.equal(a, b) for a, b in zip(one.params, [*first.params, *rest.params]))
    mixed = [grads[0].bfloat16(), *grads[1:]]
    norm = fl.grad_norm(mixed)
    want = torch.cat([x.double() for x in mixed]).norm().item()
    assert abs(norm.item() - want) <= 9 * 2.0 ** -24 * want
    half = fl.AdamW([torch.ones(1000, device="cuda").bfloat16()], lr=1e-2, master=True)
    half.step(mixed[:1], grad_scale=(0.5 / (norm + 1e-6)).clamp(max=1))
    # a first moment below 2^-8, of a factor, 1 - beta and a product that are an fp32 rounding or two off each
    assert abs(half.exp_avg[0].double() - 0.1 * 0.5 / want * mixed[0].double()).max().item() <= 2.0 ** -28
