"""A clipped step without gradients: its norm is that of none, not the last step's."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def fl():
    from conftest import build_library

    build_library()
    import lm_head_jsd_gb300 as fl

    return fl


def test_norm_is_zero(fl):
    opt = fl.AdamW([torch.ones(100, device="cuda"), torch.ones(7, device="cuda")])
    opt.step([None, None], max_norm=1.0)
    assert opt.grad_norm.item() == 0 and opt.grad_norm.dtype == torch.float32 and opt.grad_norm.is_cuda and opt.steps == 0
    opt.step([torch.ones(100, device="cuda"), None], max_norm=1.0)
    last, kept = opt.grad_norm, [p.clone() for p in opt.params]
    assert last.item() == 10
    side = torch.cuda.Stream()
    opt.step([None, None], max_norm=1.0, stream=side)
    side.synchronize()
    assert opt.grad_norm.item() == 0 and last.item() == 10 and opt.steps == 1
    assert all(torch.equal(a, b) for a, b in zip(opt.params, kept))
    opt.step([None, None])  # (without max_norm it is left as it is)
    assert opt.grad_norm.item() == 0
