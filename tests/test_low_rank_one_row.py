"""One token's row in place: where the row after it would lie says nothing."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "fp32"])
def test_in_place_whatever_the_strides(dtype):
    from conftest import build_library

    build_library()
    import lm_head_jsd_gb300 as fl

    g = torch.Generator("cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    buf, x, a, b = r(3, 200).to(dtype), r(1, 64).to(BF), r(2, 8, 64).to(BF), r(2, 100, 8).to(BF)
    index, before = torch.ones(1, dtype=torch.int64, device="cuda"), buf.clone()
    y, out = buf[:1, :100], buf[0, :100][None]
    assert y.stride(0) != out.stride(0)
    want = fl.low_rank_add(y, x, a, b, index)
    assert fl.low_rank_add(y, x, a, b, index, out=out) is out
    assert torch.equal(buf[:1, :100], want) and torch.equal(buf[:, 100:], before[:, 100:]) and torch.equal(buf[1:], before[1:])
    with pytest.raises(ValueError, match="shares memory with y"):
        fl.low_rank_add(y, x, a, b, index, out=buf[0, 1:101][None])
