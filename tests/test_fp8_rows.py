"""Codes in rows of any length: what lies past the columns is zeros."""
import pytest
import torch

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols,ldq", [(3, 100, 112), (3, 100, 128), (130, 100, 256), (130, 128, 144),
                                           (5, 200, 1040), (1, 1, 400)])
def test_columns_past_the_end_are_zeros(rows, cols, ldq, block_rows):
    from lm_head_jsd_gb300 import fljsd_fp8_quantize, fp8_quantize

    x = torch.randn(rows, cols, generator=torch.Generator().manual_seed(ldq)).cuda()
    q, s = fp8_quantize(x, block_rows=block_rows)
    codes = torch.full((rows + 1, ldq), 255, dtype=torch.uint8, device="cuda")
    scales = torch.empty_like(s)
    fljsd_fp8_quantize(rows, cols, "fp32", block_rows, x, cols, codes, ldq, scales)
    assert torch.equal(codes[:rows, :cols], q.view(torch.uint8)) and torch.equal(scales, s)
    assert not codes[:rows, cols:].any() and (codes[rows] == 255).all()
