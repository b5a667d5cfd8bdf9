"""The status word of calls whose workspace is their own."""
import pytest
import torch

gpu = pytest.mark.gpu
INVALID = 1


def _word():
    return torch.full((1,), 77, dtype=torch.int32, device="cuda")


@gpu
@pytest.mark.parametrize("bt", [3, 40])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("form", ["logits", "token", "fused", "fused_backward"])
def test_labels_outside_are_told(form, dtype, bt):
    from lm_head_jsd_gb300 import fused_linear_logprobs, logits_logprobs, token_logprobs

    g = torch.Generator().manual_seed(1)
    x, w = torch.randn(bt, 64, generator=g).to(dtype).cuda(), torch.randn(500, 64, generator=g).to(dtype).cuda()
    z = (x.float() @ w.float().T).to(dtype)
    side = torch.cuda.Stream()
    for label, want in ((0, 0), (499, 0), (-100, 0), (500, INVALID), (-1, INVALID), (1, 0)):
        y = torch.full((bt,), 7, device="cuda")
        y[bt - 1] = label
        s = _word()
        torch.cuda.synchronize()
        if form == "logits":
            logits_logprobs(z, y, status=s)
            assert s.item() == want
            logits_logprobs(z, y, status=s.zero_().view(()), stream=side)
            side.synchronize()
        elif form == "token":
            token_logprobs(z, y, status=s)
        elif form == "fused":
            fused_linear_logprobs(x, w, y, status=s)
        else:
            xr = x.clone().requires_grad_()
            r = fused_linear_logprobs(xr, w, y, status=s)
            assert s.item() == want
            s.fill_(77)
            r.logp.sum().backward()
        assert s.item() == want, label


@gpu
def test_products_report():
    from lm_head_jsd_gb300 import FusedLinearLogprobs, fp8_linear, fp8_quantize

    w = torch.randn(500, 64, device="cuda").bfloat16()
    q = fp8_quantize(w)
    for m in (3, 40):
        s = _word()
        x = torch.randn(m, 64, device="cuda").bfloat16()
        fp8_linear(x, *q, status=s)
        assert s.item() == 0
        run = FusedLinearLogprobs(m, 64, 500)
        run.forward(x, w, torch.full((m,), 500, device="cuda"))
        run.report(s)
        assert s.item() == INVALID


@gpu
def test_words_that_are_no_status():
    from lm_head_jsd_gb300 import fp8_linear, fp8_quantize, fused_linear_logprobs, logits_logprobs

    w = torch.randn(500, 64, device="cuda").bfloat16()
    for bad in (torch.zeros(1, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"),
                torch.zeros(1, dtype=torch.int32)):
        for call in (lambda: logits_logprobs(w, status=bad), lambda: fused_linear_logprobs(w, w, status=bad),
                     lambda: fp8_linear(w, *fp8_quantize(w), status=bad)):
            with pytest.raises(ValueError):
                call()
