"""What the operators' entry points refuse on the host."""
import pytest
import torch

gpu = pytest.mark.gpu
F8 = torch.float8_e4m3fn
fl = None


@pytest.fixture(scope="module", autouse=True)
def _package():
    from conftest import build_library

    build_library()
    global fl
    import lm_head_jsd_gb300 as fl


def _logits():
    z, y = torch.randn(3, 50), torch.tensor([0, 1, 49])
    r = fl.Logprobs(torch.zeros(3), torch.zeros(3), torch.zeros(3), torch.zeros(3, 2), None, None)
    return z, y, r


def _fp8():
    return torch.zeros(3, 64), torch.zeros(5, 64).to(F8), torch.ones(1, 1)


HOST = {
    "logits": lambda: fl.logits_logprobs(*_logits()[:2]),
    "logits_top": lambda: fl.logits_logprobs(_logits()[0], top_k=2),
    "logits_backward": lambda: fl.logits_logprobs_backward(*_logits(), torch.ones(3)),
    "token": lambda: fl.token_logprobs(_logits()[0].requires_grad_(), _logits()[1]),
    "fp8_quantize": lambda: fl.fp8_quantize(torch.zeros(5, 64)),
    "fp8_linear": lambda: fl.fp8_linear(*_fp8()),
    "adamw": lambda: fl.AdamW([torch.zeros(4)]).step([torch.zeros(4)]),
    "adamw8": lambda: fl.AdamW([torch.zeros(4).bfloat16()], state_bits=8, master=True).step(
        [torch.zeros(4).bfloat16()]),
    "fused": lambda: fl.fused_linear_logprobs(torch.zeros(3, 8), torch.zeros(5, 8)),
    "plan": lambda: fl.FusedLinearLogprobs(3, 8, 5, device="cpu", free_hbm_bytes=1 << 30),
}


@pytest.mark.parametrize("name", HOST)
def test_host_tensors_are_refused(name):
    with pytest.raises(ValueError, match="expected a CUDA device"):
        HOST[name]()


def test_calls_run_on_their_tensors_device(monkeypatch):
    from lm_head_jsd_gb300 import _streams

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    ctx = _streams.on(None, torch.device("cuda", 1))
    assert isinstance(ctx, torch.cuda.device) and ctx.idx == 1
    assert not isinstance(_streams.on(None, torch.device("cuda", 0)), torch.cuda.device)
