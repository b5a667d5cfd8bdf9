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

    monkeypatch.setattr(_streams, "_device", lambda: 0)
    ctx = _streams.on(None, torch.device("cuda", 1))
    assert isinstance(ctx, torch.cuda.device) and ctx.idx == 1
    assert not isinstance(_streams.on(None, torch.device("cuda", 0)), torch.cuda.device)


# ---- results and outputs that are given ----
def _result(rows=4, k=2, device="cpu", **other):
    f = lambda *s: torch.zeros(s, device=device)  # noqa: E731
    r = dict(logp=f(rows), entropy=f(rows), lse=f(rows), norm=f(rows, 2), top_logp=f(rows, k),
             top_id=f(rows, k).long())
    return fl.Logprobs(**{**r, **other})


def _bad_results(device):
    f = lambda *s: torch.zeros(s, device=device)  # noqa: E731
    return [dict(entropy=f(3)), dict(norm=f(4)), dict(norm=f(4, 4)[:, ::2]), dict(entropy=f(4).double()),
            dict(logp=f(4).half()), dict(logp=None), dict(norm=None),
            dict(entropy=torch.zeros(4, device="meta"))]


def _bad_outs(device):
    f = lambda *s: torch.zeros(s, device=device)  # noqa: E731
    return _bad_results(device) + [dict(lse=f(5)), dict(top_logp=f(4, 1)), dict(top_id=None),
                                   dict(top_id=f(4, 2)), dict(top_id=f(4, 3).long()[:, :2])]


def test_results_are_checked():
    from lm_head_jsd_gb300.logprobs import _check_result

    cpu = torch.device("cpu")
    _check_result(_result(), 4, True, cpu, 2)
    _check_result(_result(logp=None), 4, False, cpu, 2)
    _check_result(_result(lse=None, top_logp=None, top_id=None), 4, True, cpu)
    _check_result(_result(top_logp=None, top_id=None), 4, True, cpu, 0)
    for bad in _bad_outs(cpu):
        with pytest.raises((ValueError, TypeError)):
            _check_result(_result(**bad), 4, True, cpu, 2)
    for bad in _bad_results(cpu):
        with pytest.raises((ValueError, TypeError)):
            _check_result(_result(**bad), 4, True, cpu)


@gpu
def test_given_results_and_outputs_are_refused_on_the_host():
    """Nothing is launched: each of these would be written or read past its end."""
    x, w = torch.randn(4, 64).bfloat16().cuda(), torch.randn(50, 64).bfloat16().cuda()
    y = torch.tensor([0, 1, 2, 49]).cuda()
    g = torch.ones(4, device="cuda")
    run = fl.FusedLinearLogprobs(4, 64, 50, top_k=2, keep_for_backward=True)
    r = run.forward(x, w, y)
    launched = fl.fljsd_launch_count()
    for bad in _bad_outs("cuda"):
        with pytest.raises((ValueError, TypeError)):
            run.forward(x, w, y, out=_result(device="cuda", **bad))
    for bad in _bad_results("cuda"):
        q = _result(device="cuda", **bad)
        with pytest.raises((ValueError, TypeError)):
            run.backward(x, w, y, q, g)
        with pytest.raises((ValueError, TypeError)):
            fl.logits_logprobs_backward(x.float() @ w.float().T, y, q, g)
    e = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    for bad in ((e(3, 64), e(50, 64)), (e(4, 64), e(49, 64)), (e(64, 4).T, None), (None, e(50, 65)[:, :64]),
                (e(4, 64, dtype=torch.float32), None), (None,)):
        with pytest.raises(ValueError):
            run.backward(x, w, y, r, g, out=bad)
    assert fl.fljsd_launch_count() == launched
    # what was refused leaves the plan as it was
    gx, gw = torch.empty_like(x), torch.empty_like(w)
    assert run.backward(x, w, y, r, g, out=(gx, gw))[0] is gx
    assert torch.equal(gw, run.backward(x, w, y, r, g)[1])


# ---- what carries no gradient ----
def test_fp8_linear_does_not_cut_a_graph_silently():
    x, w, s = _fp8()
    with pytest.raises(ValueError, match="requires a gradient"):
        fl.fp8_linear(x.requires_grad_(), w, s)
    with pytest.raises(ValueError, match="requires a gradient"):
        fl.fp8_linear(x * 2, w, s)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA device"):
        fl.fp8_linear(x, w, s)
    with pytest.raises(ValueError, match="CUDA device"):
        fl.fp8_linear(x.detach(), w, s)


@gpu
def test_fp8_linear_without_a_graph():
    x = torch.randn(3, 64, device="cuda", requires_grad=True)
    q = fl.fp8_quantize(torch.randn(200, 64, device="cuda"))
    want = fl.fp8_linear(x.detach(), *q)
    with torch.no_grad():
        assert torch.equal(fl.fp8_linear(x, *q), want)
    with torch.inference_mode():
        assert torch.equal(fl.fp8_linear(x, *q), want)


@gpu
def test_adamw_gradients_elsewhere_are_refused():
    opt = fl.AdamW([torch.zeros(4, device="cuda"), torch.zeros(3, device="cuda")])
    good = [torch.ones(4, device="cuda"), torch.ones(3, device="cuda")]
    for bad in ([good[0], good[1].cpu()], [good[0].cpu(), good[1].cpu()], [good[0], good[1].to("meta")],
                [None, good[1].cpu()]):
        with pytest.raises((ValueError, RuntimeError)):
            opt.step(bad)
    assert opt.steps == 0 and not opt.params[0].any()
    opt.step(good)
    assert opt.params[0].all()
