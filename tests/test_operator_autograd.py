"""The operators inside autograd: what they write in place is seen by the graphs that saved
it, and a graph's own values are those of its forward."""
import pytest
import torch

gpu = pytest.mark.gpu


def _problem(dtype=torch.bfloat16, bt=20, h=64, v=300):
    g = torch.Generator().manual_seed(bt)
    x, w = torch.randn(bt, h, generator=g), torch.randn(v, h, generator=g) / 8
    y = torch.randint(0, v, (bt,), generator=g).cuda()
    return x.to(dtype).cuda().requires_grad_(), w.to(dtype).cuda().requires_grad_(), y


@gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("master", [None, True])
def test_a_step_is_seen_by_the_graphs_before_it(bits, master):
    from lm_head_jsd_gb300 import AdamW, fused_linear_logprobs

    x, w, y = _problem()
    other = torch.ones(5, dtype=torch.bfloat16, device="cuda").requires_grad_()
    square = (other * other).sum()
    opt = AdamW([w, other], lr=0.1, state_bits=bits, master=master)
    loss = fused_linear_logprobs(x, w, y).logp.sum()
    loss.backward(retain_graph=True)
    opt.step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    square.backward()  # had no gradient: not stepped
    version = w._version
    w.grad = None
    opt.step()
    assert w._version == version and other._version > 0
    with torch.inference_mode():  # (tensors without a version)
        p = torch.ones(5, device="cuda")
        AdamW([p]).step([torch.ones(5, device="cuda")])
        assert (p != 1).all()


@gpu
def test_given_outputs_are_seen_by_the_graphs_that_saved_them():
    import lm_head_jsd_gb300 as fl

    x, w, y = (t.detach() for t in _problem())
    z = (x.float() @ w.float().T)
    q = fl.fp8_quantize(w)
    leaf = torch.ones((), device="cuda", requires_grad=True)
    saved = lambda t: (leaf * t).sum()  # (the product saves t)  # noqa: E731
    run = fl.FusedLinearLogprobs(20, 64, 300, keep_for_backward=True)
    r = run.forward(x, w, y)
    gx, gw = torch.empty_like(x), torch.empty_like(w)
    a = torch.ones(20, device="cuda")
    zl = fl.logits_logprobs(z, y)
    out = torch.empty(20, 300, device="cuda", dtype=torch.bfloat16)
    graph = fl.token_logprobs(z.requires_grad_(), y).logp.sum()  # keeps z for its gradient
    z = z.detach()
    for write, t in ((lambda: run.forward(x, w, y, out=r), r.lse),
                     (lambda: run.backward(x, w, y, r, a, out=(gx, gw)), gx),
                     (lambda: run.backward(x, w, y, r, a, out=(None, gw)), gw),
                     (lambda: fl.fp8_linear(x, *q, out=out), out),
                     (lambda: fl.logits_logprobs_backward(z, y, zl, a, out=z), z)):
        loss = saved(t)
        write()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        graph.backward()


@gpu
@pytest.mark.parametrize("form", ["fused", "token"])
@pytest.mark.parametrize("name", ["logp", "entropy", "norm"])
def test_results_written_over_before_their_backward(form, name):
    from lm_head_jsd_gb300 import fused_linear_logprobs, token_logprobs

    x, w, y = _problem()

    def graph():
        r = (fused_linear_logprobs(x, w, y) if form == "fused" else token_logprobs(x @ w.T, y))
        return r, r.logp.sum() + r.entropy.sum()

    _, loss = graph()
    want = torch.autograd.grad(loss, (x, w))
    r, loss = graph()
    changed = getattr(r, name).detach().clone()  # a copy may be changed
    changed.zero_()
    got = torch.autograd.grad(loss, (x, w), retain_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    getattr(r, name).detach().zero_()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@gpu
def test_a_dropped_graph_frees_its_memory():
    import gc

    from lm_head_jsd_gb300 import fused_linear_logprobs, token_logprobs

    x, w, y = _problem()
    torch.autograd.grad(fused_linear_logprobs(x, w, y).logp.sum(), x)
    gc.collect()
    gc.disable()
    try:
        before = torch.cuda.memory_allocated()
        for _ in range(3):
            r, t = fused_linear_logprobs(x, w, y, top_k=2), token_logprobs(x @ w.T, y)
            loss = r.logp.sum() + t.entropy.sum()
            del r, t, loss
        assert torch.cuda.memory_allocated() == before
        loss = fused_linear_logprobs(x, w, y).logp.sum()
        torch.autograd.grad(loss, (x, w))
        del loss
        assert torch.cuda.memory_allocated() == before
    finally:
        gc.enable()
