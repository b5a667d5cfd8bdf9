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


@gpu
@pytest.mark.parametrize("form", ["fused", "token"])
def test_a_second_derivative_is_refused(form):
    from lm_head_jsd_gb300 import fused_linear_logprobs, token_logprobs

    x, w, y = _problem(torch.float32)
    z = (x @ w.T).detach().requires_grad_()
    to = x if form == "fused" else z
    loss = (fused_linear_logprobs(x, w, y) if form == "fused" else token_logprobs(z, y)).logp.sum()
    (want,) = torch.autograd.grad(loss, to, retain_graph=True)
    (g,) = torch.autograd.grad(loss, to, create_graph=True)
    assert torch.equal(g, want)
    other = (to * to).sum()  # (a term that the derivative could be taken of)
    with pytest.raises(RuntimeError, match="differentiable once"):
        torch.autograd.grad(other + (g * g).sum(), to)


@gpu
@pytest.mark.parametrize("form", ["fused", "token"])
def test_inputs_that_were_copied_may_change(form):
    """Inputs of other strides are copied; writing over the originals leaves the gradient."""
    from lm_head_jsd_gb300 import fused_linear_logprobs, token_logprobs

    x, w, y = _problem(torch.float32)
    z = (x @ w.T).detach()
    y2 = torch.stack([y, y], 1)[:, 0]
    x2, z2 = x.detach().T.contiguous().T.requires_grad_(), z.T.contiguous().T.requires_grad_()
    if form == "fused":
        want = torch.autograd.grad(fused_linear_logprobs(x, w, y).logp.sum(), (x, w))
        loss, to, base = fused_linear_logprobs(x2, w, y2).logp.sum(), (x2, w), x2
    else:
        z.requires_grad_()
        want = torch.autograd.grad(token_logprobs(z, y).logp.sum(), (z,))
        loss, to, base = token_logprobs(z2, y2).logp.sum(), (z2,), z2
    with torch.no_grad():
        base.zero_()
        y2.zero_()
    got = torch.autograd.grad(loss, to)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
