"""What a forward keeps in the workspace for its backward pass, where calls are captured into
graphs: a captured call runs again at each replay, and an eager one does not see it."""
import pytest
import torch

import test_logprobs as base

gpu = pytest.mark.gpu


def _setup(bt=50, h=64, v=700):
    x, w, y = (t.cuda() for t in base._inputs(bt, h, v, torch.bfloat16, 5, ignored=0.1))
    x2 = base._inputs(bt, h, v, torch.bfloat16, 6)[0].cuda()
    a = torch.randn(bt, generator=torch.Generator().manual_seed(2)).cuda()
    from lm_head_jsd_gb300 import FusedLinearLogprobs

    def fresh(x, r=None):
        run = FusedLinearLogprobs(bt, h, v, keep_for_backward=True)
        return run.backward(x, w, y, run.forward(x, w, y), a, a)

    run = FusedLinearLogprobs(bt, h, v, keep_for_backward=True)
    run.backward(x, w, y, run.forward(x, w, y), a, a)
    torch.cuda.synchronize()
    return run, x, x2, w, y, a, fresh


def _capture(f):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f()
    return graph, out


def _same(got, want):
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_a_captured_backward_of_an_eager_forward():
    run, x, _, w, y, a, fresh = _setup()
    want = fresh(x)
    r = run.forward(x, w, y)
    graph, got = _capture(lambda: run.backward(x, w, y, r, a, a))
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        _same(got, want)


@gpu
def test_forward_and_backward_captured_apart():
    run, x, x2, w, y, a, fresh = _setup()
    want, want2 = fresh(x), fresh(x2)
    at = x.clone()
    forward, r = _capture(lambda: run.forward(at, w, y))
    backward, got = _capture(lambda: run.backward(at, w, y, r, a, a))
    for value, ref in ((x, want), (x2, want2)):
        at.copy_(value)
        forward.replay()
        for _ in range(3):
            backward.replay()
            _same(got, ref)


@gpu
def test_a_replay_between_an_eager_forward_and_its_backward():
    run, x, x2, w, y, a, fresh = _setup()
    want, want2 = fresh(x), fresh(x2)
    graph, r2 = _capture(lambda: run.forward(x2, w, y))
    r = run.forward(x, w, y)
    graph.replay()  # overwrites what the eager one kept
    _same(run.backward(x, w, y, r, a, a), want)
    _same(run.backward(x2, w, y, r2, a, a), want2)


@gpu
def test_both_in_one_capture_keep():
    run, x, x2, w, y, a, fresh = _setup()
    want, want2 = fresh(x), fresh(x2)
    at = x.clone()
    from lm_head_jsd_gb300 import fljsd_launch_count

    n0 = fljsd_launch_count()
    graph, got = _capture(lambda: run.backward(at, w, y, run.forward(at, w, y), a, a))
    n1 = fljsd_launch_count()
    run.backward(at, w, y, run.forward(at, w, y), a, a)
    run.forward(at, w, y)
    n2 = fljsd_launch_count()
    for value, ref in ((x, want), (x2, want2), (x, want)):
        at.copy_(value)
        graph.replay()
        _same(got, ref)
    assert n1 - n0 <= n2 - n1  # (the captured backward did not form the product again)
