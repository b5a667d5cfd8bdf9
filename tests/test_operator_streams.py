"""Calls on a stream that is given (a Stream or its handle) while another is current: where
their memory comes from, and what may be done with it meanwhile."""
import pytest
import torch

gpu = pytest.mark.gpu
PAUSE = 200_000_000  # clock cycles, some 100 ms: far longer than the calls below


def _problem(bt=40, h=128, v=3000, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(bt)
    x, w = torch.randn(bt, h, generator=g), torch.randn(v, h, generator=g) / 8
    return x.to(dtype).cuda(), w.to(dtype).cuda(), torch.randint(0, v, (bt,), generator=g).cuda()


def _calls():
    """Each operator as a call of a stream that returns tensors."""
    import lm_head_jsd_gb300 as fl

    x, w, y = _problem()
    z = (x.float() @ w.float().T).bfloat16()
    q = fl.fp8_quantize(w)
    a = torch.linspace(-1, 1, 40, device="cuda")
    r = fl.logits_logprobs(z, y, top_k=5)
    run = fl.FusedLinearLogprobs(40, 128, 3000, top_k=5, keep_for_backward=True)
    kept = run.forward(x, w, y)
    return {
        "logits": lambda s: list(fl.logits_logprobs(z, y, top_k=5, stream=s)),
        "logits_backward": lambda s: [fl.logits_logprobs_backward(z, y, r, a, a, stream=s)],
        "fp8_quantize": lambda s: [t.view(torch.uint8) if t.element_size() == 1 else t
                                   for t in fl.fp8_quantize(w, stream=s)],
        "fp8_linear": lambda s: [fl.fp8_linear(x, *q, stream=s)],
        "fused": lambda s: list(run.forward(x, w, y, stream=s)),
        "fused_backward": lambda s: list(run.backward(x, w, y, kept, a, a, stream=s)),
    }


NAMES = ["logits", "logits_backward", "fp8_quantize", "fp8_linear", "fused", "fused_backward"]


def _stream_of(t):
    """The stream that the allocator took t's memory for."""
    at = t.untyped_storage().data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]


@gpu
@pytest.mark.parametrize("handle", [False, True], ids=["Stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_results_are_allocated_for_the_stream(name, handle):
    call = _calls()[name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(side.cuda_stream if handle else side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert {_stream_of(t) for t in got} == {side.cuda_stream}
    assert torch.cuda.current_stream() != side
    same = call(0)  # the default stream's handle
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, same)) and {_stream_of(t) for t in same} == {0}


@gpu
@pytest.mark.parametrize("handle", [False, True], ids=["Stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_memory_taken_meanwhile_is_other_memory(name, handle):
    """The call waits on its stream; what the current stream allocates and fills in the
    meantime is neither its workspace nor its results."""
    call = _calls()[name]
    want = call(None)
    side = torch.cuda.Stream()

    def fill():
        return [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
                for n in (16, 160, 512, 1024, 4096, 1 << 14, 1 << 16, 1 << 18, 1 << 20, 1 << 22)
                for _ in range(4)]

    call(side), fill()  # (a first allocation may wait for the device)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(PAUSE)
    got = call(side.cuda_stream if handle else side)
    full = fill()
    torch.cuda.current_stream().synchronize()
    assert not side.query()  # (the call had not run yet)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and len(full) == 40


@gpu
def test_results_dropped_while_the_caller_reads_them():
    from lm_head_jsd_gb300 import logits_logprobs

    z = torch.randn(50, 1000, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = logits_logprobs(z, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(PAUSE)
    seen, at = r.norm.clone(), r.norm.data_ptr()
    del r
    with torch.cuda.stream(side):
        later = [torch.empty(50, 2, device="cuda").fill_(-7.0) for _ in range(20)]
    assert at not in [t.data_ptr() for t in later]
    assert not torch.cuda.current_stream().query()  # (the pause was not over)
    torch.cuda.synchronize()
    assert torch.equal(seen, logits_logprobs(z).norm)


@gpu
@pytest.mark.parametrize("handle", [False, True], ids=["Stream", "handle"])
def test_first_use_of_kept_memory_waits_for_the_stream_it_was_made_on(handle):
    from lm_head_jsd_gb300 import AdamW, FusedLinearLogprobs

    x, w, y = _problem()
    p, g = torch.ones(1000, device="cuda"), torch.ones(1000, device="cuda")
    ref = AdamW([p.clone()], state_bits=8)
    ref.step([g])
    want = FusedLinearLogprobs(40, 128, 3000).forward(x, w, y)
    side = torch.cuda.Stream()
    s = side.cuda_stream if handle else side
    torch.cuda.synchronize()
    torch.cuda._sleep(PAUSE)
    opt = AdamW([p], state_bits=8)  # (its states are zeroed behind the pause)
    after = torch.cuda.Event()
    after.record()
    opt.step([g], stream=s)
    side.synchronize()
    assert after.query() and torch.equal(p, ref.params[0])
    torch.cuda._sleep(PAUSE)
    run = FusedLinearLogprobs(40, 128, 3000)
    after.record()
    r = run.forward(x, w, y, stream=s)
    side.synchronize()
    assert after.query() and torch.equal(r.logp, want.logp)
    # later uses do not wait for work that has nothing to do with it
    torch.cuda._sleep(PAUSE)
    after.record()
    r = run.forward(x, w, y, stream=s)
    opt.step([g], stream=s)
    side.synchronize()
    assert not after.query() and torch.equal(r.logp, want.logp)


@gpu
def test_given_streams_in_a_capture():
    """A captured call on a stream that joins the capture, its handle given."""
    from lm_head_jsd_gb300 import FusedLinearLogprobs, fp8_linear, fp8_quantize, logits_logprobs

    x, w, y = _problem()
    q = fp8_quantize(w)
    run = FusedLinearLogprobs(40, 128, 3000, top_k=3)
    want = run.forward(x, w, y)
    wl = logits_logprobs(fp8_linear(x, *q), y, top_k=3)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = run.forward(x, w, y, stream=side.cuda_stream)
        o = fp8_linear(x, *q, stream=side)
        gl = logits_logprobs(o, y, top_k=3, stream=side.cuda_stream)
        torch.cuda.current_stream().wait_stream(side)
    for t in (*got, *gl, o):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*want, *wl), (*got, *gl)))
