"""A student's head trained with a clipped step, and served: adapters on the 8-bit head, drafted tokens verified.
The operators together, as a program uses them: eagerly, captured, on streams of their own."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle.verify_oracle import accept_ratio, draw_error, request_ref

gpu = pytest.mark.gpu
BF = torch.bfloat16
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def fl():
    from conftest import build_library

    build_library()
    import lm_head_jsd_gb300 as fl

    return fl


# ---- training ----
def _student(h=128, v=1500, bt=96, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, xt = r(bt, h).to(BF).cuda(), r(bt, h).to(BF).cuda()
    w, wt = (r(v, h) / 8).to(BF).cuda(), (r(v, h) / 8).to(BF).cuda()
    return x, w, xt, wt, torch.randint(0, v, (bt,), generator=g).cuda()


def _grads(fl, x, w, xt, wt, y):
    x, w = x.detach().requires_grad_(), w.detach().requires_grad_()
    fl.fused_linear_jsd(x, w, xt, wt, y, beta=0.5).backward()
    return [w.grad, x.grad]


@gpu
def test_distil_clip_and_step(fl):
    """The loss's gradients, their norm, and the step by the clipped ones, in two forms bit by bit."""
    x, w, xt, wt, y = _student()
    g = _grads(fl, x, w, xt, wt, y)
    norm = fl.grad_norm(g)
    want = torch.cat([t.double().flatten() for t in g]).norm().item()
    assert abs(norm.item() - want) <= 9 * U * want  # (see the norm's own tests)
    most = want / 3
    a, b = (fl.AdamW([w.clone(), x.clone()], lr=1e-2, master=True) for _ in range(2))
    a.step(g, max_norm=most)
    assert torch.equal(a.grad_norm, norm)
    factor = np.float32(most) / (np.float32(norm.item()) + np.float32(1e-6))
    b.step(g, grad_scale=torch.tensor(float(factor), device="cuda"))
    assert all(torch.equal(p, q) for p, q in zip(a.params + list(a.master), b.params + list(b.master)))
    clipped = [t.clone() for t in g]
    fl.clip_grads(clipped, most)
    assert all(torch.equal(c, (t.float() * float(factor)).to(BF)) for c, t in zip(clipped, g))


@gpu
def test_captured_step_beside_an_eager_graph(fl):
    """A capture of loss, gradients and clipped step while an eager graph of the same leaves lives."""
    x, w, xt, wt, y = _student(seed=1)
    ref_w = w.clone()
    leaf_x, leaf_w = x.detach().requires_grad_(), w.detach().requires_grad_()
    eager = fl.fused_linear_jsd(leaf_x, leaf_w, xt, wt, y, beta=0.5)  # stays
    run = fl.FusedLinearJSD(96, 128, 128, 1500, BF, beta=0.5)
    opt, other = fl.AdamW([w], lr=1e-2), fl.AdamW([ref_w], lr=1e-2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        run.forward(x, ref_w.clone(), xt, wt, y)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        _, _, gw = run.forward(x, w, xt, wt, y)
        opt.step([gw], max_norm=0.01)
    graph.replay()
    torch.cuda.synchronize()
    _, _, gw2 = run.forward(x, ref_w, xt, wt, y)
    other.step([gw2], max_norm=0.01)
    assert torch.equal(w, ref_w) and torch.equal(opt.grad_norm, other.grad_norm)
    eager.backward()
    assert torch.isfinite(leaf_w.grad).all()


# ---- serving ----
def _serving(fl, h=192, v=3001, counts=(3, 0, 2, 4, 1), seed=2, rank=16, adapters=3):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    n, b = sum(counts), len(counts)
    ends = np.concatenate([[0], np.cumsum(counts)])
    owner = np.repeat(np.arange(b), np.array(counts) + 1)
    x = r(n + b, h).to(BF)
    row = [i + j for j in range(b) for i in range(ends[j], ends[j + 1])]
    t = dict(x=x, x_draft=(x[row].float() + 0.2 * r(n, h)).to(BF), a=(r(adapters, rank, h) / h ** 0.5).to(BF),
             b=(r(adapters, v, rank) / 8).to(BF), index=torch.tensor([-1, 0, 1, 2, 1])[owner].contiguous(), scales=torch.rand(adapters, generator=g),
             tokens=torch.randint(0, v, (n,), generator=g), u=torch.rand(n, generator=g) * 0.2, u_draw=torch.rand(b, generator=g),
             offsets=torch.tensor(ends), t=torch.tensor([0.8, 1.0, 0.0, 1.2, 0.8]))
    t = {k: q.cuda() for k, q in t.items()}
    head = fl.fp8_quantize((r(v, h) * 3 / h ** 0.5).cuda())
    return t, head, ends


def _serve(fl, t, head, stream=None):
    z = fl.fp8_linear(t["x"], *head, adapters=(t["a"], t["b"], t["index"], t["scales"]), stream=stream)
    zd = fl.fp8_linear(t["x_draft"], *head, stream=stream)
    return z, zd, fl.verify_drafts(z, t["tokens"], t["u"], t["u_draw"], draft_logits=zd, offsets=t["offsets"], max_drafts=4,
                                   temperature=t["t"], stream=stream)


@gpu
def test_adapters_then_verification(fl):
    t, head, ends = _serving(fl)
    # drafted tokens that may be accepted: the drafter's most likely ones
    t["tokens"] = fl.fp8_linear(t["x_draft"], *head).float().argmax(1)
    z, zd, r = _serve(fl, t, head)
    base = fl.fp8_linear(t["x"], *head)
    s = torch.einsum("tk,trk->tr", t["x"].double(), t["a"].double()[t["index"]]) * t["scales"].double()[t["index"]][:, None]
    d = torch.einsum("tr,tvr->tv", s, t["b"].double()[t["index"]])
    want = base.double() + torch.where(t["index"] >= 0, 1.0, 0.0)[:, None] * d
    # the sum's rounding to bf16 (2^-8), and what its terms lose before (|s| < 8 sixteen times |b| < 1, 2^-15)
    assert ((z.double() - want).abs() <= 2.0 ** -8 * want.abs() + 16 * 8 * 2.0 ** -15).all()
    zt, zq = z.double().cpu().numpy(), zd.double().cpu().numpy()
    tok, u, ud, temp = (t[k].cpu().numpy() for k in ("tokens", "u", "u_draw", "t"))
    got, acc, prob = r.tokens.cpu().numpy(), r.accepted.cpu().numpy(), r.accept_prob.cpu().numpy()
    off = 4 * 96 * 2.0 ** -24  # (as in the verification's own tests)
    for b in range(5):
        e0, e1 = ends[b], ends[b + 1]
        may = [m for m in request_ref(zt[e0 + b:e1 + b + 1], zq[e0:e1], tok[e0:e1], u[e0:e1], ud[b], temp[b], eps=off) if m[0] == acc[b]]
        assert may and list(got[b][:acc[b]]) == list(tok[e0:e0 + acc[b]])
        w = may[0][1]
        assert draw_error(w, ud[b], got[b][acc[b]]) <= 2 * off / w.sum() if isinstance(w, np.ndarray) else got[b][acc[b]] == w
        for i in range(e0, e1):
            a = accept_ratio(zt[i + b], zq[i], int(tok[i]), temp[b])
            assert abs(prob[i] - a) <= 2 * off * a + 2.0 ** -100
    assert acc.sum() > 0


@gpu
def test_serving_captured(fl):
    t, head, _ = _serving(fl)
    _serve(fl, t, head)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z, zd, r = _serve(fl, t, head)
    for seed in (3, 4):
        new, _, _ = _serving(fl, seed=seed, counts=(2, 4, 0, 1, 3))
        for k in t:
            t[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        z2, zd2, r2 = _serve(fl, t, head)
        assert torch.equal(z, z2) and torch.equal(zd, zd2) and all(torch.equal(p, q) for p, q in zip(r, r2))


@gpu
def test_two_captures_share_no_memory(fl):
    t, head, _ = _serving(fl)
    graphs, results = [], []
    _serve(fl, t, head)
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(_serve(fl, t, head))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(10):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    want = _serve(fl, t, head)
    for got in results:
        assert torch.equal(got[0], want[0]) and all(torch.equal(p, q) for p, q in zip(got[2], want[2]))


@gpu
@pytest.mark.parametrize("handle", [False, True], ids=["Stream", "handle"])
def test_serving_on_streams_at_once(fl, handle):
    ts = [_serving(fl, seed=s) for s in (5, 6)]
    want = [_serve(fl, t, head) for t, head, _ in ts]
    streams = [torch.cuda.Stream() for _ in ts]
    torch.cuda.synchronize()
    got = [[_serve(fl, t, head, stream=s.cuda_stream if handle else s) for (t, head, _), s in zip(ts, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, want):
            assert torch.equal(a[0], b[0]) and all(torch.equal(p, q) for p, q in zip(a[2], b[2]))


@gpu
@pytest.mark.parametrize("name", ["clip", "verify", "adapters"])
def test_memory_is_taken_for_the_stream(fl, name):
    """What the current stream allocates and fills while a call on another stream waits is neither its workspace nor its results."""
    t, head, _ = _serving(fl)
    z, zd, _ = _serve(fl, t, head)
    gs = [torch.randn(5000, device="cuda") for _ in range(3)]
    calls = {"clip": lambda s: [fl.grad_norm(gs, stream=s)],
             "verify": lambda s: list(fl.verify_drafts(z, t["tokens"], t["u"], t["u_draw"], draft_logits=zd, offsets=t["offsets"], max_drafts=4,
                                                       temperature=t["t"], stream=s)),
             "adapters": lambda s: [fl.low_rank_add(z, t["x"], t["a"], t["b"], t["index"], stream=s)]}
    want = calls[name](None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # clock cycles: far longer than the calls
    got = calls[name](side)
    fills = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (16, 512, 4096, 1 << 14, 1 << 16, 1 << 18, 1 << 20) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all(f.eq(255).all() for f in fills)


@gpu
def test_the_example(fl):
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "draft_and_verify.py")
    spec = importlib.util.spec_from_file_location("draft_and_verify", at)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    lines = []
    answers = example.run(7, 128, 1000, 3, 4, log=lines.append)
    assert len(lines) == 4 and len(answers) == 7 and all(4 <= len(a) <= 16 and all(0 <= x < 1000 for x in a) for a in answers)
