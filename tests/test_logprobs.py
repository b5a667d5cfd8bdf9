"""Token log probabilities: the float64 oracle's own pins and the refusals (CPU), and
the GPU library against the oracle over head sizes, ragged vocabularies, ties, masked
and empty rows, strides, chunks and streams."""
import math

import numpy as np
import pytest
import torch

from oracle import lp_grad_ref, lp_rows_ref
from parity_util import f64, rel_fro

gpu = pytest.mark.gpu
IGN = -100

# A product on the tensor cores adds 16 products at a time to an fp32 sum; taking each
# of those additions as off by one step of the sum (2^-23 of its size), a logit is off
# by at most (H / 16) 2^-23 times the largest partial sum, itself at most sum |x w|.
# Everything after it is fp32: ex2/lg2 are good to 2^-22, and sums over V in trees add
# about log2(V) + V / (parts * threads) steps; 2^-18 covers both.
EPS32 = 2.0 ** -18


def _logit_bound(x, w, t):
    mag = (x.abs().double().cpu() @ w.abs().double().cpu().T).max().item()
    return (x.shape[1] / 16 + 2) * 2.0 ** -23 * mag / t


# three roundings to bf16 on the way (probabilities, dz, the result), each at most
# eps / 2 = 2^-8 of its value
GRAD_TOL = {torch.bfloat16: 3 * 2.0 ** -8, torch.float32: 1e-5}


def _inputs(bt, h, v, dtype, seed, grid=False, ignored=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(bt, h, generator=g)
    w = torch.randn(v, h, generator=g) * (3 / math.sqrt(h))
    if grid:  # sums exact in 32 bits: the ranks are a matter of the inputs alone
        x = (x * 16).round().clamp(-64, 64) / 16
        u = 2.0 ** round(math.log2(0.375 / math.sqrt(h)))
        w = (w / u).round().clamp(-32, 32) * u
    y = torch.randint(0, v, (bt,), generator=g)
    y[torch.rand(bt, generator=g) < ignored] = IGN
    return x.to(dtype), w.to(dtype), y


def _close(got, ref, atol, what):
    got, ref = f64(got), np.asarray(ref)
    assert np.array_equal(np.isfinite(got), np.isfinite(ref)), what
    ok = np.isfinite(ref)
    assert np.array_equal(got[~ok], ref[~ok], equal_nan=True), what
    err = np.abs(got[ok] - ref[ok])
    lim = atol + EPS32 * np.maximum(1.0, np.abs(ref[ok]))
    assert (err <= lim).all(), f"{what}: off by {err.max()} (limit {lim.min()})"


def _check_rows(r, ref, atol, what, ids=True):
    for name, got, want in zip(("logp", "entropy", "lse", "top_logp"), (*r[:3], r[4]), ref[:4]):
        if want is None:
            assert got is None
        else:
            # entropy: a sum of p log p, moved by z's error times log V at most
            a = atol * (1 + math.log(2 ** 17)) if name == "entropy" else 2 * atol
            _close(got, want, a, f"{what} {name}")
    if ref[4] is not None and ids:
        assert np.array_equal(r[5].cpu().numpy(), ref[4]), f"{what} top_id"


# ---- the oracle ----
def test_oracle_rows_against_torch():
    z = torch.randn(5, 40, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    y = torch.tensor([3, IGN, 39, 0, 40])
    logp, ent, lse, tl, ti = lp_rows_ref(z.numpy(), y.numpy(), top_k=4, temperature=0.7)
    ref = torch.log_softmax(z / 0.7, 1)
    assert np.allclose(lse, torch.logsumexp(z / 0.7, 1), rtol=1e-14)
    assert np.allclose(logp, [ref[0, 3], 0, ref[2, 39], ref[3, 0], 0], rtol=1e-13)
    e = torch.distributions.Categorical(logits=z / 0.7).entropy()
    assert np.allclose(ent, [e[0], 0, e[2], e[3], 0], rtol=1e-12)
    top = ref.topk(4, 1)
    assert np.array_equal(ti, top.indices) and np.allclose(tl, top.values, rtol=1e-13)


def test_oracle_ties_masks_and_empty_rows():
    z = np.array([[1.0, 2.0, 2.0, -np.inf, 2.0], [-np.inf] * 5, [0.0, -np.inf, -np.inf, -np.inf, 0.0]])
    logp, ent, lse, tl, ti = lp_rows_ref(z, np.array([3, 0, 4]), top_k=4)
    assert ti.tolist() == [[1, 2, 4, 0], [-1] * 4, [0, 4, -1, -1]]
    assert logp[0] == -np.inf and logp[1] == -np.inf and logp[2] == pytest.approx(-math.log(2))
    assert ent[1] == 0 and ent[2] == pytest.approx(math.log(2)) and lse[1] == -np.inf
    dz = lp_grad_ref(z, np.array([3, 0, 4]), np.ones(3), np.ones(3))
    assert np.isfinite(dz).all() and not dz[1].any() and dz[0, 3] == 1.0


@pytest.mark.parametrize("t", [1.0, 0.5, 2.0])
def test_oracle_gradient_against_differences(t):
    rng = np.random.default_rng(2)
    z, y = rng.normal(size=(3, 7)), np.array([2, IGN, 6])
    a, b = rng.normal(size=3), rng.normal(size=3)

    def f(z):
        logp, ent, *_ = lp_rows_ref(z, y, temperature=t)
        return (a * logp + b * ent).sum()

    dz = lp_grad_ref(z, y, a, b, temperature=t)
    for i in np.ndindex(*z.shape):
        h = np.zeros_like(z)
        h[i] = 1e-5
        assert (f(z + h) - f(z - h)) / 2e-5 == pytest.approx(dz[i], rel=1e-7, abs=1e-9)


# ---- plans and refusals (no GPU) ----
@pytest.fixture(scope="module")
def L():
    from conftest import build_library

    build_library()
    from lm_head_jsd_gb300 import _lib

    return _lib


@pytest.mark.parametrize("kw,status", [
    (dict(bt=0), 1), (dict(h=-1), 1), (dict(v=0), 1), (dict(top_k=-1), 1), (dict(top_k=101), 1),
    (dict(temperature=0.0), 1), (dict(temperature=float("nan")), 1),
    (dict(temperature=float("inf")), 1), (dict(temperature=1e-40), 1), (dict(dtype=7), 1), (dict(chunk_rows=-1), 1),
    (dict(v=1 << 31), 2), (dict(v=1000, top_k=33), 2), (dict(h=1 << 21), 2)])
def test_plan_refusals(L, kw, status):
    base = dict(bt=4, h=64, v=100, dtype="bf16")
    with pytest.raises(L.FljsdError) as e:
        L.fljsd_lp_plan(L.make_lp_problem(**{**base, **kw}))
    assert e.value.status == status


@pytest.mark.parametrize("h", [64, 12])
@pytest.mark.parametrize("backward", [False, True])
def test_plan_chunks_fit_the_budget(L, h, backward):
    p = L.make_lp_problem(5000, h, 32000, "bf16", top_k=4, backward=backward)
    whole = L.fljsd_lp_plan(p)
    assert whole.num_chunks == 1
    for budget in (whole.workspace_bytes, whole.workspace_bytes // 3, whole.workspace_bytes // 50):
        plan = L.fljsd_lp_plan(p, 2 * budget)
        assert plan.workspace_bytes <= budget
        assert plan.num_chunks == -(-5000 // plan.chunk_rows)
    with pytest.raises(L.FljsdError) as e:
        L.fljsd_lp_plan(p, 4096)
    assert e.value.status == 3


def test_call_refusals_launch_nothing(L):
    buf = 4096  # an aligned address that is never read: every call below is refused
    p = L.make_lp_problem(4, 64, 100, "bf16", top_k=2)
    plan = L.fljsd_lp_plan(p)
    n = plan.workspace_bytes

    def fwd(x=buf, w=buf, y=buf, lp=buf, en=buf, ls=buf, nm=buf, tl=buf, ti=buf, ws=buf, nb=n, plan=plan):
        return L.fljsd_lp_forward(p, plan, x, w, y, lp, en, ls, nm, tl, ti, ws, nb, 0, False)

    for bad in (dict(x=None), dict(w=None), dict(lp=None), dict(en=None), dict(ls=None), dict(nm=None), dict(nm=buf + 4),
                dict(tl=None), dict(ti=None), dict(ws=None), dict(x=buf + 8), dict(y=buf + 4),
                dict(ws=buf + 8), dict(lp=buf + 2)):
        assert fwd(**bad) == 1, bad
    assert fwd(nb=n - 1) == 3
    other = L.fljsd_lp_plan(L.make_lp_problem(4, 64, 108, "bf16", top_k=2))
    assert fwd(plan=other) == 1

    def bwd(problem, plan, kept=0, y=buf, gl=buf, gx=buf, gw=buf):
        return L.fljsd_lp_backward(problem, plan, buf, buf, y, buf, buf, buf, gl, buf, kept, gx, gw,
                                   buf, plan.workspace_bytes, 0, False)

    assert bwd(p, plan) == 1  # a plan without FLJSD_LP_BACKWARD
    q = L.make_lp_problem(4, 64, 100, "bf16", backward=True, chunk_rows=2)
    qp = L.fljsd_lp_plan(q)
    assert bwd(q, qp, kept=1) == 1  # two chunks keep nothing
    assert bwd(q, qp, kept=2) == 1
    assert bwd(q, qp, y=None) == 1  # grad_logp without labels
    assert bwd(q, qp, gx=None, gw=None) == 1
    rows = dict(rows=4, v=100, ld=100, dtype="bf16", top_k=2, temperature=1.0)

    def logits(z=buf, nb=1 << 20, **kw):
        a = {**rows, **kw}
        return L.fljsd_logits_lp(a["rows"], a["v"], a["ld"], a["dtype"], a["top_k"], a["temperature"],
                                 IGN, z, buf, buf, buf, buf, buf, buf, buf, buf, nb, 0, False)

    for bad in (dict(rows=0), dict(v=-3), dict(ld=99), dict(dtype=5), dict(top_k=101),
                dict(temperature=-1.0), dict(z=None), dict(z=buf + 1)):
        assert logits(**bad) == 1, bad
    assert logits(v=1000, ld=1000, top_k=33) == 2
    assert logits(nb=16) == 3


# ---- GPU: the fused product ----
def _fused(x, w, y, dev="cuda", **kw):
    from lm_head_jsd_gb300 import FusedLinearLogprobs

    run = FusedLinearLogprobs(x.shape[0], x.shape[1], w.shape[0], x.dtype, device=dev, **kw)
    args = x.to(dev), w.to(dev), None if y is None else y.to(dev)
    return run, args, run.forward(*args)


# one token to several tiles (up to 16 rows by the product for few rows, its x kept in
# shared memory up to h of about 4300), odd vocabularies, rows that fill half a pair, hidden sizes
# of less than one k-block; (_, 12, _) and fp32 run on the CUDA cores
SHAPES = [(1, 64, 1000), (1, 512, 32000), (2, 8, 33), (7, 136, 129), (33, 64, 4099), (128, 256, 2048),
          (129, 320, 1027), (257, 512, 513), (300, 1024, 5000), (5, 12, 777), (3, 16, 1),
          (16, 4096, 700), (17, 4096, 700), (15, 8200, 300)]


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_fused_forward(shape, dtype):
    bt, h, v = shape
    x, w, y = _inputs(bt, h, v, dtype, 10 + bt, grid=True, ignored=0.2 if bt > 4 else 0.0)
    k = min(v, (0, 1, 5, 8, 20, 32)[bt % 6])
    t = (1.0, 0.5, 1.7)[bt % 3]
    run, args, r = _fused(x, w, y, top_k=k, temperature=t)
    ref = lp_rows_ref(f64(x) @ f64(w).T, y.numpy(), top_k=k, temperature=t)
    _check_rows(r, ref, _logit_bound(x, w, t), str(shape))
    from lm_head_jsd_gb300 import fljsd_workspace_status

    assert fljsd_workspace_status(run.plan, run.workspace) == 0


@gpu
@pytest.mark.parametrize("k", [1, 8, 9, 32])
def test_fused_alternatives_ties_and_order(k):
    # every logit of a row equal; ascending and descending ids; all k in one tile
    h, v = 64, 3000
    x = torch.zeros(4, h)
    x[:, 0] = 1.0
    x[1, 1], x[2, 1] = 1.0, -1.0
    x[3, 2] = 1.0
    w = torch.zeros(v, h)
    w[:, 0] = 2.0
    w[:, 1] = torch.arange(v).div(16, rounding_mode="floor").float()  # runs of 16 equal logits
    w[700:800, 2] = 1.0
    x, w = x.bfloat16(), w.bfloat16()
    _, _, r = _fused(x, w, None, top_k=k)
    ref = lp_rows_ref(f64(x) @ f64(w).T, None, top_k=k)
    assert r.logp is None
    assert np.array_equal(r.top_id.cpu().numpy(), ref[4])
    _check_rows(r, ref, _logit_bound(x, w, 1.0), "ties")


@gpu
@pytest.mark.parametrize("bt,v", [(1, 128256), (5, 70001), (130, 50000), (300, 40960)])
def test_fused_alternatives_at_length(bt, v):
    """Thresholds, written-out columns and read-again chunks at a vocabulary's length,
    the largest logits all in one place or spread out."""
    h, k = 64, 20
    x, w, y = _inputs(bt, h, v, torch.bfloat16, 40 + bt, grid=True)
    w[v - 90:] = w[v - 90:] * 2  # the last part holds most of them
    w[1000:1040, 0] = 8.0
    x[0, 0] = 4.0  # one row: equal logits far above the rest
    x[0, 1:] = 0
    _, _, r = _fused(x, w, y, top_k=k)
    ref = lp_rows_ref(f64(x) @ f64(w).T, y.numpy(), top_k=k)
    _check_rows(r, ref, _logit_bound(x, w, 1.0), f"{bt}x{v}")


@gpu
def test_fused_unusual_rows():
    from lm_head_jsd_gb300 import fljsd_workspace_status

    x, w, y = _inputs(6, 64, 500, torch.bfloat16, 3)
    x[0] = 0  # uniform
    x[1] = float("nan")
    x[2, 0] = float("inf")
    w[:, 0] = w[:, 0].abs() + 0.01
    x[3] *= 300  # one token takes all
    y[4], y[5] = 500, 0
    run, _, r = _fused(x, w, y, top_k=3)
    z = f64(x) @ f64(w).T
    ref = lp_rows_ref(z[[0, 3, 4, 5]], y.numpy()[[0, 3, 4, 5]], top_k=3)
    keep = [0, 3, 4, 5]
    _check_rows([None if t is None else t[keep] for t in r], ref, _logit_bound(x[keep], w, 1.0), "unusual")
    assert torch.isnan(r.logp[1]) and torch.isnan(r.entropy[1]) and torch.isnan(r.lse[1:3]).all()
    assert r.top_id[1].tolist() == [-1] * 3
    assert fljsd_workspace_status(run.plan, run.workspace) == 1  # label 500


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(1, 64, 1000), (5, 12, 777), (129, 320, 1027), (300, 256, 4099)],
                         ids=lambda s: "x".join(map(str, s)))
def test_fused_gradient(shape, dtype):
    bt, h, v = shape
    x, w, y = _inputs(bt, h, v, dtype, 20 + bt, ignored=0.2 if bt > 4 else 0.0)
    g = torch.Generator().manual_seed(5)
    a, b = torch.randn(bt, generator=g), torch.randn(bt, generator=g)
    run, args, r = _fused(x, w, y, temperature=1.3, keep_for_backward=True)
    dz = lp_grad_ref(f64(x) @ f64(w).T, y.numpy(), a.numpy(), b.numpy(), temperature=1.3)
    first = run.backward(*args, r, a.cuda(), b.cuda())
    again = run.backward(*args, r, a.cuda(), b.cuda())  # computed again
    tol = GRAD_TOL[dtype]
    for gx, gw in (first, again):
        assert rel_fro(f64(gx), dz @ f64(w)) <= tol
        assert rel_fro(f64(gw), dz.T @ f64(x)) <= tol
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    if bt > 4:
        assert (y == IGN).any() and not f64(first[0])[(y == IGN).numpy()].any()
    # one of the two gradients, and one of the two upstream gradients
    r = run.forward(*args)
    gx, gw = run.backward(*args, r, a.cuda(), need=(True, False))
    dza = lp_grad_ref(f64(x) @ f64(w).T, y.numpy(), a.numpy(), None, temperature=1.3)
    assert gw is None and rel_fro(f64(gx), dza @ f64(w)) <= tol
    gx, gw = run.backward(*args, r, None, b.cuda(), need=(False, True))
    dzb = lp_grad_ref(f64(x) @ f64(w).T, y.numpy(), None, b.numpy(), temperature=1.3)
    assert gx is None and rel_fro(f64(gw), dzb.T @ f64(x)) <= tol


@gpu
@pytest.mark.parametrize("dtype,acc", [(torch.bfloat16, False), (torch.bfloat16, True), (torch.float32, False)])
def test_fused_chunks(dtype, acc):
    x, w, y = _inputs(70, 64, 1000, dtype, 30, grid=True, ignored=0.1)
    a, b = torch.randn(70).cuda(), torch.randn(70).cuda()
    run, args, r = _fused(x, w, y, top_k=4, keep_for_backward=True)
    one = run.backward(*args, r, a, b)
    cut, _, rc = _fused(x, w, y, top_k=4, keep_for_backward=True, chunk_rows=32, accum_fp32=acc)
    assert cut.plan.num_chunks == 3
    assert all(torch.equal(p, q) for p, q in zip(r, rc))
    gx, gw = cut.backward(*args, rc, a, b)
    assert torch.equal(gx, one[0])
    # two more roundings of the running sum, or none
    tol = 1e-6 if dtype == torch.float32 else 2.0 ** -8 * (1 if acc else 3)
    assert rel_fro(f64(gw), f64(one[1])) <= tol


@gpu
def test_fused_is_deterministic_and_stream_safe():
    x, w, y = _inputs(200, 512, 9000, torch.bfloat16, 31, ignored=0.1)
    run, args, r = _fused(x, w, y, top_k=8, keep_for_backward=True)
    a = torch.randn(200).cuda()
    g = run.backward(*args, r, a)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            r2 = run.forward(*args)
            g2 = run.backward(*args, r2, a)
            assert all(torch.equal(p, q) for p, q in zip(r, r2))
            assert torch.equal(g[0], g2[0]) and torch.equal(g[1], g2[1])


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_fused_autograd(dtype):
    from lm_head_jsd_gb300 import fused_linear_logprobs

    x, w, y = _inputs(40, 64, 300, dtype, 33, ignored=0.2)
    xr, wr = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    r = fused_linear_logprobs(xr, wr, y.cuda(), top_k=2, temperature=0.8)
    assert not r.top_logp.requires_grad and not r.lse.requires_grad
    loss = r.logp.mean() + 0.1 * r.entropy.sum()
    loss.backward(retain_graph=True)
    dz = lp_grad_ref(f64(x) @ f64(w).T, y.numpy(), np.full(40, 1 / 40), np.full(40, 0.1), temperature=0.8)
    tol = GRAD_TOL[dtype]
    assert rel_fro(f64(xr.grad), dz @ f64(w)) <= tol and rel_fro(f64(wr.grad), dz.T @ f64(x)) <= tol
    g1 = xr.grad.clone()
    xr.grad = None
    loss.backward()
    assert torch.equal(xr.grad, g1)
    with torch.no_grad():
        assert not fused_linear_logprobs(xr, wr, y.cuda()).logp.requires_grad
    frozen = fused_linear_logprobs(xr, wr.detach(), y.cuda())
    (gx,) = torch.autograd.grad(frozen.logp.sum(), xr)
    dz = lp_grad_ref(f64(x) @ f64(w).T, y.numpy(), np.ones(40), None)
    assert rel_fro(f64(gx), dz @ f64(w)) <= tol


@gpu
def test_fused_step_in_a_graph():
    x, w, y = _inputs(96, 128, 2000, torch.bfloat16, 34, ignored=0.1)
    run, args, r = _fused(x, w, y, top_k=4, keep_for_backward=True)
    a, b = torch.randn(96).cuda(), torch.randn(96).cuda()
    g = run.backward(*args, r, a, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rg = run.forward(*args)
        gg = run.backward(*args, rg, a, b)
    for t in (*rg, *gg):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(r, rg)) and all(torch.equal(p, q) for p, q in zip(g, gg))


@gpu
def test_fused_autograd_in_a_graph_beside_an_eager_one():
    from lm_head_jsd_gb300 import fused_linear_logprobs

    x, w, y = _inputs(50, 64, 400, torch.bfloat16, 35, ignored=0.1)
    xr, wr, yc = x.cuda().requires_grad_(), w.cuda().requires_grad_(), y.cuda()
    eager = fused_linear_logprobs(xr, wr, yc)  # its graph stays alive
    want = torch.autograd.grad(fused_linear_logprobs(xr, wr, yc).logp.sum(), (xr, wr))
    def step():
        leaves = xr.detach().requires_grad_(), wr.detach().requires_grad_()  # of the capture's own
        return torch.autograd.grad(fused_linear_logprobs(*leaves, yc).logp.sum(), leaves)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    eager.logp.sum().backward()
    assert torch.equal(xr.grad, want[0]) and torch.equal(wr.grad, want[1])


@gpu
def test_fused_offsets_past_32_bits():
    """More than 2^31 probabilities kept for the backward pass; rows and gradients of the
    end are those of the end alone."""
    from lm_head_jsd_gb300 import FusedLinearLogprobs

    bt, h, v, last = 17000, 64, 130000, 700  # (as many rows as are joined in the same order)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(bt, h, device="cuda", generator=g).bfloat16()
    w = torch.randn(v, h, device="cuda", generator=g).div_(2).bfloat16()
    y = torch.randint(0, v, (bt,), device="cuda", generator=g)
    a = torch.randn(bt, device="cuda", generator=g)
    run = FusedLinearLogprobs(bt, h, v, top_k=4, keep_for_backward=True)
    assert run.plan.num_chunks == 1
    r = run.forward(x, w, y)
    gx, _ = run.backward(x, w, y, r, a, need=(True, False))
    tail = FusedLinearLogprobs(last, h, v, top_k=4, keep_for_backward=True)
    s = slice(bt - last, bt)
    q = tail.forward(x[s], w, y[s])
    hx, _ = tail.backward(x[s], w, y[s], q, a[s].contiguous(), need=(True, False))
    assert all(torch.equal(t[s], u) for t, u in zip(r, q))
    # (the product over v may be split differently for few rows)
    assert rel_fro(f64(gx[s]), f64(hx)) <= 2.0 ** -8


# ---- GPU: given logits ----
@gpu
def test_logits_offsets_past_32_bits():
    from lm_head_jsd_gb300 import logits_logprobs, logits_logprobs_backward

    rows, v = 17000, 128256
    z = torch.empty(rows, v, dtype=torch.bfloat16, device="cuda").normal_(0, 3)
    y = torch.randint(0, v, (rows,), device="cuda")
    r = logits_logprobs(z, y, top_k=3)
    n = 700  # (as many rows as are joined in the same order)
    q = logits_logprobs(z[-n:], y[-n:], top_k=3)
    assert all(torch.equal(t[-n:], u) for t, u in zip(r, q))
    a = torch.randn(rows, device="cuda")
    want = logits_logprobs_backward(z[-n:], y[-n:], q, a[-n:].contiguous())
    assert torch.equal(logits_logprobs_backward(z, y, r, a, out=z)[-n:], want)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("rows,v,k", [(1, 1, 1), (1, 8190, 8), (2, 8192, 32), (3, 8193, 20), (5, 8191, 0),
                                      (40, 77, 5), (1, 128256, 8), (3, 32001, 1), (2, 128255, 32)])
def test_logits_rows(rows, v, k, dtype):
    from lm_head_jsd_gb300 import logits_logprobs, logits_logprobs_backward

    g = torch.Generator().manual_seed(rows * 7 + v)
    z = (3 * torch.randn(rows, v, generator=g)).to(dtype)
    y = torch.randint(0, v, (rows,), generator=g)
    if rows > 2:
        y[1] = IGN
    a, b = torch.randn(rows, generator=g), torch.randn(rows, generator=g)
    zc, yc = z.cuda(), y.cuda()
    r = logits_logprobs(zc, yc, top_k=k, temperature=0.9)
    _check_rows(r, lp_rows_ref(f64(z), y.numpy(), top_k=k, temperature=0.9), 0.0, f"{rows}x{v}")
    dz = logits_logprobs_backward(zc, yc, r, a.cuda(), b.cuda(), temperature=0.9)
    ref = lp_grad_ref(f64(z), y.numpy(), a.numpy(), b.numpy(), temperature=0.9)
    tol = 1e-5 if dtype == torch.float32 else 2.0 ** -8
    assert rel_fro(f64(dz), ref) <= tol
    same = logits_logprobs_backward(zc, yc, r, a.cuda(), b.cuda(), temperature=0.9, out=zc)
    assert same.data_ptr() == zc.data_ptr() and torch.equal(same, dz)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("k", [1, 8, 32])
def test_logits_masks_ties_strides(dtype, k):
    from lm_head_jsd_gb300 import logits_logprobs, logits_logprobs_backward

    v = 20011
    z = torch.randn(9, v, generator=torch.Generator().manual_seed(4))
    low = torch.finfo(dtype).min
    z[0] = -math.inf  # nothing left
    z[1, :] = -math.inf
    z[1, 17], z[1, 20000] = 1.0, 1.0  # two left
    z[2, ::2] = -math.inf
    z[3, 1:] = low  # masked by the type's lowest value
    z[4] = low
    z[5] = 1.5  # all equal
    z[6, 9000:] = 2.0
    z[7, 5] = math.nan
    z[8, 6] = math.inf
    y = torch.tensor([3, 17, 1, 0, 8, 20010, 9000, 0, 0])
    z = z.to(dtype)
    wide = torch.full((9, v + 5), 7.0, dtype=dtype)
    wide[:, 3:3 + v] = z
    zc, yc = wide.cuda()[:, 3:3 + v], y.cuda()
    r = logits_logprobs(zc, yc, top_k=k)
    ref = lp_rows_ref(f64(z[:7]), y.numpy()[:7], top_k=k)
    _check_rows([t[:7] for t in r], ref, 0.0, "masks")
    assert torch.isnan(r.logp[7:]).all() and torch.isnan(r.lse[7:]).all() and torch.isnan(r.entropy[7:]).all()
    assert 5 not in r.top_id[7].tolist() and r.top_id[8, 0] == 6
    a, b = torch.randn(9), torch.randn(9)
    dz = logits_logprobs_backward(zc[:7], yc[:7], type(r)(*(t[:7] for t in r)), a.cuda()[:7], b.cuda()[:7])
    refg = lp_grad_ref(f64(z[:7]), y.numpy()[:7], a.numpy(), b.numpy())
    assert np.isfinite(f64(dz)).all() and rel_fro(f64(dz), refg) <= (1e-5 if dtype == torch.float32 else 2.0 ** -8)


@gpu
def test_logits_autograd_and_refusals():
    from lm_head_jsd_gb300 import logits_logprobs, token_logprobs

    z = torch.randn(6, 50, dtype=torch.float64, generator=torch.Generator().manual_seed(6))
    y = torch.tensor([1, 2, IGN, 4, 5, 49])
    zr = z.float().cuda().requires_grad_()
    r = token_logprobs(zr, y.cuda(), top_k=3)
    (r.logp.sum() * 2 - r.entropy.mean()).backward()  # (the upstream gradients are expanded scalars)
    ref = lp_grad_ref(z.float().numpy(), y.numpy(), np.full(6, 2.0), np.full(6, -1 / 6))
    assert rel_fro(f64(zr.grad), ref) <= 1e-5
    one = z.float().cuda()[:1].requires_grad_()
    wide = token_logprobs(one.expand(3, 50), torch.tensor([1, 2, 3]).cuda())  # rows share memory
    wide.logp.sum().backward()
    refw = lp_grad_ref(z[:1].expand(3, 50).float().numpy(), np.array([1, 2, 3]), np.ones(3), None)
    assert rel_fro(f64(one.grad), refw.sum(0, keepdims=True)) <= 1e-5
    zt = z.float().cuda().T.contiguous().T.requires_grad_()  # columns contiguous
    r2 = token_logprobs(zt, y.cuda())
    r2.logp.sum().backward()
    assert torch.equal(r2.logp, r.logp)
    with pytest.raises(ValueError):
        logits_logprobs(zt.detach(), y.cuda())
    with pytest.raises(ValueError):
        logits_logprobs(zr.detach(), y.cuda().int())
    with pytest.raises(ValueError):
        logits_logprobs(zr.detach(), y.cuda()[:5])
    with pytest.raises(ValueError):
        logits_logprobs(zr.detach().half(), y.cuda())
