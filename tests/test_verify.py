"""Drafted tokens verified from given random numbers: the oracle's pins and the refusals (CPU), and the GPU
against the float64 oracle, over types, odd and unaligned rows, ragged requests, masks and bad rows, and
against the same whole numbers in torch, bit by bit."""
import itertools
import math

import numpy as np
import pytest
import torch

from oracle.verify_oracle import accept_ratio, draw_error, draw_weights, first_largest, probabilities, request_ref

gpu = pytest.mark.gpu
BF, INF, NAN = torch.bfloat16, math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def fl():
    from conftest import build_library

    build_library()
    import lm_head_jsd_gb300 as fl

    return fl


# ---- the oracle ----
def test_oracle_tokens_follow_the_target():
    """Whatever the draft, accepted and drawn together have the target's probabilities: summed exactly."""
    rng = np.random.default_rng(0)
    for _ in range(20):
        zt, zd, t = rng.normal(size=7) * 2, rng.normal(size=7) * 2, 0.7
        p, q = probabilities(zt, t), probabilities(zd, t)
        got = np.zeros(7)
        for d in range(7):
            a = accept_ratio(zt, zd, d, t)
            got[d] += q[d] * a
            r = draw_weights(p, q)
            got += q[d] * (1 - a) * r / r.sum()
        assert np.allclose(got, p, atol=1e-14)


def test_oracle_without_draft_probabilities():
    zt = np.array([0.0, 1.0, -INF, 2.0])
    p = probabilities(zt, 1.0)
    q = np.eye(4)[1]
    a = accept_ratio(zt, None, 1, 1.0)
    r = draw_weights(p, q)
    assert a == p[1] and r[1] == 0 and np.allclose(a * q + (1 - a) * r / r.sum(), p)
    assert accept_ratio(zt, None, 2, 1.0) == 0 and accept_ratio(zt, None, 4, 1.0) == 0
    assert accept_ratio(zt, None, 3, 0) == 1 and first_largest([1.0, 3.0, 3.0]) == 1
    assert probabilities([-INF, -INF], 1.0) is None and probabilities([NAN, 1.0], 1.0) is None


def test_oracle_runs():
    zt = np.array([[5.0, 0.0], [5.0, 0.0], [0.0, 5.0]])
    ref = lambda tok, u, **kw: request_ref(zt, None, tok, u, 0.5, 1.0, **kw)  # noqa: E731
    assert [r[0] for r in ref([0, 0], [0.1, 0.1])] == [2]
    assert [r[0] for r in ref([0, 1], [0.1, 0.9])] == [1]
    p = probabilities(zt[0], 1.0)[0]
    assert [r[0] for r in ref([0, 1], [p, 0.9], eps=1e-6)] == [0, 1]
    assert [r[0] for r in ref([0, 1], [NAN, 0.9])] == [0]
    assert draw_error(np.array([1.0, 3.0]), 0.25, 1) == 0 and draw_error(np.array([1.0, 3.0]), 0.35, 0) == pytest.approx(0.1)


# ---- refusals (no GPU) ----
GOOD = dict(requests=2, drafts=4, v=100, max_drafts=2, dtype=1, target=4096, ld_target=100, draft=8192, ld_draft=100,
            tokens=64, u_accept=64, u_draw=64, offsets=None, temperatures=None, temperature=1.0, out=64, accepted=64,
            accept_prob=64, workspace=4096, workspace_bytes=1 << 20)
BAD = [dict(requests=0), dict(drafts=-1), dict(v=0), dict(max_drafts=-1), dict(dtype=2), dict(target=None), dict(target=4097),
       dict(draft=8193), dict(ld_target=99), dict(ld_draft=99), dict(tokens=None), dict(tokens=68), dict(u_accept=None),
       dict(u_accept=66), dict(u_draw=None), dict(u_draw=66), dict(offsets=68), dict(temperatures=66), dict(temperature=-1.0),
       dict(temperature=NAN), dict(temperature=INF), dict(temperature=1e-40), dict(out=None), dict(out=68), dict(accepted=None), dict(accepted=4),
       dict(accept_prob=None), dict(accept_prob=66), dict(workspace=None), dict(workspace=8), dict(drafts=3), dict(max_drafts=3)]


@pytest.mark.parametrize("bad", BAD, ids=str)
def test_refused(fl, bad):
    assert fl.fljsd_verify(**{**GOOD, **bad}, stream=0, check=False) == 1


def test_refused_sizes(fl):
    call = lambda **kw: fl.fljsd_verify(**{**GOOD, **kw}, stream=0, check=False)  # noqa: E731
    assert call(v=1 << 20, ld_target=1 << 20, ld_draft=1 << 20) == 2
    assert call(requests=(1 << 20) + 1, offsets=64) == 2 and call(drafts=(1 << 24) + 1, offsets=64) == 2
    assert call(max_drafts=1025, offsets=64) == 2 and call(requests=1 << 20, max_drafts=200, offsets=64) == 2
    assert call(workspace_bytes=fl.fljsd_verify_workspace_bytes(2, 4) - 1) == 3


def test_refused_in_python(fl):
    z, n = torch.zeros(6, 10), 4
    tok, u, ud = torch.zeros(n).long(), torch.zeros(n), torch.zeros(2)
    with pytest.raises(ValueError, match="expected a CUDA device"):
        fl.verify_drafts(z, tok, u, ud)
    with pytest.raises(ValueError, match="target_logits"):
        fl.verify_drafts(z.double(), tok, u, ud)


# ---- on the GPU ----
# A weight's relative error: 2^-22 of the exponential, and three roundings of its argument x (the difference, log2(e) / T
# and their product), 3 ln 2 2^-24 |x|; below 2^-44 it counts as nothing, so |x| <= 44 and it is at most 96 2^-24. A
# probability has this twice. The difference's rounding and its count's (2^-44 for each column) stay far below.
W = 96 * 2.0 ** -24
P = 2 * W


def _check(r, zt, zd, tok, u, ud, ends, t, kmax):
    """Every request's result against the oracle. zt, zd: tensors of any type; t: a number for each request."""
    zt = zt.double().cpu().numpy()
    zd = None if zd is None else zd.double().cpu().numpy()
    got, acc, prob = r.tokens.cpu().numpy(), r.accepted.cpu().numpy(), r.accept_prob.double().cpu().numpy()
    assert got.shape == (len(acc), kmax + 1) and got.dtype == np.int64 and acc.dtype == np.int64
    v = zt.shape[1]
    for b in range(len(acc)):
        s, e = ends[b], ends[b + 1]
        k = e - s
        rows, drows = zt[s + b:e + b + 1], None if zd is None else zd[s:e]
        may = request_ref(rows, drows, tok[s:e], u[s:e], ud[b], t[b], eps=2 * P)
        at = [m for m in may if m[0] == acc[b]]
        assert at, (b, acc[b], [m[0] for m in may])
        n, w = at[0]
        assert list(got[b][:n]) == list(tok[s:s + n]) and (got[b][n + 1:] == -1).all()
        if isinstance(w, np.ndarray):
            # a column's part of p - q is off by P (p + q) at most, its border by the sum of that over the columns
            off = (2 * P + 2 * v * 2.0 ** -43) / w.sum()
            un = min(max(0.0 if ud[b] != ud[b] else ud[b], 0.0), 1.0)
            assert draw_error(w, un, got[b][n]) <= 2 * off
        else:
            assert got[b][n] == w
        for i in range(k):
            a = accept_ratio(rows[i], None if drows is None else drows[i], int(tok[s + i]), t[b])
            assert abs(prob[s + i] - a) <= 2 * P * a + 2.0 ** -24 * a + 2.0 ** -126, (b, i, prob[s + i], a)


def _make(counts, v, dtype, seed=0, draft=True, std=3.0, near=0.7):
    g = torch.Generator().manual_seed(seed)
    n, b = sum(counts), len(counts)
    ends = np.concatenate([[0], np.cumsum(counts)]).astype(int)
    zt = (torch.randn(n + b, v, generator=g) * std).to(dtype)
    rows = [i for j in range(b) for i in range(ends[j] + j, ends[j + 1] + j)]
    zd = (zt[rows].float() + near * torch.randn(n, v, generator=g)).to(dtype) if draft else None
    from_ = torch.softmax((zd if draft else zt[rows]).float(), 1)
    tok = torch.multinomial(from_, 1, generator=g)[:, 0] if n else torch.zeros(0).long()
    return zt, zd, tok, torch.rand(n, generator=g), torch.rand(b, generator=g), ends


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _run(fl, zt, zd, tok, u, ud, ends, t=1.0, ragged=True, **kw):
    zt, zd, tok, u, ud = _cuda(zt, zd, tok, u, ud)
    if ragged:
        kw.setdefault("max_drafts", int(np.diff(ends).max()))
        kw["offsets"] = torch.tensor(ends).cuda()
    return fl.verify_drafts(zt, tok, u, ud, draft_logits=zd, temperature=t.cuda() if torch.is_tensor(t) else t, **kw)


@gpu
@pytest.mark.parametrize("draft", [True, False], ids=["draft", "lookup"])
@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("counts,v", [([4], 1), ([1, 0, 3], 2), ([0], 37), ([2] * 5, 1000), ([3, 0, 7, 1], 5003), ([1, 2], 16384),
                                      ([5], 32771), ([2, 1], 131073)])
def test_against_the_oracle(fl, counts, v, dtype, draft):
    x = _make(counts, v, dtype, seed=v, draft=draft)
    for t in (1.0, 0.6, 0.0):
        r = _run(fl, *x, t=t)
        _check(r, *x[:2], x[2].numpy(), x[3].numpy(), x[4].numpy(), x[5],
               [np.float32(t)] * len(counts), max(counts))
    if len(set(counts)) == 1:
        a, b = _run(fl, *x), _run(fl, *x, ragged=False)
        assert all(torch.equal(p, q) for p, q in zip(a, b))


@gpu
def test_longest_rows(fl):
    v = (1 << 20) - 1
    for dtype in (torch.float32, BF):
        x = _make([1], v, dtype, seed=1)
        r = _run(fl, *x)
        _check(r, *x[:2], x[2].numpy(), x[3].numpy(), x[4].numpy(), x[5], [1.0], 1)
    flat = torch.zeros(2, v)  # all alike: the largest sum, and the last column
    tok = torch.tensor([5])
    r = _run(fl, flat, None, tok, torch.tensor([0.999]), torch.tensor([1.0 - 2.0 ** -24]), np.array([0, 1]))
    assert r.accepted.item() == 0 and r.tokens[0, 0].item() == v - 1
    assert abs(r.accept_prob.item() - 1 / v) <= 4 * 2.0 ** -24 / v


def _whole(z, t):
    e = torch.exp2((z - z.amax(1, keepdim=True)) * np.float32(1.4426950408889634 / float(np.float32(t))).item())
    return e, torch.round(e.double() * 2.0 ** 43).to(torch.int64)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("v", [999, 50001, 128256])
def test_whole_numbers(fl, v, dtype):
    """Bit by bit what the definition gives: draws at the borders of the running sum, and between them."""
    zt, zd, _, _, _, _ = _make([1], v, dtype, seed=v)
    zt, zd = zt.cuda(), zd.cuda()
    (e, w), (eq, wq) = _whole(zt.float(), 0.9), _whole(zd.float(), 0.9)
    inv = lambda w: (1.0 / (w.sum(1).double() / 2.0 ** 43)).float()[:, None]  # noqa: E731
    p, q = e * inv(w), eq * inv(wq)
    for r, accept in (((p[:1] - q).clamp_min(0), 2.0), (p[1:], -1.0)):
        run = torch.round(r.double() * 2.0 ** 43).to(torch.int64).cumsum(1)[0]
        total = run[-1].item()
        u = torch.cat([torch.rand(300, generator=torch.Generator().manual_seed(v)).cuda(),
                       (run[:: max(1, v // 300)].double() / total).float().clamp(max=1 - 2.0 ** -24)])
        b = u.numel()
        want = torch.searchsorted(run, (u.double() * total).floor().to(torch.int64).clamp(max=total - 1), right=True)
        # one row for all: the batch's rows repeat it
        z2 = zt.repeat(b, 1) if accept < 0 else torch.stack([zt[0], zt[1]]).repeat(b, 1)
        d = torch.full((b,), int(p[0].argmax()) if accept < 0 else int((q - p[:1]).argmax()), device="cuda")
        got = fl.verify_drafts(z2, d, torch.full((b,), accept, device="cuda"), u, draft_logits=zd.repeat(b, 1), temperature=0.9)
        assert torch.equal(got.tokens[torch.arange(b), got.accepted], want)
        assert (got.accepted == (1 if accept < 0 else 0)).all()


@gpu
def test_same_alone_and_in_a_batch(fl):
    counts = [3, 0, 5, 2, 1, 4, 0, 2]
    x = _make(counts, 20011, BF, seed=4)
    r = _run(fl, *x, t=0.8)
    zt, zd, tok, u, ud, ends = x
    for b, k in enumerate(counts):
        s, e = ends[b], ends[b + 1]
        one = _run(fl, zt[s + b:e + b + 1], zd[s:e], tok[s:e], u[s:e], ud[b:b + 1], np.array([0, k]), t=0.8)
        assert torch.equal(one.tokens[0], r.tokens[b, :k + 1]) and one.accepted[0] == r.accepted[b]
        assert torch.equal(one.accept_prob, r.accept_prob[s:e])


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["fp32", "bf16"])
def test_rows_apart_and_unaligned(fl, dtype):
    x = _make([2, 3], 3001, dtype, seed=5)
    want = _run(fl, *x)
    for pad, off in ((1, 1), (7, 3), (8, 0), (40, 5)):
        wide = [torch.full((z.shape[0], 3001 + pad), 99.0).to(dtype) for z in x[:2]]  # (read, they would be the largest)
        for w, z in zip(wide, x[:2]):
            w[:, min(off, pad):min(off, pad) + 3001] = z
        views = [w.cuda()[:, min(off, pad):min(off, pad) + 3001] for w in wide]
        tok, u, ud = _cuda(*x[2:5])
        got = fl.verify_drafts(views[0], tok, u, ud, draft_logits=views[1], offsets=torch.tensor(x[5]).cuda(), max_drafts=3)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_temperatures_of_their_own(fl):
    counts, t = [2, 3, 1, 0, 4], torch.tensor([0.0, 0.7, 1.3, 0.0, 2.0])
    x = _make(counts, 4001, torch.float32, seed=6)
    r = _run(fl, *x, t=t)
    _check(r, *x[:2], x[2].numpy(), x[3].numpy(), x[4].numpy(), x[5], t.numpy(), 4)
    for i, ti in enumerate(t.tolist()):
        one = _run(fl, *x, t=ti)
        assert torch.equal(one.tokens[i], r.tokens[i])


@gpu
def test_numbers_at_the_ends(fl):
    zt = torch.tensor([[0.0, 0.0, -INF], [1.0, -INF, 1.0]])
    tok = torch.tensor([0])
    for u, ud, acc, token in ((0.0, 0.0, 1, 0), (0.49, 0.999, 1, 2), (0.5, 0.0, 0, 1), (NAN, 0.7, 0, 1), (INF, 0.0, 0, 1),
                              (-1.0, NAN, 1, 0), (0.0, 1.0, 1, 2), (0.0, 7.0, 1, 2), (0.0, -2.0, 1, 0), (0.0, INF, 1, 2)):
        r = _run(fl, zt, None, tok, torch.tensor([u]), torch.tensor([ud]), np.array([0, 1]))
        assert (r.accepted.item(), r.tokens[0, r.accepted.item()].item()) == (acc, token), (u, ud)
        assert r.accept_prob.item() == 0.5
    # p = q: the drafted token is never refused by a number below 1, and one that is not gives p's
    r = _run(fl, zt, zt[:1], tok, torch.tensor([1.0]), torch.tensor([0.6]), np.array([0, 1]))
    assert r.accepted.item() == 0 and r.tokens[0].tolist() == [1, -1] and r.accept_prob.item() == 1


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("v", [5, 9001])
def test_masks_and_bad_rows(fl, v, dtype):
    g = torch.Generator().manual_seed(v)
    low = torch.finfo(dtype).min
    z = torch.randn(2, v, generator=g).to(dtype)
    masked, lowest, one, empty = z.clone(), z.clone(), z.clone(), torch.full_like(z, -INF)
    masked[:, ::2] = -INF
    lowest[:, 1:] = low
    one[:, :] = -INF
    one[:, v - 1] = 3.0
    nan, inf, big = z.clone(), z.clone(), z.clone()
    nan[:, v - 2], inf[:, v - 2] = NAN, INF
    big[:, 0], big[:, 1] = torch.finfo(dtype).max, low
    rows = {"z": z, "masked": masked, "lowest": lowest, "one": one, "empty": empty, "nan": nan, "inf": inf, "big": big,
            "all_low": torch.full_like(z, low)}
    for (nt, zt), (nd, zd) in itertools.product(rows.items(), [("lookup", None), *rows.items()]):
        for d in (0, 1, v - 1):
            for u, ud in ((0.3, 0.2), (0.9999, 0.95)):
                args = (zt, None if zd is None else zd[:1], torch.tensor([d]), torch.tensor([u]), torch.tensor([ud]), np.array([0, 1]))
                for t in (1.0, 0.0):
                    r = _run(fl, *args, t=t)
                    _check(r, *args[:2], args[2].numpy(), args[3].numpy(), args[4].numpy(), args[5], [t], 1)


@gpu
def test_tokens_out_of_range(fl):
    x = _make([3, 2], 500, torch.float32, seed=8)
    status = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    _run(fl, *x, status=status)
    assert status.item() == 0
    for bad in (-1, 500, 1 << 40, -(1 << 62)):
        for draft in (x[1], None):
            tok = x[2].clone()
            tok[1] = bad
            u = torch.zeros(5)  # (0 accepts what may be)
            r = _run(fl, x[0], draft, tok, u, *x[4:], status=status)
            assert status.item() == 1 and r.accepted.tolist() == [1, 2] and r.accept_prob[1].item() == 0
            _check(r, x[0], draft, tok.numpy(), u.numpy(), x[4].numpy(), x[5], [1.0] * 2, 3)


@gpu
def test_offsets_and_temperatures_out_of_range(fl):
    x = _make([2, 2, 2], 300, BF, seed=9)
    want = _run(fl, *x)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for ends, ok in (([0, 2, 1, 3], [0]), ([0, 2, 4, 7], [0, 1]), ([-2, 2, 4, 6], [1, 2]), ([0, 2, 4, 1 << 40], [0, 1]),
                     ([0, 2, 4, -(1 << 40)], [0, 1])):
        r = _run(fl, *x[:5], np.array(ends), max_drafts=2, status=status)
        assert status.item() == 1
        for b in range(3):
            if b in ok:
                assert torch.equal(r.tokens[b], want.tokens[b]) and r.accepted[b] == want.accepted[b]
            elif not 0 <= ends[b] <= ends[b + 1] <= 6:
                assert r.accepted[b] == 0 and (r.tokens[b] == -1).all()
    r = _run(fl, *x, max_drafts=2, status=status)
    assert status.item() == 0
    r = _run(fl, *x, max_drafts=1, status=status)  # more drafts than there is room for
    assert status.item() == 1 and (r.tokens == -1).all() and not r.accepted.any()
    r = _run(fl, *x, t=torch.tensor([NAN, 1.0, -1.0]), status=status)
    assert status.item() == 1 and (r.tokens[[0, 2]] == -1).all() and torch.equal(r.tokens[1], want.tokens[1])
    r = _run(fl, *x, t=torch.tensor([1.0, 1e-40, INF]), status=status)
    assert status.item() == 1 and torch.equal(r.tokens[0], want.tokens[0]) and (r.tokens[1:] == -1).all()


@gpu
def test_a_longer_buffer(fl):
    """Rows before the first request's and behind the last one's are not read."""
    x = _make([2, 0, 3], 700, BF, seed=10)
    want = _run(fl, *x)
    zt, zd, tok, u, ud, ends = x
    bad = lambda n: torch.full((n, 700), NAN).to(BF)  # noqa: E731
    ones = lambda n: torch.full((n,), 1 << 50)  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = _run(fl, torch.cat([bad(2), zt, bad(4)]), torch.cat([bad(2), zd, bad(4)]), torch.cat([ones(2), tok, ones(4)]),
             torch.cat([torch.zeros(2), u, torch.zeros(4)]), ud, ends + 2, max_drafts=6, status=status)
    assert status.item() == 0 and torch.equal(r.accepted, want.accepted)
    assert torch.equal(r.tokens[:, :4], want.tokens) and (r.tokens[:, 4:] == -1).all()
    assert torch.equal(r.accept_prob[2:-4], want.accept_prob) and not r.accept_prob[:2].any() and not r.accept_prob[-4:].any()


@gpu
def test_many_drafts(fl):
    x = _make([100, 33, 32, 31, 64], 64, torch.float32, seed=11, near=0.02)
    for u in (x[3], x[3] * 0, x[3] * 0.5):
        r = _run(fl, *x[:3], u, *x[4:])
        _check(r, *x[:2], x[2].numpy(), u.numpy(), x[4].numpy(), x[5], [1.0] * 5, 100)
    assert r.accepted.max() > 32


@gpu
@pytest.mark.parametrize("draft", [True, False], ids=["draft", "lookup"])
def test_tokens_follow_the_target(fl, draft):
    g = torch.Generator("cuda").manual_seed(12)
    b, v = 400_000, 6
    zt, zd = torch.tensor([[1.0, 0.0, -1.0, 2.0, 0.5, -INF]]).cuda(), torch.tensor([[0.0, 1.0, 2.0, -1.0, 0.5, 1.0]]).cuda()
    p, q = torch.softmax(zt[0].double(), 0), torch.softmax(zd[0].double(), 0)
    tok = torch.multinomial(q.float(), b, replacement=True, generator=g) if draft else torch.randint(0, v, (b,), device="cuda", generator=g)
    r = fl.verify_drafts(zt.repeat(2 * b, 1), tok, torch.rand(b, device="cuda", generator=g), torch.rand(b, device="cuda", generator=g),
                         draft_logits=zd.repeat(b, 1) if draft else None)
    share = torch.bincount(r.tokens[:, 0], minlength=v).double() / b
    # six standard deviations of a share
    assert ((share - p).abs() <= 6 * (p * (1 - p) / b).sqrt() + 1e-12).all()
    a = torch.minimum(p, q).sum().item() if draft else (p / v).sum().item()
    assert abs(r.accepted.double().mean().item() - a) <= 6 * math.sqrt(a * (1 - a) / b)


@gpu
def test_captured(fl):
    x = _make([2, 3], 2003, BF, seed=13)
    zt, zd, tok, u, ud = _cuda(*x[:5])
    off = torch.tensor(x[5]).cuda()
    call = lambda: fl.verify_drafts(zt, tok, u, ud, draft_logits=zd, offsets=off, max_drafts=3)  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for seed in (14, 15):
        y = _make([3, 2], 2003, BF, seed=seed)
        for a, c in zip((zt, zd, tok, u, ud, off), (*y[:5], torch.tensor(y[5]))):
            a.copy_(c)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(got, call()))


@gpu
def test_on_a_given_stream(fl):
    x = _make([2, 3], 2003, BF, seed=13)
    want = _run(fl, *x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (side, side.cuda_stream):
        got = _run(fl, *x, stream=s)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_refusals_on_the_gpu(fl):
    x = _make([2, 2], 100, BF, seed=1)
    zt, zd, tok, u, ud = _cuda(*x[:5])
    off = torch.tensor(x[5]).cuda()
    good = dict(target_logits=zt, draft_tokens=tok, u_accept=u, u_draw=ud, draft_logits=zd)
    fl.verify_drafts(**good)
    for bad in (dict(target_logits=zt[:5]), dict(target_logits=zt[:, ::2]), dict(target_logits=zt.half()), dict(draft_logits=zd.float()),
                dict(draft_logits=zd[:3]), dict(draft_logits=zd.cpu()), dict(draft_tokens=tok.int()), dict(draft_tokens=tok[:3]),
                dict(u_accept=u.double()), dict(u_accept=u[:3]), dict(u_draw=ud[:0]), dict(u_draw=ud.cpu()), dict(offsets=off),
                dict(offsets=off.int(), max_drafts=2), dict(offsets=off[:2], max_drafts=2), dict(offsets=off, max_drafts=-1),
                dict(max_drafts=3), dict(temperature=torch.ones(3, device="cuda")), dict(temperature=torch.ones(2)),
                dict(status=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            fl.verify_drafts(**{**good, **bad})
    for t in (-1.0, NAN, 1e-40):
        with pytest.raises(fl.FljsdError):
            fl.verify_drafts(**good, temperature=t)
