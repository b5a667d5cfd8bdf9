"""The norm of many gradients together, clipping, and AdamW's clipped step: refusals (CPU),
and the GPU against 64 bits, over types, sizes, alignments and fp32's whole range."""
import ctypes
import math

import numpy as np
import pytest
import torch

gpu = pytest.mark.gpu
U = 2.0 ** -24  # an fp32 rounding
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def fl():
    from conftest import build_library

    build_library()
    import lm_head_jsd_gb300 as fl

    return fl


# ---- refusals (no GPU) ----
def _entries(fl, *rows):
    t = (fl._lib.fljsd_grad_tensor * max(1, len(rows)))()
    for e, r in zip(t, rows):
        for k, v in {**dict(grad=4096, out=8192, n=0, dtype=0), **r}.items():
            setattr(e, k, v)
    return t


def _c(fl, entry="fljsd_grad_norm", rows=({},), kind=2, max_norm=1.0, scale=None, norm=64, factor=None, ws=256,
       bytes_=1 << 20, count=None):
    t = _entries(fl, *rows)
    args = (ctypes.addressof(t), len(rows) if count is None else count, kind, max_norm)
    if entry == "fljsd_grad_norm":
        return fl.fljsd_grad_norm(*args, scale, norm, factor, ws, bytes_, stream=0, check=False)
    return fl.fljsd_clip_grads(*args, norm, ws, bytes_, stream=0, check=False)


BAD = [dict(kind=1), dict(norm=None), dict(norm=66), dict(ws=None), dict(ws=8), dict(count=-1),
       dict(rows=({"n": -1},)), dict(rows=({"dtype": 2},)), dict(rows=({"n": 4, "grad": None},)),
       dict(rows=({"n": 4, "grad": 4098},)), dict(rows=({"n": 4, "grad": 4097, "dtype": 1},))]


@pytest.mark.parametrize("entry", ["fljsd_grad_norm", "fljsd_clip_grads"])
@pytest.mark.parametrize("bad", BAD, ids=str)
def test_refused(fl, entry, bad):
    assert _c(fl, entry, **bad) == 1


@pytest.mark.parametrize("entry", ["fljsd_grad_norm", "fljsd_clip_grads"])
def test_refused_sizes(fl, entry):
    assert _c(fl, entry, rows=({"n": (1 << 40) + 1},)) == 2
    assert _c(fl, entry, bytes_=fl.fljsd_grad_norm_workspace_bytes(1) - 1) == 3
    assert fl.fljsd_grad_norm_workspace_bytes(5000) > fl.fljsd_grad_norm_workspace_bytes(1)


def test_refused_where_looked_at(fl):
    for m in (-1.0, math.nan):
        assert _c(fl, factor=64, max_norm=m) == 1
        assert _c(fl, "fljsd_clip_grads", max_norm=m) == 1
    assert _c(fl, scale=2) == 1 and _c(fl, factor=2) == 1
    assert _c(fl, "fljsd_clip_grads", rows=({"n": 4, "out": None},)) == 1
    assert _c(fl, "fljsd_clip_grads", rows=({"n": 4, "out": 8194},)) == 1


def test_refused_in_python(fl):
    g = torch.zeros(4)
    for call in (fl.grad_norm, lambda x, **kw: fl.clip_grads(x, 1.0, **kw)):
        with pytest.raises(ValueError, match="no gradients"):
            call([])
        with pytest.raises(ValueError, match="no gradients"):
            call([None])
        with pytest.raises(ValueError, match="norm_type"):
            call([g], norm_type=1)
        with pytest.raises(ValueError, match="expected a CUDA device"):
            call([g])
    for m in (-1.0, math.nan):
        with pytest.raises(ValueError, match="max_norm"):
            fl.clip_grads([g], m)
        with pytest.raises(ValueError, match="max_norm"):
            fl.AdamW([torch.zeros(4)]).step([g], max_norm=m)


def _pointers(*rows):
    from lm_head_jsd_gb300 import clip

    t = np.zeros(len(rows), dtype=clip._ENTRY)
    for i, (g, o, n) in enumerate(rows):
        t[i] = (g, o, n, 0, 0)
    return clip, t


def test_overlaps_are_found():
    clip, t = _pointers((0, 0, 4), (16, 16, 4))
    clip._apart(t, False)
    for rows, given in (([(0, 0, 4), (0, 0, 4)], False), ([(0, 0, 5), (16, 16, 4)], False),
                        ([(0, 64, 4), (32, 76, 4)], True), ([(0, 16, 4), (16, 64, 4)], True),
                        ([(0, 4, 4)], True), ([(0, 0, 100), (64, 64, 1), (80, 80, 4)], False),
                        ([(0, 64, 4), (32, 0, 4)], True)):
        clip, t = _pointers(*rows)
        with pytest.raises(ValueError, match="overlap"):
            clip._apart(t, given)
    clip, t = _pointers((0, 64, 4), (0, 128, 4), (32, 32, 4), (0, 0, 0))  # one gradient to two places
    clip._apart(t, True)


# ---- on the GPU ----
def _grads(sizes, dtypes, seed=0, std=1.0, offset=0):
    """Each in an allocation of its own, `offset` elements behind its start."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        x = (torch.randn(n + offset, generator=g) * std).to(dtypes[i % len(dtypes)])
        out.append(x.cuda()[offset:])
    return out


def _want(grads, kind=2.0):
    x = torch.cat([g.double().cpu() for g in grads])
    return (x.abs().max().item() if kind == math.inf else x.square().sum().sqrt().item())


SIZES = {"one": [1], "odd": [3, 127, 4097, 1], "empty": [0, 5, 0], "many": [7] * 70 + [1000] * 3,
         "tables": [5] * 1700, "chunks": [4096, 8192, 40000, 8193, 1]}


@gpu
@pytest.mark.parametrize("kind", [2.0, math.inf])
@pytest.mark.parametrize("dtypes", [[torch.float32], [BF], [torch.float32, BF]], ids=["fp32", "bf16", "mixed"])
@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("sizes", SIZES)
def test_norm(fl, sizes, offset, dtypes, kind):
    grads = _grads(SIZES[sizes], dtypes, offset=offset)
    got, want = fl.grad_norm(grads, norm_type=kind), _want(grads, kind)
    assert got.shape == () and got.dtype == torch.float32
    # a thread adds at most 8 squares to each of 4 sums, joins them, and adds few such: 16 roundings
    # of the sum are 8 of its root, whose own is one more; a largest magnitude is not rounded
    assert abs(got.item() - want) <= (0 if kind == math.inf else 9 * U * want)
    assert torch.equal(got, fl.grad_norm(grads, norm_type=kind))


@gpu
def test_norm_of_a_tensor_longer_than_a_round_of_the_gpu(fl):
    n = 30_000_001
    g = torch.randn(n, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    # 4 chunks of 16 KB reach a CTA at most: 16 roundings of 64 bytes' sum, and 8 of the thread's
    for x in (g, g.bfloat16()):
        want = x.double().square().sum().sqrt().item()
        assert abs(fl.grad_norm(x).item() - want) <= 13 * U * want
        assert fl.grad_norm(x, norm_type=math.inf).item() == x.abs().max().item()


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("std", [1e-44, 1e-38, 1e-30, 1e-19, 1e-15, 1e15, 1e19, 1e30])
def test_norm_over_the_range(fl, std, dtype):
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(9001, generator=g, dtype=torch.float64) * std).to(dtype).cuda()
    x[100:5000] = 0
    want = x.double().square().sum().sqrt().item()
    # (results below fp32's normal numbers are rounded to its least step)
    assert abs(fl.grad_norm([x]).item() - want) <= max(9 * U * want, 2.0 ** -150)


@gpu
def test_norm_of_far_apart_magnitudes(fl):
    for big, small in ((1e25, 1.0), (1.0, 1e-30)):
        xs = [torch.full((5000,), small, device="cuda"), torch.full((5000,), big, device="cuda")]
        want = math.sqrt(5000.0) * float(xs[1][0].item())
        assert abs(fl.grad_norm(xs).item() - want) <= 9 * U * want
    huge = torch.full((16,), 3e38, device="cuda")  # the norm itself is not a number of fp32
    assert fl.grad_norm(huge).item() == math.inf and fl.grad_norm(huge, norm_type=math.inf).item() == huge[0].item()


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["fp32", "bf16"])
def test_zeros_nan_and_infinity(fl, dtype):
    z = torch.zeros(5000, device="cuda", dtype=dtype)
    z[7] = -0.0
    assert fl.grad_norm(z).item() == 0 and fl.grad_norm(z, norm_type=math.inf).item() == 0
    x = _grads([5000], [dtype])[0]
    for i in (0, 4099, 4999):
        for v, same in ((math.nan, math.isnan), (math.inf, lambda r: r == math.inf), (-math.inf, lambda r: r == math.inf)):
            y = x.clone()
            y[i] = v
            for kind in (2.0, math.inf):
                assert same(fl.grad_norm([x, y], norm_type=kind).item())
    y = x.clone()
    y[3], y[4] = math.inf, math.nan
    assert math.isnan(fl.grad_norm(y).item()) and math.isnan(fl.grad_norm(y, norm_type=math.inf).item())


def _factor(norm, max_norm):
    return min(np.float32(1), np.float32(max_norm) / (np.float32(norm) + np.float32(1e-6)))


@gpu
@pytest.mark.parametrize("kind", [2.0, math.inf])
@pytest.mark.parametrize("dtypes", [[torch.float32], [BF], [torch.float32, BF]], ids=["fp32", "bf16", "mixed"])
@pytest.mark.parametrize("sizes,offset", [("odd", 0), ("many", 1), ("tables", 0), ("chunks", 3), ("empty", 0)])
def test_clip(fl, sizes, offset, dtypes, kind):
    grads = _grads(SIZES[sizes], dtypes, offset=offset)
    kept = [g.clone() for g in grads]
    norm = fl.grad_norm(grads, norm_type=kind)
    out = _grads(SIZES[sizes], dtypes, seed=9, offset=(offset + 1) % 4)  # another alignment
    assert torch.equal(fl.clip_grads(grads, 0.5, norm_type=kind, out=out), norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, kept))
    f = float(_factor(norm.item(), 0.5))
    want = [(g.float() * f).to(g.dtype) for g in grads]  # one product and its rounding, as torch's
    assert f < 1 and all(torch.equal(a, b) for a, b in zip(out, want))
    assert torch.equal(fl.clip_grads(grads, 0.5, norm_type=kind), norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
    # what is short enough stays, or is copied as it is
    kept = [g.clone() for g in grads]
    fl.clip_grads(grads, 1.0, norm_type=kind)
    fl.clip_grads(grads, 1.0, norm_type=kind, out=out)
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(grads, kept, out))


@gpu
def test_clip_to_zero_infinite_and_not_a_number(fl):
    x = _grads([5000], [torch.float32])[0]
    a = x.clone()
    fl.clip_grads(a, math.inf)
    assert torch.equal(a, x)
    fl.clip_grads(a, 0.0)
    assert not a.any()
    a = x.clone()
    a[5] = math.inf  # factor 0
    assert fl.clip_grads(a, 1.0).item() == math.inf
    assert torch.isnan(a[5]) and a.nan_to_num(0.0).abs().sum() == 0
    a = x.clone()
    a[5] = math.nan
    assert math.isnan(fl.clip_grads(a, 1.0).item()) and torch.isnan(a).all()


@gpu
def test_clip_leaves_neighbours(fl):
    for dtype in (torch.float32, BF):
        flat = torch.ones(9000, device="cuda", dtype=dtype)
        fl.clip_grads([flat[3:4000], flat[4001:8999]], 1.0)
        assert flat[[0, 1, 2, 4000, 8999]].eq(1).all() and flat[3:4000].lt(1).all() and flat[4001:8999].lt(1).all()


@gpu
def test_clip_refusals(fl):
    x = torch.ones(100, device="cuda")
    for grads, out in (([x, x], None), ([x[:60], x[50:]], None), ([x[:50]], [x[20:70]]), ([x[:50], x[50:]], [x[50:], x[:50]])):
        with pytest.raises(ValueError, match="overlap"):
            fl.clip_grads(grads, 1.0, out=out)
    for bad in (x[::2], x.double(), x.half()):
        with pytest.raises(ValueError):
            fl.grad_norm([bad])
        with pytest.raises(ValueError):
            fl.clip_grads([x], 1.0, out=[bad])
    for out in ([], [None], [x[:50].clone()], [x.bfloat16()]):
        with pytest.raises(ValueError):
            fl.clip_grads([x], 1.0, out=out)
    assert x.eq(1).all()


@gpu
def test_versions_rise(fl):
    w = torch.ones(10, device="cuda", requires_grad=True)
    g = torch.ones(10, device="cuda")
    y = (w * g).sum()
    fl.clip_grads([g], 1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


@gpu
def test_clip_captured(fl):
    grads = _grads(SIZES["many"], [torch.float32, BF])
    src = [g.clone() for g in grads]
    norm = fl.clip_grads(grads, 0.5)
    want = [g.clone() for g in grads]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fl.clip_grads(grads, 0.5)
    for k in (1.0, 2.0):  # the second replay has other gradients
        for g, s in zip(grads, src):
            g.copy_(s * k)
        graph.replay()
        torch.cuda.synchronize()
        assert abs(got.item() - k * norm.item()) <= 4 * U * got.item()
        if k == 1:
            assert all(torch.equal(a, b) for a, b in zip(grads, want))


@gpu
def test_clip_on_a_given_stream(fl):
    grads = _grads(SIZES["chunks"], [torch.float32, BF])
    side = torch.cuda.Stream()
    want = fl.grad_norm(grads)
    torch.cuda.synchronize()
    for s in (side, side.cuda_stream):
        got = fl.grad_norm(grads, stream=s)
        side.synchronize()
        assert torch.equal(got, want)
    got = fl.clip_grads(grads, 0.5, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and abs(fl.grad_norm(grads).item() - 0.5) <= 2.0 ** -9


# ---- the clipped step ----
def _steppers(fl, bits, master, sizes=(1000, 7, 4097), n=2):
    ps = [torch.randn(s, generator=torch.Generator().manual_seed(s)).to(BF if master else torch.float32) for s in sizes]
    return [fl.AdamW([p.clone().cuda() for p in ps], lr=1e-2, state_bits=bits, master=master) for _ in range(n)]


def _state(opt):
    return [*opt.params, *(opt.master or ()), *(t.view(torch.uint8) for t in opt.exp_avg), *(t.view(torch.uint8) for t in opt.exp_avg_sq)]


@gpu
@pytest.mark.parametrize("bits,master", [(32, False), (8, True)])
@pytest.mark.parametrize("scale", [None, 0.25])
def test_clipped_step(fl, bits, master, scale):
    """Bit by bit the step by the factor that the norm gives, for gradients that are longer and shorter."""
    a, b = _steppers(fl, bits, master or None)
    sc = None if scale is None else torch.tensor(scale, device="cuda")
    for step, std in enumerate((1.0, 1e-4, 1.0)):
        g = _grads([p.numel() for p in a.params], [a.dtype], seed=step, std=std)
        kept = [x.clone() for x in g]
        a.step(g, grad_scale=sc, max_norm=0.5)
        assert all(torch.equal(x, y) for x, y in zip(g, kept))
        norm = np.float32(fl.grad_norm(g).item() * (scale or 1.0))  # (a power of two)
        assert a.grad_norm.item() == norm
        f = np.float32(_factor(norm, 0.5) * np.float32(scale or 1.0))
        assert (f == (scale or 1.0)) == (step == 1)
        b.step(g, grad_scale=torch.tensor(float(f), device="cuda"))
        assert all(torch.equal(x, y) for x, y in zip(_state(a), _state(b)))


@gpu
def test_clipped_step_of_some(fl):
    a, b = _steppers(fl, 32, None)
    g = _grads([p.numel() for p in a.params], [torch.float32])
    g[1] = None
    a.step(g, max_norm=0.5)
    norm = fl.grad_norm(g)
    assert torch.equal(a.grad_norm, norm)
    b.step(g, grad_scale=torch.tensor(float(_factor(norm.item(), 0.5)), device="cuda"))
    assert all(torch.equal(x, y) for x, y in zip(_state(a), _state(b))) and a.param_steps == [1, 0, 1]
