"""AdamW over many tensors: the float64 oracle's pins and the refusals (CPU), and the
GPU step against the oracle and, bit by bit, against the same fp32 operations in
NumPy, over types, odd sizes, unaligned tensors, and tables of more than one launch."""
import math

import numpy as np
import pytest
import torch

from oracle import adamw_ref, e4m3_values, quantise_ref
from parity_util import f64

gpu = pytest.mark.gpu
HY = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
F8 = torch.float8_e4m3fn


# ---- the oracle ----
def test_oracle_against_torch():
    g = torch.Generator().manual_seed(0)
    p = torch.nn.Parameter(torch.randn(50, dtype=torch.float64, generator=g))
    opt = torch.optim.AdamW([p], **HY)
    q, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        p.grad = torch.randn(50, dtype=torch.float64, generator=g)
        opt.step()
        q, m, v = adamw_ref(q, p.grad.numpy(), m, v, t, **HY)
        assert np.allclose(q, p.detach().numpy(), rtol=1e-12)


def test_oracle_e4m3_against_torch():
    codes = torch.arange(127, dtype=torch.uint8).view(F8).double().numpy()
    assert np.array_equal(e4m3_values(), codes)
    x = torch.randn(1000, generator=torch.Generator().manual_seed(1)) * 1e-3
    x[300:428] = 0
    val, sc = quantise_ref(x.numpy())
    for i in range(8):
        b = x[i * 128:(i + 1) * 128]
        amax = b.abs().max().clamp_min(2.0 ** -100)
        assert sc[i] == (amax * torch.tensor(1 / 448)).item()
        assert np.array_equal(val[i * 128:(i + 1) * 128], (b * (448 * (1 / amax))).to(F8).double().numpy())


# ---- refusals (no GPU) ----
@pytest.fixture(scope="module")
def L():
    from conftest import build_library

    build_library()
    from lm_head_jsd_gb300 import _lib

    return _lib


def _call(L, entry=None, count=1, scale=None, **kw):
    import ctypes

    o = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, step=1)
    opt = L.make_adamw_options(**{**o, **kw})
    e = dict(grad=4096, param=8192, exp_avg=12288, exp_avg_sq=16384, n=0)
    e.update(entry or {})
    t = L.fljsd_adamw_tensor(**e)
    return L.fljsd_adamw_step(opt, ctypes.addressof(t), count, scale, stream=0, check=False)


@pytest.mark.parametrize("kw", [dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=float("nan")),
                                dict(eps=-1.0), dict(lr=float("inf")), dict(weight_decay=float("nan")),
                                dict(step=0), dict(state_bits=16), dict(param_dtype=9),
                                dict(grad_dtype=-1), dict(master=1, param_dtype="fp32"),
                                dict(master=2), dict(count=-1), dict(scale=4097)])
def test_option_refusals(L, kw):
    assert _call(L, **kw) == 1


def test_tensor_refusals(L):
    assert _call(L, dict(n=-1)) == 1
    for name in ("grad", "param", "exp_avg", "exp_avg_sq"):
        assert _call(L, {name: None, "n": 8}) == 1
        assert _call(L, {name: 4097, "n": 8}) == 1
    assert _call(L, dict(n=8), state_bits=8) == 1  # no scales
    assert _call(L, dict(n=8), master=1) == 1  # no master weights
    assert _call(L, dict(n=8, master=4096)) == 1  # master weights that would not be stepped
    assert _call(L, dict(n=(1 << 40) + 1)) == 2
    assert _call(L, dict(n=0, grad=None, param=None)) == 0  # nothing to do, nothing launched


def test_wrapper_refusals():
    from lm_head_jsd_gb300 import AdamW

    p = [torch.zeros(4), torch.zeros(3, 2)]
    for kw in (dict(state_bits=4), dict(master=True), dict(exp_avg=p),
               dict(exp_avg=p, exp_avg_sq=[p[0], p[0]]), dict(exp_avg=p[:1], exp_avg_sq=p),
               dict(exp_avg=p, exp_avg_sq=p, state_bits=8)):
        with pytest.raises(ValueError):
            AdamW(p, **kw)
    with pytest.raises(ValueError):
        AdamW([])
    with pytest.raises(ValueError):
        AdamW([torch.zeros(4), torch.zeros(4).bfloat16()])
    with pytest.raises(ValueError):
        AdamW([torch.zeros(4, 4).T[1:]])
    opt = AdamW(p)
    for g in ([p[0]], [p[0], p[0]], [p[0].bfloat16(), p[1]], [p[0], torch.zeros(2, 3).T]):
        with pytest.raises(ValueError):
            opt.step(g)
    opt.step([None, None])  # nothing to do
    assert opt.steps == 0


# ---- GPU ----
def _f32_step(p, g, m, r2, t, scale=np.float32(1)):
    """The step in fp32, one rounding to an operation."""
    f = np.float32
    b1, b2 = HY["betas"]
    g = g * scale
    m = m * f(b1) + g * f(1 - b1)
    v = r2 * f(b2) + g * f(1 - b2) * g
    den = np.sqrt(v) * f(1 / math.sqrt(1 - b2 ** t)) + f(HY["eps"])
    return p * f(1 - HY["lr"] * HY["weight_decay"]) - (m / den) * f(HY["lr"] / (1 - b1 ** t)), m, v


SIZES = [1, 7, 8, 127, 128, 129, 2047, 2048, 2049, 5000, 0, 333]


def _tensors(sizes, dtype, std, seed, pos=False):
    g = torch.Generator().manual_seed(seed)
    ts = [torch.randn(n, generator=g) * std for n in sizes]
    return [(t.abs() if pos else t).to(dtype) for t in ts]


def _np(t):
    return t.detach().float().cpu().numpy()


@gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pd,gd,master", [(torch.float32, torch.float32, False),
                                          (torch.float32, torch.bfloat16, False),
                                          (torch.bfloat16, torch.bfloat16, False),
                                          (torch.bfloat16, torch.float32, False),
                                          (torch.bfloat16, torch.bfloat16, True),
                                          (torch.bfloat16, torch.float32, True)])
@pytest.mark.parametrize("scale", [None, 0.37])
def test_steps(bits, pd, gd, master, scale):
    from lm_head_jsd_gb300 import AdamW

    params = [t.cuda() for t in _tensors(SIZES, pd, 0.02, 1)]
    opt = AdamW(params, state_bits=bits, master=True if master else None, **HY)
    sc = None if scale is None else torch.tensor([scale], device="cuda")
    base = [_np(t) for t in (opt.master or params)]
    m, v = [np.zeros_like(t) for t in base], [np.zeros_like(t) for t in base]
    for t in range(1, 4):
        grads = [x.cuda() for x in _tensors(SIZES, gd, 10.0 ** -t, 10 + t)]
        grads[3] = grads[3] * 0 if t == 1 else grads[3]  # an 8-bit block of zeros
        before = [(_np(a), *s) for a, *s in zip(opt.master or params, m, v)]
        opt.step(grads, grad_scale=sc)
        for i, g in enumerate(grads):
            p1, m1, v1 = _f32_step(*before[i][:1], _np(g), *before[i][1:], t, np.float32(scale or 1))
            ref = adamw_ref(before[i][0], _np(g).astype(np.float64) * np.float32(scale or 1),
                            before[i][1], before[i][2], t, **HY)
            got = _np((opt.master or params)[i])
            if master or pd == torch.float32:
                assert np.array_equal(got, p1), i
                # p: two roundings of p, six of the update
                upd = np.abs(ref[0] - before[i][0]) + HY["lr"]
                assert (np.abs(got - ref[0]) <= 2 ** -23 * np.abs(ref[0]) + 2 ** -21 * upd).all()
            if pd == torch.bfloat16:
                assert np.array_equal(_np(params[i]), torch.from_numpy(p1).bfloat16().float().numpy())
            if bits == 32:
                assert np.array_equal(_np(opt.exp_avg[i]), m1) and np.array_equal(_np(opt.exp_avg_sq[i]), v1)
                assert np.allclose(m1, ref[1], rtol=0, atol=2 ** -22 * (np.abs(ref[1]).max(initial=0) + 1e-30))
                assert np.allclose(v1, ref[2], rtol=2 ** -21)
                m[i], v[i] = m1, v1
            elif g.numel():
                (qm, sm), (qr, sr) = quantise_ref(m1), quantise_ref(np.sqrt(v1))
                assert np.array_equal(f64(opt.exp_avg[i]), qm) and np.array_equal(_np(opt.exp_avg_scale[i]), sm)
                assert np.array_equal(f64(opt.exp_avg_sq[i]), qr)
                assert np.array_equal(_np(opt.exp_avg_sq_scale[i]), sr)
                n = qm.size
                m[i] = qm * np.repeat(sm, 128)[:n]
                r = qr * np.repeat(sr, 128)[:n]
                v[i] = r * r
                # each state within half a step of what it stands for (2^-4, or half of
                # the least e4m3 step 2^-9 in units of the scale)
                for q, s, x in ((m[i], sm, m1), (r, sr, np.sqrt(v1))):
                    lim = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * np.repeat(s, 128)[:n])
                    assert (np.abs(q - x) <= lim * 1.0001).all()


@gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_unaligned_and_guarded(bits, dtype):
    """Tensors at odd offsets give what aligned ones give, and their neighbours stay."""
    from lm_head_jsd_gb300 import AdamW

    n = 3001
    p, g = _tensors([n], dtype, 0.02, 3)[0], _tensors([n], dtype, 0.01, 4)[0]
    ref = AdamW([p.clone().cuda()], state_bits=bits, **HY)
    ref.step([g.cuda()])
    sd = torch.float32 if bits == 32 else torch.uint8

    def odd(t, off=3):
        buf = torch.full((n + 16,), 5, dtype=t.dtype).cuda()
        buf[off:off + n] = t
        return buf, buf[off:off + n]

    pb, pv = odd(p)
    gb, gv = odd(g)
    mb, mv = odd(torch.zeros(n, dtype=sd))
    vb, vv = odd(torch.zeros(n, dtype=sd))
    kw = {}
    if bits == 8:
        mv, vv = mv.view(F8), vv.view(F8)
        kw = dict(exp_avg_scale=[torch.zeros(24, device="cuda")], exp_avg_sq_scale=[torch.zeros(24, device="cuda")])
    opt = AdamW([pv], state_bits=bits, exp_avg=[mv], exp_avg_sq=[vv], **kw, **HY)
    opt.step([gv])
    assert torch.equal(pv, ref.params[0]) and torch.equal(mv.float(), ref.exp_avg[0].float())
    assert torch.equal(vv.float(), ref.exp_avg_sq[0].float())
    for b in (pb, gb, mb, vb):
        assert (b[:3].float() == 5).all() and (b[3 + n:].float() == 5).all()


@gpu
@pytest.mark.parametrize("count", [48, 49, 450, 900])
def test_many_tensors(count):
    from lm_head_jsd_gb300 import AdamW

    sizes = [(i * 37) % 300 + 1 for i in range(count)]
    ps, gs = _tensors(sizes, torch.float32, 0.02, 5), _tensors(sizes, torch.float32, 0.01, 6)
    opt = AdamW([p.cuda() for p in ps], **HY)
    gs = [None if i % 7 == 3 else g.cuda() for i, g in enumerate(gs)]
    opt.step(gs)
    for p, g, q in zip(ps, gs, opt.params):
        want = p.numpy() if g is None else _f32_step(p.numpy(), _np(g), 0 * p.numpy(), 0 * p.numpy(), 1)[0]
        assert np.array_equal(_np(q), want)


@gpu
def test_nan_stays_in_its_element_or_block_and_replaced_storage():
    from lm_head_jsd_gb300 import AdamW

    p = torch.nn.Parameter(torch.ones(300, device="cuda"))
    opt = AdamW([p], state_bits=8, **HY)
    p.grad = torch.ones(300, device="cuda")
    p.grad[5] = math.nan
    opt.step()
    assert torch.isnan(p.detach()).nonzero().flatten().tolist() == [5]
    assert torch.isfinite(opt.exp_avg_scale[0]).all()
    old = p.detach()
    p.data = torch.ones(300, device="cuda")
    kept = old.clone()
    p.grad = torch.ones(300, device="cuda")
    opt.step()
    assert torch.equal(old[10:], kept[10:]) and not torch.equal(p.detach()[10:], torch.ones(290, device="cuda"))


@gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_step_in_a_graph_on_another_stream(bits):
    from lm_head_jsd_gb300 import AdamW

    p = torch.randn(5000, device="cuda")
    q = p.clone()
    g = torch.randn(5000, device="cuda")
    a, b = AdamW([p], state_bits=bits, **HY), AdamW([q], state_bits=bits, **HY)
    a.step([g])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        b.step([g])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(p, q) and torch.equal(a.exp_avg[0].float(), b.exp_avg[0].float())


@gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_offsets_past_32_bits(bits):
    from lm_head_jsd_gb300 import AdamW

    n, tail = (1 << 31) + 3001, 3001 + 128 * 7
    p = torch.empty(n, dtype=torch.bfloat16, device="cuda").normal_(0, 0.02)
    g = torch.empty(n, dtype=torch.bfloat16, device="cuda").normal_(0, 0.01)
    small = AdamW([p[-tail:].clone()], state_bits=bits, **HY)
    AdamW([p], state_bits=bits, **HY).step([g])
    small.step([g[-tail:].clone()])
    assert torch.equal(p[-tail:], small.params[0])
