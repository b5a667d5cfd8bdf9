"""8-bit product with a scale for each block of 128: refusals (CPU), codes and scales
bit by bit and the product against float64 over odd sizes, strides and types (GPU)."""
import numpy as np
import pytest
import torch

from oracle import quantise_ref
from parity_util import f64

gpu = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def L():
    from conftest import build_library

    build_library()
    from lm_head_jsd_gb300 import _lib

    return _lib


def test_refusals_launch_nothing(L):
    b = 4096  # an aligned address that is never read: every call below is refused
    base = dict(m=4, n=100, k=64, xt="bf16", x=b, ldx=64, w=b, ldw=64, s=b, ot="bf16", o=b, ldo=100, ws=b,
                nb=1 << 20)

    def lin(**kw):
        return L.fljsd_fp8_linear(*{**base, **kw}.values(), stream=0, check=False)

    for bad in (dict(m=0), dict(n=-1), dict(k=0), dict(ldx=63), dict(ldw=63), dict(ldw=72), dict(ldo=99),
                dict(xt=7), dict(ot=-1), dict(x=None), dict(w=None), dict(s=None), dict(o=None),
                dict(ws=None), dict(x=b + 1), dict(w=b + 8), dict(s=b + 2), dict(o=b + 1), dict(ws=b + 8)):
        assert lin(**bad) == 1, bad
    assert lin(m=1 << 31) == 2 and lin(k=1 << 21, ldx=1 << 21, ldw=1 << 21) == 2
    assert lin(nb=L.fljsd_fp8_linear_workspace_bytes(4, 64) - 1) == 3
    base = dict(rows=4, cols=64, t="fp32", br=128, x=b, ldx=64, q=b, ldq=64, s=b)

    def quant(**kw):
        return L.fljsd_fp8_quantize(*{**base, **kw}.values(), stream=0, check=False)

    for bad in (dict(rows=0), dict(cols=0), dict(t=3), dict(br=64), dict(ldx=63), dict(ldq=48), dict(ldq=72),
                dict(x=None), dict(q=None), dict(s=None), dict(x=b + 2), dict(q=b + 8), dict(s=b + 1)):
        assert quant(**bad) == 1, bad
    assert L.fljsd_fp8_linear_workspace_bytes(0, 64) == 0


def test_wrapper_refusals():
    from lm_head_jsd_gb300 import fp8_linear, fp8_quantize

    x, w, s = torch.zeros(3, 64), torch.zeros(5, 64).to(F8), torch.zeros(1, 1)
    for args in ((x[0], w, s), (x.double(), w, s), (x, w.float(), s), (x, w[:, :32], s), (x, w, s.double()),
                 (x, w, torch.zeros(2, 1)), (torch.zeros(64, 3).T, w, s)):
        with pytest.raises(ValueError):
            fp8_linear(*args)
    with pytest.raises(ValueError):
        fp8_linear(x, w, s, out=torch.zeros(3, 4))
    for bad in (x[0], x.half(), torch.zeros(64, 3).T):
        with pytest.raises(ValueError):
            fp8_quantize(bad)


def _wide(q, s, block_rows):
    q, s = f64(q), f64(s)
    rows, cols = q.shape
    if block_rows == 1:
        return q * np.repeat(s.T, 128, 1)[:, :cols]
    return q * np.repeat(np.repeat(s, 128, 0)[:rows], 128, 1)[:, :cols]


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 130), (128, 128), (129, 200), (300, 1000)])
def test_quantise(rows, cols, dtype):
    from lm_head_jsd_gb300 import fp8_quantize

    x = torch.randn(rows, cols + 5, generator=torch.Generator().manual_seed(rows)).to(dtype)
    x[0] *= 1e-3
    if rows > 2:
        x[2] = 0
    xc = x.cuda()[:, 3:3 + cols]  # rows that start anywhere
    x = f64(x)[:, 3:3 + cols]
    q, s = fp8_quantize(xc, block_rows=1)
    for r in range(rows):
        val, sc = quantise_ref(x[r])
        assert np.array_equal(f64(q)[r], val) and np.array_equal(f64(s)[:, r], sc)
    q, s = fp8_quantize(xc)
    for i in range(0, rows, 128):
        for j in range(0, cols, 128):
            b = x[i:i + 128, j:j + 128]
            val, sc = quantise_ref(b.ravel(), block=b.size)
            assert np.array_equal(f64(q)[i:i + 128, j:j + 128], val.reshape(b.shape))
            assert f64(s)[i // 128, j // 128] == sc[0]


# an inner block is 128 products added 32 at a time to fp32, blocks are scaled and added
# in fp32, each addition off by at most a step of its sum; bf16 out adds half a step
def _limit(xq, wq, k, out_dtype, ref):
    mag = np.abs(xq) @ np.abs(wq).T
    lim = (k / 32 + 2 * k / 128 + 4) * 2.0 ** -23 * mag
    return lim + (2.0 ** -8 * np.abs(ref) if out_dtype == torch.bfloat16 else 0)


@gpu
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 1000, 64), (3, 257, 130), (128, 256, 128), (129, 512, 1000),
                                   (300, 1027, 512), (65, 2056, 2048), (2, 40960, 384),
                                   (16, 300, 8200), (3, 130, 40000), (17, 300, 8200), (1300, 2304, 256)])
def test_linear(m, n, k, out_dtype):
    from lm_head_jsd_gb300 import fp8_linear, fp8_quantize

    g = torch.Generator().manual_seed(m + n)
    x, w = torch.randn(m, k, generator=g), torch.randn(n, k, generator=g) / 8
    x = x.bfloat16() if m % 2 else x
    xc, wc = x.cuda(), w.cuda()
    wq, ws = fp8_quantize(wc)
    xq, xs = fp8_quantize(xc, block_rows=1)
    xv, wv = _wide(xq, xs, 1), _wide(wq, ws, 128)
    ref = xv @ wv.T
    lim = _limit(xv, wv, k, out_dtype, ref) + 1e-30
    got = fp8_linear(xc, wq, ws, out_dtype=out_dtype)
    assert (np.abs(f64(got) - ref) <= lim).all(), np.abs((f64(got) - ref) / lim).max()
    # into a wider buffer, from a wider x: nothing beside the result changes
    wide = torch.full((m, n + 9), 7.0, dtype=out_dtype, device="cuda")
    xw = torch.zeros(m, k + 3, dtype=x.dtype, device="cuda")
    xw[:, 3:] = xc
    fp8_linear(xw[:, 3:], wq, ws, out_dtype=out_dtype, out=wide[:, 2:2 + n])
    assert torch.equal(wide[:, 2:2 + n], got)
    assert (wide[:, :2] == 7).all() and (wide[:, 2 + n:] == 7).all()


@gpu
def test_linear_special_values_and_streams():
    from lm_head_jsd_gb300 import fp8_linear, fp8_quantize

    x = torch.randn(6, 256, generator=torch.Generator().manual_seed(0)).cuda()
    w = torch.randn(300, 256, generator=torch.Generator().manual_seed(1)).cuda()
    x[1] = 0
    x[2, 3] = float("nan")
    x[3] *= 1e-35  # blocks below the floor of amax
    x[4] *= 1e30
    wq, ws = fp8_quantize(w)
    out = fp8_linear(x, wq, ws, out_dtype=torch.float32)
    assert not out[1].any() and torch.isnan(out[2]).all() and out[3].abs().max() < 1e-28
    assert torch.isfinite(out[[0, 4, 5]]).all()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = fp8_linear(x, wq, ws, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(again.nan_to_num(), out.nan_to_num())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = fp8_linear(x, wq, ws, out_dtype=torch.float32)
    cap.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cap.nan_to_num(), out.nan_to_num())


@gpu
def test_linear_offsets_past_32_bits():
    from lm_head_jsd_gb300 import fp8_linear, fp8_quantize

    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(17000, 64, device="cuda", generator=g).bfloat16()
    wq, ws = fp8_quantize(torch.randn(128257, 64, device="cuda", generator=g))
    out = fp8_linear(x, wq, ws)
    assert torch.equal(out[-300:], fp8_linear(x[-300:], wq, ws))
