"""Low-rank adapters on a shared projection: refusals (CPU), and the GPU against 64 bits over ranks, ragged groups
of tokens, odd sizes, strides and alignments, and on the 8-bit head."""
import math

import pytest
import torch

gpu = pytest.mark.gpu
BF, NAN, INF = torch.bfloat16, math.nan, math.inf


@pytest.fixture(scope="module", autouse=True)
def fl():
    from conftest import build_library

    build_library()
    import lm_head_jsd_gb300 as fl

    return fl


# ---- refusals (no GPU) ----
GOOD = dict(tokens=4, k=64, n=100, rank=16, adapters=2, x=4096, ldx=64, a=8192, b=16384, index=64, scales=None, dtype=1,
            y=256, ldy=100, out=512, ldo=100, workspace=4096, workspace_bytes=1 << 20)
BAD = [dict(tokens=0), dict(k=0), dict(n=0), dict(rank=0), dict(rank=12), dict(adapters=0), dict(x=None), dict(x=4097), dict(ldx=63),
       dict(a=None), dict(a=8193), dict(b=None), dict(b=16392), dict(index=None), dict(index=68), dict(scales=66), dict(dtype=2),
       dict(y=None), dict(y=257), dict(y=258, dtype=0), dict(ldy=99), dict(out=None), dict(out=513), dict(ldo=99),
       dict(out=256, ldo=101), dict(workspace=None), dict(workspace=8)]


@pytest.mark.parametrize("bad", BAD, ids=str)
def test_refused(fl, bad):
    assert fl.fljsd_low_rank_add(**{**GOOD, **bad}, stream=0, check=False) == 1


def test_refused_sizes(fl):
    call = lambda **kw: fl.fljsd_low_rank_add(**{**GOOD, **kw}, stream=0, check=False)  # noqa: E731
    assert call(tokens=(1 << 20) + 1) == 2 and call(k=(1 << 20) + 8, ldx=1 << 21) == 2 and call(rank=136) == 2
    assert call(n=(1 << 26) + 1, ldy=1 << 27, ldo=1 << 27) == 2 and call(adapters=4097) == 2
    assert call(workspace_bytes=fl.fljsd_low_rank_workspace_bytes(4, 2, 16) - 1) == 3


def _host(**kw):
    z = dict(y=torch.zeros(3, 10).to(BF), x=torch.zeros(3, 8).to(BF), a=torch.zeros(2, 8, 8).to(BF), b=torch.zeros(2, 10, 8).to(BF),
             index=torch.zeros(3).long())
    return {**z, **kw}


def test_refused_in_python(fl):
    with pytest.raises(ValueError, match="expected a CUDA device"):
        fl.low_rank_add(**_host())
    from lm_head_jsd_gb300.low_rank import check_adapters

    h = _host()
    args = lambda **kw: [kw.get(i, v) for i, v in (("x", h["x"]), ("n", 10), ("a", h["a"]), ("b", h["b"]), ("index", h["index"]),  # noqa: E731
                                                    ("scales", None))]
    assert check_adapters(*args()) == (2, 8)
    for bad in (dict(x=h["x"].float()), dict(a=h["a"][0]), dict(a=h["a"].float()), dict(a=h["a"][:, :, :4]), dict(a=h["a"][:, :4]),
                dict(a=h["a"].transpose(1, 2)), dict(b=h["b"][:1]), dict(b=h["b"][:, :9]), dict(b=h["b"].float()), dict(n=11),
                dict(index=h["index"].int()), dict(index=h["index"][:2]), dict(scales=torch.ones(3)), dict(scales=torch.ones(2).double()),
                dict(b=h["b"].clone().requires_grad_()), dict(x=h["x"].clone().requires_grad_())):
        with pytest.raises(ValueError):
            check_adapters(*args(**bad))
    with torch.no_grad():
        check_adapters(*args(b=h["b"].clone().requires_grad_()))


# ---- on the GPU ----
def _index(kind, tokens, adapters, g):
    r = torch.randint(0, adapters, (tokens,), generator=g)
    if kind == "sorted":
        return r.sort().values
    if kind == "some":
        return torch.where(torch.rand(tokens, generator=g) < 0.4, -1, r)
    if kind == "one":
        return torch.full((tokens,), adapters - 1)
    if kind == "none":
        return torch.full((tokens,), -1)
    return torch.arange(tokens) % adapters if kind == "own" else r


def _make(tokens, k, n, rank, adapters, kind="any", dtype=BF, seed=0):
    g = torch.Generator().manual_seed(seed + tokens + k + n + rank)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    z = dict(y=r(tokens, n).to(dtype), x=r(tokens, k).to(BF), a=(r(adapters, rank, k) / math.sqrt(k)).to(BF), b=r(adapters, n, rank).to(BF),
             index=_index(kind, tokens, adapters, g), scales=torch.rand(adapters, generator=g) + 0.5)
    return {key: v.cuda() for key, v in z.items()}


def _want(z):
    """(result, how far a kernel's may be from it) in 64 bits."""
    y, x, sc = z["y"].double(), z["x"].double(), z["scales"].double()
    want, far = y.clone(), torch.zeros_like(y)
    k, rk = x.shape[1], (z["a"].shape[1] + 15) // 16 * 16
    for i in range(z["a"].shape[0]):
        at = (z["index"] == i).nonzero()[:, 0]
        if len(at):
            a, b = z["a"][i].double(), z["b"][i].double()
            s, s_abs = sc[i] * (x[at] @ a.T), sc[i] * (x[at].abs() @ a.abs().T)
            d, d_abs = s @ b.T, s.abs() @ b.abs().T
            want[at] += d
            # sums: a rounding (2^-22, whichever way the tensor core rounds) for each instruction of 16 products and each
            # of eight parts; s as two bf16 2^-16, as three 2^-24; the second product likewise, of twice or three times the
            # rank; the sum with y
            lost, parts = (2.0 ** -16, 2) if z["y"].dtype == BF else (2.0 ** -24, 3)
            far[at] = (((k + 15) // 16 + 10) * 2.0 ** -22 * s_abs + lost * s.abs()) @ b.abs().T
            far[at] += (parts * rk / 16 + 2) * 2.0 ** -22 * d_abs + 2.0 ** -24 * (y[at].abs() + d_abs)
    return want, far + torch.finfo(z["y"].dtype).eps / 2 * want.abs()


def _near(got, z):
    want, far = _want(z)
    assert ((got.double() - want).abs() <= far).all(), ((got.double() - want).abs() / far).max()


CASES = [(1, 64, 256, 16, 1, "one"), (1, 8, 1, 8, 1, "one"), (2, 100, 2, 8, 3, "any"), (5, 1, 257, 24, 2, "some"), (63, 130, 255, 16, 1, "one"),
         (64, 520, 1000, 64, 4, "own"), (65, 63, 1025, 128, 1, "one"), (200, 1000, 2049, 40, 3, "some"), (130, 264, 511, 16, 70, "any"),
         (70, 512, 1300, 16, 70, "own"), (300, 64, 300, 32, 5, "sorted"), (33, 4096, 129, 128, 2, "any"), (20, 72, 600, 16, 4, "none")]


@gpu
@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_against_64_bits(fl, case, dtype):
    z = _make(*case, dtype=dtype)
    kept = {k: v.clone() for k, v in z.items()}
    status = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    got = fl.low_rank_add(**z, status=status)
    assert got.dtype == dtype and got.data_ptr() != z["y"].data_ptr() and status.item() == 0
    _near(got, z)
    assert all(torch.equal(z[k], kept[k]) for k in z)
    none = z["index"] == -1
    assert torch.equal(got[none], z["y"][none])
    assert fl.low_rank_add(**z, out=z["y"]) is z["y"] and torch.equal(z["y"], got)
    z = {**kept, "scales": None}
    one = fl.low_rank_add(**z)
    _near(one, {**z, "scales": torch.ones(case[4], device="cuda")})


@gpu
@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "fp32"])
def test_strides_and_alignments(fl, dtype):
    z = _make(77, 136, 515, 16, 3, "some", dtype)
    want = fl.low_rank_add(**z)
    wide = lambda t, pad, off, fill: torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device="cuda")[:, off:off + t.shape[1]]  # noqa: E731
    for pad, off in ((1, 0), (1, 1), (8, 0), (9, 3), (13, 8)):
        x, y, out = wide(z["x"], pad, off, NAN), wide(z["y"], pad, off, NAN), torch.full((77, 515 + pad), 7.0, dtype=dtype, device="cuda")
        x.copy_(z["x"])
        y.copy_(z["y"])
        view = out[:, off:off + 515]
        fl.low_rank_add(y, x, *[z[k] for k in ("a", "b", "index", "scales")], out=view)
        assert torch.equal(view, want)
        view.fill_(7.0)
        assert out.eq(7).all()  # what lies between the rows is as it was
        fl.low_rank_add(y, x, *[z[k] for k in ("a", "b", "index", "scales")], out=y)
        assert torch.equal(y, want)
    flat = torch.empty(1 + z["a"].numel(), dtype=BF, device="cuda")
    a = flat[1:].view_as(z["a"]).copy_(z["a"])  # a need not be aligned
    assert torch.equal(fl.low_rank_add(**{**z, "a": a}), want)


@gpu
def test_a_row_depends_on_its_own_alone(fl):
    z = _make(150, 200, 700, 16, 4, "some")
    want = fl.low_rank_add(**z)
    for t in (0, 7, 149):
        one = {k: v[t:t + 1] if k in ("x", "y", "index") else v for k, v in z.items()}
        assert torch.equal(fl.low_rank_add(**one)[0], want[t])
    order = torch.randperm(150, generator=torch.Generator().manual_seed(1)).cuda()
    moved = {k: v[order].contiguous() if k in ("x", "y", "index") else v for k, v in z.items()}
    assert torch.equal(fl.low_rank_add(**moved), want[order])
    # NaN and infinities stay in their rows
    bad = {**z, "x": z["x"].clone(), "y": z["y"].clone()}
    at = (z["index"] >= 0).nonzero()[:, 0][[0, 3, 5]]
    bad["x"][at[0], 5], bad["x"][at[1], 6], bad["y"][at[2], 9] = NAN, INF, INF
    got = fl.low_rank_add(**bad)
    rest = torch.ones(150, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(got[rest], want[rest]) and torch.isnan(got[at[0]]).all() and not torch.isfinite(got[at[1]]).any()
    assert got[at[2], 9] == INF and torch.equal(got[at[2], :9], want[at[2], :9])


@gpu
def test_nan_in_adapters_that_are_not_used(fl):
    z = _make(40, 64, 300, 24, 5, "any")
    z["index"] = torch.where(z["index"] == 2, 3, z["index"])
    want = fl.low_rank_add(**z)
    z["a"][2], z["b"][2] = NAN, NAN
    z["scales"][2] = NAN
    assert torch.equal(fl.low_rank_add(**z), want)


@gpu
def test_index_out_of_range(fl):
    z = _make(50, 64, 300, 16, 3, "any")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in (3, -2, 1 << 40, -(1 << 60)):
        i = z["index"].clone()
        i[7] = bad
        got = fl.low_rank_add(**{**z, "index": i}, status=status)
        assert status.item() == 1 and torch.equal(got[7], z["y"][7])
        i[7] = -1
        assert torch.equal(fl.low_rank_add(**{**z, "index": i}, status=status), got) and status.item() == 0


@gpu
def test_many_tokens_and_adapters(fl):
    z = _make(5000, 64, 40, 8, 4096, "any")
    z["index"] = torch.randint(0, 4096, (5000,), device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    got = fl.low_rank_add(**z)
    s = torch.einsum("tk,trk->tr", z["x"].double(), z["a"].double()[z["index"]]) * z["scales"].double()[z["index"]][:, None]
    want = z["y"].double() + torch.einsum("tr,tnr->tn", s, z["b"].double()[z["index"]])
    # |s| < 8, |b| < 6 and |x||a| sums below 16: sums and s (2^-16) within 8 * 6 * 8 * 2^-15, and bf16's own
    assert ((got.double() - want).abs() <= 384 * 2.0 ** -15 + 2.0 ** -8 * want.abs()).all()


@gpu
def test_offsets_past_32_bits(fl):
    n, tokens, adapters, rank = 1 << 18, 9000, 70, 128
    b = torch.empty(adapters, n, rank, dtype=BF, device="cuda")
    a = torch.empty(adapters, rank, 64, dtype=BF, device="cuda")
    g = torch.Generator("cuda").manual_seed(3)
    a[-1].normal_(generator=g)
    b[-1].normal_(generator=g)
    y = torch.zeros(tokens, n, dtype=BF, device="cuda")
    index = torch.full((tokens,), -1, device="cuda")
    index[-1] = adapters - 1
    x = torch.zeros(tokens, 64, dtype=BF, device="cuda")
    x[-1].normal_(generator=g)
    fl.low_rank_add(y, x, a, b, index, out=y)
    assert not y[:-1].any()
    _near(y[-1:], dict(y=torch.zeros(1, n, dtype=BF, device="cuda"), x=x[-1:], a=a[-1:], b=b[-1:], index=torch.zeros(1, device="cuda").long(),
                       scales=torch.ones(1, device="cuda")))


@gpu
def test_captured(fl):
    z = _make(90, 128, 900, 16, 4, "some")
    graph = torch.cuda.CUDAGraph()
    fl.low_rank_add(**z)
    with torch.cuda.graph(graph):
        got = fl.low_rank_add(**z)
    for seed, kind in ((1, "own"), (2, "one"), (3, "none")):  # other groups than those of the capture
        new = _make(90, 128, 900, 16, 4, kind, seed=seed)
        for k in z:
            z[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, fl.low_rank_add(**z))


@gpu
def test_on_a_given_stream(fl):
    z = _make(90, 128, 900, 16, 4, "some")
    want = fl.low_rank_add(**z)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (side, side.cuda_stream):
        got = fl.low_rank_add(**z, stream=s)
        side.synchronize()
        assert torch.equal(got, want)


@gpu
def test_two_streams_at_once(fl):
    zs = [_make(300, 256, 5000, 32, 6, "some", seed=i) for i in range(2)]
    want = [fl.low_rank_add(**z) for z in zs]
    streams = [torch.cuda.Stream() for _ in zs]
    torch.cuda.synchronize()
    got = [[fl.low_rank_add(**z, stream=s) for z, s in zip(zs, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for pair in got for a, b in zip(pair, want))


@gpu
def test_refusals_on_the_gpu(fl):
    z = _make(6, 64, 100, 16, 2)
    for bad in (dict(x=z["x"][:5]), dict(x=z["x"].cpu()), dict(y=z["y"].half()), dict(y=z["y"][0]), dict(y=z["y"][:, ::2]),
                dict(index=z["index"].cpu()), dict(out=z["y"][:5]), dict(out=z["y"].float()), dict(y=z["y"].clone().requires_grad_()),
                dict(status=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            fl.low_rank_add(**{**z, **bad})
    buf = torch.zeros(7, 100, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="shares memory"):
        fl.low_rank_add(**{**z, "y": buf[:6]}, out=buf[1:])
    flat = torch.zeros(1 + z["b"].numel(), dtype=BF, device="cuda")
    with pytest.raises(fl.FljsdError):
        fl.low_rank_add(**{**z, "b": flat[1:].view_as(z["b"])})


def test_what_shares_memory(fl):
    from lm_head_jsd_gb300.low_rank import check_apart

    buf = torch.zeros(6, 64, dtype=BF)
    out = buf[:, 16:48]
    for t in (buf[:, :16], buf[:, 48:], buf[:, 48:64], torch.zeros(6, 32, dtype=BF), None):
        check_apart(out, x=t)
    for t in (out, buf, buf[:, :17], buf[:, 47:], buf[2:, 20:24], buf[:, :16].view(torch.int32)[:, :8].as_strided((6, 9), (32, 1)),
              buf.view(-1)[100:120], buf.view(-1)[64 + 16:64 + 17], buf[1:, :].as_strided((2, 3, 8), (24, 8, 1))):
        with pytest.raises(ValueError, match="out shares memory with x"):
            check_apart(out, x=t)


@gpu
@pytest.mark.parametrize("name", ["x", "a", "b", "index", "scales"])
def test_a_result_on_an_input_is_refused(fl, name):
    z = _make(64, 64, 64, 16, 2)
    q = fl.fp8_quantize(torch.randn(64, 64, device="cuda"))
    buf = torch.zeros(64, 64, dtype=BF, device="cuda")
    if name == "x":
        z["x"] = buf
    else:
        t = z[name]
        z[name] = buf.view(-1)[:t.numel() * t.element_size() // 2].view(t.dtype).view(t.shape)
    with pytest.raises(ValueError, match=f"out shares memory with {name}"):
        fl.low_rank_add(**z, out=buf)
    with pytest.raises(ValueError, match=f"out shares memory with {name}"):
        fl.fp8_linear(z["x"], *q, adapters=(z["a"], z["b"], z["index"], z["scales"]), out=buf)


@gpu
def test_input_and_result_in_columns_of_one_matrix(fl):
    z = _make(70, 64, 100, 16, 3)
    want = fl.low_rank_add(**z)
    buf = torch.full((70, 200), 7.0, dtype=BF, device="cuda")
    x, out = buf[:, 8:72], buf[:, 80:180]
    x.copy_(z["x"])
    before = buf.clone()
    fl.low_rank_add(**{**z, "x": x}, out=out)
    assert torch.equal(out, want)
    assert torch.equal(buf[:, :80], before[:, :80]) and torch.equal(buf[:, 180:], before[:, 180:])


@gpu
def test_versions_rise(fl):
    z = _make(6, 64, 100, 16, 2, dtype=torch.float32)
    w = torch.ones(6, 100, device="cuda", requires_grad=True)
    out = (w * z["y"]).sum()
    fl.low_rank_add(**z, out=z["y"])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.backward()


@gpu
@pytest.mark.parametrize("m", [1, 16, 17, 200])
@pytest.mark.parametrize("out_dtype", [BF, torch.float32], ids=["bf16", "fp32"])
def test_on_the_8_bit_head(fl, m, out_dtype):
    z = _make(m, 256, 1003, 16, 3, "some" if m > 1 else "one")
    q = fl.fp8_quantize(torch.randn(1003, 256, device="cuda"))
    status = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    y = fl.fp8_linear(z["x"], *q, out_dtype=out_dtype)
    want = fl.low_rank_add(y, z["x"], z["a"], z["b"], z["index"], z["scales"])
    got = fl.fp8_linear(z["x"], *q, out_dtype=out_dtype, adapters=(z["a"], z["b"], z["index"], z["scales"]), status=status)
    assert torch.equal(got, want) and status.item() == 0
    into = torch.empty(m, 1010, dtype=out_dtype, device="cuda")[:, 3:1006]
    fl.fp8_linear(z["x"], *q, out_dtype=out_dtype, adapters=(z["a"], z["b"], z["index"], z["scales"]), out=into)
    assert torch.equal(into, want)
    one = fl.fp8_linear(z["x"], *q, out_dtype=out_dtype, adapters=(z["a"], z["b"], z["index"]))
    assert torch.equal(one, fl.low_rank_add(y, z["x"], z["a"], z["b"], z["index"]))
    i = z["index"].clone()
    i[0] = 99
    fl.fp8_linear(z["x"], *q, adapters=(z["a"], z["b"], i), status=status)
    assert status.item() == 1
    with pytest.raises(ValueError, match="adapters expect"):
        fl.fp8_linear(z["x"].float(), *q, adapters=(z["a"], z["b"], z["index"]))
