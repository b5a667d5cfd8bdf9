"""A serving step with nothing to adapt: no tokens are an empty result, and arguments are checked as for some."""
import pytest
import torch

gpu = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def fl():
    from conftest import build_library

    build_library()
    import lm_head_jsd_gb300 as fl

    return fl


def _args(device, dtype=BF, tokens=0):
    z = lambda *s: torch.zeros(*s, device=device)  # noqa: E731
    return dict(y=z(tokens, 100).to(dtype), x=z(tokens, 64).to(BF), a=z(2, 8, 64).to(BF), b=z(2, 100, 8).to(BF),
                index=torch.zeros(tokens, dtype=torch.int64, device=device))


def test_are_no_error_of_the_shape(fl):
    with pytest.raises(ValueError, match="expected a CUDA device"):
        fl.low_rank_add(**_args("cpu"))
    for bad in (dict(y=torch.zeros(0, 0)), dict(y=torch.zeros(0)), dict(x=torch.zeros(0, 0).to(BF))):
        with pytest.raises(ValueError, match="must be a matrix"):
            fl.low_rank_add(**{**_args("cpu"), **bad})


@gpu
@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "fp32"])
def test_give_an_empty_result(fl, dtype):
    z, status = _args("cuda", dtype), torch.full((1,), 77, dtype=torch.int32, device="cuda")
    got = fl.low_rank_add(**z, status=status)
    assert got.shape == (0, 100) and got.dtype == dtype and got.is_cuda and status.item() == 0
    assert fl.low_rank_add(**z, out=z["y"]) is z["y"]
    side = torch.cuda.Stream()
    status.fill_(77)
    torch.cuda.synchronize()
    assert fl.low_rank_add(**z, out=got, status=status, stream=side) is got
    side.synchronize()
    assert status.item() == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fl.low_rank_add(**z, status=status)
    status.fill_(77)
    graph.replay()
    assert status.item() == 0


@gpu
def test_are_checked_as_some_are(fl):
    z = _args("cuda")
    for bad in (dict(x=z["x"][:, :32]), dict(x=_args("cuda", tokens=1)["x"]), dict(a=z["a"][0]), dict(b=z["b"][:, :99]), dict(index=z["index"].int()),
                dict(scales=torch.ones(3, device="cuda")), dict(out=z["y"].float()), dict(out=z["y"][:, :50]), dict(y=z["y"].half()),
                dict(status=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            fl.low_rank_add(**{**z, **bad})
