"""Failure detection without a GPU fault: the bounded waits of verification and of the adapters. What others wait for is
left out, their waits expire after 50 ms, and the status word says so; the next call on the same context is right."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, TIMEOUT = torch.bfloat16, 5


@pytest.fixture(scope="module", autouse=True)
def fl():
    from conftest import build_library

    build_library()
    import lm_head_jsd_gb300 as fl

    return fl


@pytest.fixture
def stall(fl):
    """Switches a kernel's stall on, and off again whatever happens."""
    yield fl._lib.fljsd_test_stall
    fl._lib.fljsd_test_stall(0)
    torch.cuda.synchronize()


def _drafts(v, dtype, requests=3, drafts=5, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    n = requests * drafts
    z = (torch.randn(n + requests, v, device="cuda", generator=g) * 3).to(dtype)
    zd = (torch.randn(n, v, device="cuda", generator=g) * 3).to(dtype)
    tok = torch.randint(0, v, (n,), device="cuda", generator=g)
    return dict(target_logits=z, draft_tokens=tok, u_accept=torch.rand(n, device="cuda", generator=g),
                u_draw=torch.rand(requests, device="cuda", generator=g), draft_logits=zd)


# one CTA to a row, clusters of two and more, rows of which each CTA keeps a part only
@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("v", [500, 20000, 128256, 400000])
def test_verification(fl, stall, v, dtype):
    x = _drafts(v, dtype)
    want = fl.verify_drafts(**x)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    stall(fl._lib.FLJSD_STALL_VERIFY)
    fl.verify_drafts(**x, status=status)
    torch.cuda.synchronize()
    assert status.item() == TIMEOUT
    stall(0)
    got = fl.verify_drafts(**x, status=status)
    assert status.item() == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


def test_verification_of_more_rows_than_clusters(fl, stall):
    x = _drafts(3000, BF, requests=400)
    want = fl.verify_drafts(**x)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    stall(fl._lib.FLJSD_STALL_VERIFY)
    fl.verify_drafts(**x, status=status)
    torch.cuda.synchronize()
    assert status.item() == TIMEOUT
    stall(0)
    got = fl.verify_drafts(**x, status=status)
    assert status.item() == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("bad", ["token", "temperature", "offsets"])
def test_verification_of_a_bad_request(fl, stall, bad):
    """That there are no results is known whatever is wrong with a request."""
    x, status = _drafts(3000, BF), torch.zeros(1, dtype=torch.int32, device="cuda")
    if bad == "token":
        x["draft_tokens"][2] = -1
    elif bad == "temperature":
        x["temperature"] = torch.tensor([1.0, -1.0, 1.0], device="cuda")
    else:
        x |= dict(offsets=torch.tensor([0, 5, 11, 15], device="cuda"), max_drafts=5)
    fl.verify_drafts(**x, status=status)
    assert status.item() == 1
    stall(fl._lib.FLJSD_STALL_VERIFY)
    fl.verify_drafts(**x, status=status)
    torch.cuda.synchronize()
    assert status.item() == TIMEOUT


def _adapters(tokens, k, n, rank, adapters, dtype):
    g = torch.Generator("cuda").manual_seed(tokens + n)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return dict(y=r(tokens, n).to(dtype), x=r(tokens, k).to(BF), a=(r(adapters, rank, k) / k ** 0.5).to(BF), b=r(adapters, n, rank).to(BF),
                index=torch.randint(0, adapters, (tokens,), device="cuda", generator=g))


# few tiles and many, one CTA on an SM and two, rows on 16 bytes and others, jobs of one block and of several
@pytest.mark.parametrize("name", ["FIRST", "SECOND", "Y"])
@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("case", [(5, 200, 512, 16, 2), (100, 520, 4099, 16, 70), (130, 64, 20000, 64, 3), (300, 1000, 33333, 128, 4)],
                         ids=lambda c: "-".join(map(str, c)))
def test_adapters(fl, stall, case, dtype, name):
    z = _adapters(*case, dtype)
    want = fl.low_rank_add(**z)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    stall(getattr(fl._lib, f"FLJSD_STALL_LOW_RANK_{name}"))
    fl.low_rank_add(**z, status=status)
    torch.cuda.synchronize()
    assert status.item() == TIMEOUT
    stall(0)
    assert torch.equal(fl.low_rank_add(**z, status=status), want) and status.item() == 0


def test_adapters_on_the_8_bit_head(fl, stall):
    z = _adapters(40, 256, 1000, 16, 3, BF)
    q = fl.fp8_quantize(torch.randn(1000, 256, device="cuda", generator=torch.Generator("cuda").manual_seed(1)))
    call = lambda: fl.fp8_linear(z["x"], *q, adapters=(z["a"], z["b"], index), status=status)  # noqa: E731
    status, index = torch.zeros(1, dtype=torch.int32, device="cuda"), z["index"].clone()
    want = call()
    index[3] = 7  # (an index that names no adapter does not hide it)
    stall(fl._lib.FLJSD_STALL_LOW_RANK_SECOND)
    call()
    torch.cuda.synchronize()
    assert status.item() == TIMEOUT
    stall(0)
    call()
    assert status.item() == 1
    index.copy_(z["index"])
    assert torch.equal(call(), want) and status.item() == 0
