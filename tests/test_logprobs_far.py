"""Given logits of a large size, where the product with log2(e) / T is off by whole units of
the exponent before it is put right."""
import numpy as np
import pytest
import torch

import test_logprobs as base
from oracle import lp_rows_ref
from parity_util import f64

gpu = pytest.mark.gpu


def _far(dtype, temperature):
    """Logits whose scaled value, 2^31 to 2^32, is rounded by 126 to 128, down and up."""
    c = np.float32(1.4426950408889634 / np.float64(np.float32(temperature)))
    step = 128 if dtype == torch.float32 else 1 << 23  # (a spacing of the type's values there)
    z = torch.arange(int(2.0 ** 31 / c) // step + 1, int(2.0 ** 32 / c) // step)
    z = (z[-(1 << 17):].double() * step).to(dtype).double().unique().numpy()
    lo = z * np.float64(c) - (z.astype(np.float32) * c).astype(np.float64)
    return [float(z[hit][0]) for hit in ((lo > 126.05) & (lo < 127.95), (lo < -126.05) & (lo > -127.95))
            if hit.any()]


FAR = [(d, t, s * z) for d, ts in ((torch.float32, (1.0, 0.7)), (torch.bfloat16, (0.75, 1.1, 1.5)))
       for t in ts for z in _far(d, t) for s in (1, -1)]


def test_there_are_such_logits():
    assert {p[0] for p in FAR} == {torch.float32, torch.bfloat16}


# whole segments (a row of 8192 from its start), one that ends inside, and many rows
@gpu
@pytest.mark.parametrize("rows,v", [(1, 8192), (3, 20000), (700, 16384)])
@pytest.mark.parametrize("dtype,t,z", FAR,
                         ids=[f"{str(p[0])[6:]}-{p[1]}-{p[2]:.9g}" for p in FAR])
def test_rows_of_far_equal_logits(dtype, t, z, rows, v):
    from lm_head_jsd_gb300 import logits_logprobs

    x = torch.full((rows, v), z, dtype=dtype)
    if rows > 1:
        x[rows - 1, 7] = z + abs(z) / 64  # one row with a logit above the rest
    y = torch.arange(rows) % v
    r = logits_logprobs(x.cuda(), y.cuda(), top_k=2, temperature=t)
    few = [0, rows - 1]
    ref = lp_rows_ref(f64(x[few]), y.numpy()[few], top_k=2, temperature=t)
    base._check_rows([None if q is None else q[few] for q in r], ref, 0.0, "far")
    # rows between are all alike
    assert all(torch.equal(q[:1].expand(rows - 1, *q.shape[1:])[: rows - 1], q[: rows - 1])
               for q in (r.lse, r.entropy))
