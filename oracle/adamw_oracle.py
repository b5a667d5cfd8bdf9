"""Float64 reference of an AdamW step and the 8-bit form of its states (NumPy)."""
from __future__ import annotations

import numpy as np


def adamw_ref(p, g, m, v, step, *, lr, betas, eps, weight_decay):
    """(p, m, v) after step number ``step``, in float64."""
    p, g, m, v = (np.asarray(t, dtype=np.float64) for t in (p, g, m, v))
    b1, b2 = betas
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    mhat, vhat = m / (1 - b1 ** step), v / (1 - b2 ** step)
    return p - lr * weight_decay * p - lr * mhat / (np.sqrt(vhat) + eps), m, v


def e4m3_values():
    """The 127 non-negative values of e4m3 (4 exponent bits of bias 7, 3 of mantissa, no
    infinities), ascending."""
    return np.array([(i & 7) * 2.0 ** -9 if i < 8 else (1 + (i & 7) / 8) * 2.0 ** ((i >> 3) - 7)
                     for i in range(127)])


def quantise_ref(x, block=128):
    """(codes' values, scales) of consecutive blocks: scale = amax (1 / 448) with amax not
    below 2^-100, value = the e4m3 nearest to x (448 (1 / amax)) (ties to the even
    mantissa). In float32, one rounding to an operation, as the definition has it."""
    x = np.asarray(x, dtype=np.float32)
    vals = e4m3_values()
    out, scales = np.zeros_like(x), []
    for i in range(0, x.size, block):
        b = x[i:i + block]
        amax = np.float32(max(np.abs(b).max(), np.float32(2.0 ** -100)))
        y = (np.abs(b) * (np.float32(448) * (np.float32(1) / amax))).astype(np.float64)
        k = np.clip(np.searchsorted(vals, y), 1, 126)
        lo, hi = vals[k - 1], vals[k]
        up = (y - lo > hi - y) | ((y - lo == hi - y) & (k % 2 == 0))
        out[i:i + block] = np.copysign(np.where(up, hi, lo), b)
        scales.append(amax * np.float32(1 / 448))
    return out, np.array(scales, dtype=np.float32)
