"""Products with a frozen weight held in 8-bit floating point, one scale for each block
of 128 (the C entry points fljsd_fp8_*)."""
from __future__ import annotations

import torch
from torch.autograd.graph import increment_version

from . import _lib
from ._streams import check_status, hand_over, on, report, require_cuda
from .api import _DT

BLOCK = 128


def _check_rows(name, t):
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or 0 in t.shape:
        raise ValueError(f"{name} must be a matrix")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def fp8_quantize(w, *, block_rows=BLOCK, stream=None):
    """(codes, scales) of a matrix, fp32 or bf16: e4m3 codes of its shape (rows a multiple
    of 16 bytes apart) and the fp32 scale of each 128 x 128 block, [ceil(rows / 128),
    ceil(cols / 128)]; with ``block_rows`` 1, of each 1 x 128, [ceil(cols / 128), rows]."""
    ld = _check_rows("w", w)
    if w.dtype not in _DT:
        raise ValueError(f"w has dtype {w.dtype}, expected one of {list(_DT)}")
    require_cuda("w", w)
    rows, cols = w.shape
    ldq, kb = -(-cols // 16) * 16, -(-cols // BLOCK)
    with on(stream, w.device):
        codes = torch.empty((rows, ldq), dtype=torch.uint8, device=w.device)
        scales = torch.empty((-(-rows // BLOCK), kb) if block_rows == BLOCK else (kb, rows),
                             dtype=torch.float32, device=w.device)
        _lib.fljsd_fp8_quantize(rows, cols, _DT[w.dtype], block_rows, w, ld, codes, ldq, scales)
    hand_over((codes, scales), stream, w.device)
    return codes.view(torch.float8_e4m3fn)[:, :cols], scales


def fp8_linear(x, w_codes, w_scales, *, out_dtype=torch.bfloat16, out=None, status=None, stream=None):
    """x.w^T of x [m, k] (fp32 or bf16, quantised on the way) and a weight from
    :func:`fp8_quantize`. Carries no gradient: an x that would need one is refused (pass
    ``x.detach()``, or call under ``torch.no_grad()``). ``status``: an int32 on the device
    that receives the call's status word (0, or FLJSD_ERR_TIMEOUT)."""
    if torch.is_grad_enabled() and isinstance(x, torch.Tensor) and x.requires_grad:
        raise ValueError("x requires a gradient, which fp8_linear does not give: pass x.detach()")
    ldx = _check_rows("x", x)
    ldw = _check_rows("w_codes", w_codes)
    (m, k), n, dev = x.shape, w_codes.shape[0], x.device
    require_cuda("x", x)
    check_status(status, dev)
    if x.dtype not in _DT or out_dtype not in _DT:
        raise ValueError(f"x and out_dtype must be one of {list(_DT)}")
    if w_codes.dtype != torch.float8_e4m3fn or w_codes.shape[1] != k or w_codes.device != dev:
        raise ValueError(f"w_codes must be float8_e4m3fn [n, {k}] on {dev}")
    if (w_scales.dtype != torch.float32 or not w_scales.is_contiguous() or w_scales.device != dev
            or tuple(w_scales.shape) != (-(-n // BLOCK), -(-k // BLOCK))):
        raise ValueError(f"w_scales must be fp32 [{-(-n // BLOCK)}, {-(-k // BLOCK)}] on {dev}")
    if out is not None and (out.dtype != out_dtype or tuple(out.shape) != (m, n) or out.device != dev):
        raise ValueError(f"out must be {out_dtype} [{m}, {n}] on {dev}")
    with on(stream, dev):
        y = out if out is not None else torch.empty((m, n), dtype=out_dtype, device=dev)
        ws = torch.empty(_lib.fljsd_fp8_linear_workspace_bytes(m, k), dtype=torch.uint8, device=dev)
        _lib.fljsd_fp8_linear(m, n, k, _DT[x.dtype], x, ldx, w_codes, ldw, w_scales, _DT[out_dtype],
                              y, _check_rows("out", y), ws)
        report(status, ws)
    if out is None:
        hand_over((y,), stream, dev)
    else:  # autograd's own check of what it saved: this has changed
        increment_version(out)
    return y


__all__ = ["fp8_linear", "fp8_quantize"]
