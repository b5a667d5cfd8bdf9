"""Low-rank adapters of many requests on the output of a shared projection (the C entry
point fljsd_low_rank_add)."""
from __future__ import annotations

import torch
from torch.autograd.graph import increment_version

from . import _lib
from ._streams import check_status, hand_over, on, report, require_cuda
from .api import _DT

_BF, _F32, _I64 = torch.bfloat16, torch.float32, torch.int64


def check_rows(name, t, least=1):
    """The row stride of a matrix of at least so many rows, which are contiguous."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.shape[0] < least or not t.shape[1]:
        raise ValueError(f"{name} must be a matrix")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _span(t):
    """The addresses that the elements of a tensor lie in."""
    last = sum((n - 1) * step for n, step in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + t.element_size() * (last + 1)


def check_apart(out, **inputs):
    """That out shares no memory with what is read after its first element is written."""
    lo, hi = _span(out)
    for name, t in inputs.items():
        if t is not None:
            begin, end = _span(t)
            if begin < hi and lo < end and not _beside(out, t):
                raise ValueError(f"out shares memory with {name}")


def _beside(out, t):
    """Whether two matrices are different columns of one."""
    pitch = out.stride(0) * out.element_size()
    if t.dim() != 2 or t.stride(0) * t.element_size() != pitch or not pitch:
        return False
    at = (t.data_ptr() - out.data_ptr()) % pitch
    return out.shape[1] * out.element_size() <= at <= pitch - t.shape[1] * t.element_size()


def check_adapters(x, n, a, b, index, scales):
    """That adapters fit x [tokens, k] and an output of n columns; their (number, rank)."""
    (tokens, k), dev = x.shape, x.device
    try:  # (in one expression: a call of few tokens is bound by what is looked at)
        count, rank, depth = a.shape
        fits = (x.dtype == _BF and a.dtype == _BF and b.dtype == _BF and index.dtype == _I64
                and depth == k and count > 0 and rank > 0 and rank % 8 == 0
                and b.shape == (count, n, rank) and index.shape == (tokens,)
                and a.is_contiguous() and b.is_contiguous() and index.is_contiguous()
                and a.device == dev and b.device == dev and index.device == dev
                and (scales is None or (scales.dtype == _F32 and scales.shape == (count,)
                                        and scales.is_contiguous() and scales.device == dev)))
    except (AttributeError, ValueError):  # no tensor, or not of three dimensions
        fits = False
    if not fits:
        _refuse(x, n, a, b, index, scales)
    if torch.is_grad_enabled() and (x.requires_grad or a.requires_grad or b.requires_grad
                                    or (scales is not None and scales.requires_grad)):
        raise ValueError("an input requires a gradient, which adapters here do not give: detach it")
    return count, rank


def _refuse(x, n, a, b, index, scales):
    (tokens, k), dev = x.shape, x.device
    if x.dtype != _BF:
        raise ValueError(f"x has dtype {x.dtype}, adapters expect {_BF}")
    if not isinstance(a, torch.Tensor) or a.dim() != 3 or a.shape[0] == 0 or a.shape[1] == 0:
        raise ValueError("a must be [adapters, rank, k]")
    count, rank = a.shape[:2]
    if rank % 8:
        raise ValueError(f"the rank is {rank}, expected a multiple of 8 (pad a and b with zeros)")
    for name, t, dtype, shape in (("a", a, _BF, (count, rank, k)), ("b", b, _BF, (count, n, rank)),
                                  ("index", index, _I64, (tokens,)), ("scales", scales, _F32, (count,))):
        if not (t is None and name == "scales") and (
                not isinstance(t, torch.Tensor) or t.dtype != dtype or tuple(t.shape) != shape
                or not t.is_contiguous() or t.device != dev):
            raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on {dev}")


def add(tokens, n, count, rank, x, ldx, a, b, index, scales, y, ldy, out, ldo):
    """The call, of arguments that are checked; its workspace."""
    size = _lib.lib.fljsd_low_rank_workspace_bytes(tokens, count, rank)
    ws = torch.empty(size, dtype=torch.uint8, device=y.device)
    _lib.call("fljsd_low_rank_add", tokens, x.shape[1], n, rank, count, x.data_ptr(), ldx, a.data_ptr(),
              b.data_ptr(), index.data_ptr(), scales.data_ptr() if scales is not None else None,
              _lib.DTYPES[_DT[y.dtype]], y.data_ptr(), ldy, out.data_ptr(), ldo, ws.data_ptr(), size)
    return ws


def low_rank_add(y, x, a, b, index, scales=None, *, out=None, status=None, stream=None):
    """y + scales[i] b[i] (a[i] x) for each token, i = index of the token (int64 [tokens]; -1:
    y as it is). y [tokens, n] (no tokens too) fp32 or bf16, x [tokens, k] bf16, a [adapters, rank, k] and
    b [adapters, n, rank] bf16 with a rank that is a multiple of 8 up to 128, scales fp32
    [adapters] or None (1). ``out``: receives the result, y itself or a tensor like it that
    shares no memory with any input. For serving: carries no gradient, and an input that
    would need one is refused. ``status``: an int32 on the device that receives the call's
    status word (0, FLJSD_ERR_INVALID_ARG for an index out of range, which counts as -1, or
    FLJSD_ERR_TIMEOUT)."""
    ldy = check_rows("y", y, 0)
    ldx = check_rows("x", x, 0)
    (tokens, n), dev = y.shape, y.device
    require_cuda("y", y)
    if y.dtype not in _DT:
        raise ValueError(f"y has dtype {y.dtype}, expected one of {list(_DT)}")
    if x.shape[0] != tokens or x.device != dev:
        raise ValueError(f"x must have {tokens} rows on {dev}")
    count, rank = check_adapters(x, n, a, b, index, scales)
    if torch.is_grad_enabled() and y.requires_grad:
        raise ValueError("y requires a gradient, which low_rank_add does not give: detach it")
    check_status(status, dev)
    if out is not None:
        if (not isinstance(out, torch.Tensor) or out.dtype != y.dtype or tuple(out.shape) != (tokens, n)
                or out.device != dev):
            raise ValueError(f"out must be {y.dtype} [{tokens}, {n}] on {dev}")
        ldr = check_rows("out", out, 0)
        same = out.data_ptr() == y.data_ptr() and (ldr == ldy or tokens == 1)
        if same:
            ldr = ldy
        if tokens:
            check_apart(out, y=None if same else y, x=x, a=a, b=b, index=index, scales=scales)
    with on(stream, dev):
        r = out
        if out is None:
            r, ldr = torch.empty((tokens, n), dtype=y.dtype, device=dev), n
        if tokens:
            ws = add(tokens, n, count, rank, x, ldx, a, b, index, scales, y, ldy, r, ldr)
            report(status, ws)
        elif status is not None:
            status.zero_()
    if out is None:
        hand_over((r,), stream, dev)
    else:  # autograd's own check of what it saved: this has changed
        increment_version(out)
    return r


__all__ = ["low_rank_add"]
