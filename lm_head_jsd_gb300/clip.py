"""The norm of many gradients taken together, and clipping (the C entry points
fljsd_grad_norm and fljsd_clip_grads)."""
from __future__ import annotations

import math
from operator import attrgetter

import numpy as np
import torch
from torch.autograd.graph import increment_version

from . import _lib
from ._streams import hand_over, on, require_cuda
from .api import _DT

# the layout of fljsd_grad_tensor
_ENTRY = np.dtype([("grad", np.uint64), ("out", np.uint64), ("n", np.int64), ("dtype", np.int32),
                   ("reserved", np.int32)])
_DTYPE, _DEVICE = attrgetter("dtype"), torch.Tensor.get_device  # (-1 off the GPUs)
_KINDS = {2.0: _lib.FLJSD_NORM_2, math.inf: _lib.FLJSD_NORM_MAX}


def _kind(norm_type):
    if norm_type not in _KINDS:
        raise ValueError(f"norm_type is {norm_type}, expected 2 or inf")
    return _KINDS[norm_type]


def check_max_norm(max_norm):
    if not max_norm >= 0:
        raise ValueError(f"max_norm is {max_norm}, expected a number that is not negative")


def _live(grads):
    grads = [grads] if isinstance(grads, torch.Tensor) else list(grads)
    live = [g for g in grads if g is not None]
    if not live:
        raise ValueError("no gradients")
    return grads, live


def _describe(name, ts):
    """(device, addresses, sizes, dtypes) of a list that is checked as a whole: a call of many
    small tensors is bound by this function."""
    try:
        devices, at = set(map(_DEVICE, ts)), list(map(torch.Tensor.data_ptr, ts))
    except TypeError:
        raise ValueError(f"{name} must be tensors") from None
    require_cuda(f"{name}[0]", ts[0])
    dev, dtypes = ts[0].device, list(map(_DTYPE, ts))
    if (not set(dtypes) <= _DT.keys() or devices != {dev.index}
            or not all(map(torch.Tensor.is_contiguous, ts))):
        raise ValueError(f"{name} must be contiguous, each of one dtype of {list(_DT)}, and on {dev}")
    return dev, at, list(map(torch.Tensor.numel, ts)), dtypes


def table(grads, sizes, dtypes, outs=None):
    """fljsd_grad_tensor of each, of their addresses, sizes and dtypes (or the one of all)."""
    t = np.zeros(len(grads), dtype=_ENTRY)
    t["grad"], t["n"] = grads, sizes
    one = dtypes if isinstance(dtypes, torch.dtype) else dtypes[0] if len(set(dtypes)) == 1 else None
    t["dtype"] = [_lib.DTYPES[_DT[d]] for d in dtypes] if one is None else _lib.DTYPES[_DT[one]]
    if outs is not None:
        t["out"] = outs
    return t


def workspace(count, device):
    return torch.empty(_lib.lib.fljsd_grad_norm_workspace_bytes(count), dtype=torch.uint8, device=device)


def grad_norm(grads, *, norm_type=2.0, stream=None):
    """The norm of all gradients taken together, an fp32 scalar on their device (nothing is
    read back): the root of the sum of their squares, or with ``norm_type`` inf the largest
    magnitude. ``grads``: a tensor or a list of fp32 and bf16 tensors; None is left out."""
    kind, (_, live) = _kind(norm_type), _live(grads)
    dev, at, sizes, dtypes = _describe("grads", live)
    t = table(at, sizes, dtypes)
    with on(stream, dev):
        norm = torch.empty((), dtype=torch.float32, device=dev)
        ws = workspace(len(t), dev)
        _lib.call("fljsd_grad_norm", t.ctypes.data, len(t), kind, 0.0, None, norm.data_ptr(), None,
                  ws.data_ptr(), ws.shape[0])
    hand_over((norm,), stream, dev)
    return norm


def clip_grads(grads, max_norm, *, norm_type=2.0, out=None, stream=None):
    """Scales the gradients in place by min(1, max_norm / (norm + 1e-6)), and returns their
    norm before that (as :func:`grad_norm`). ``out``: tensors like the gradients that
    receive the scaled ones instead (None where the gradient is None). A norm of NaN makes
    every gradient NaN. No tensor may be given twice, or share memory with another."""
    kind, (every, live) = _kind(norm_type), _live(grads)
    check_max_norm(max_norm)
    dev, at, sizes, dtypes = _describe("grads", live)
    outs, outs_at = live, at
    if out is not None:
        out = [out] if isinstance(out, torch.Tensor) else list(out)
        if len(out) != len(every):
            raise ValueError(f"out has {len(out)} tensors, expected {len(every)}")
        outs = [o for o, g in zip(out, every) if g is not None]
        other, outs_at, *alike = _describe("out", outs)
        if other != dev or alike != [sizes, dtypes]:
            raise ValueError(f"out must have the gradients' dtypes and sizes, on {dev}")
    t = table(at, sizes, dtypes, outs_at)
    _apart(t, out is not None)
    with on(stream, dev):
        norm = torch.empty((), dtype=torch.float32, device=dev)
        ws = workspace(len(t), dev)
        _lib.call("fljsd_clip_grads", t.ctypes.data, len(t), kind, max_norm, norm.data_ptr(),
                  ws.data_ptr(), ws.shape[0])
    hand_over((norm,), stream, dev)
    # autograd's own check of what it saved: these have changed
    increment_version(outs)
    return norm


def _apart(t, given):
    """That what is written overlaps nothing else of the call."""
    t = t[t["n"] > 0]
    size = np.where(t["dtype"] == _lib.DTYPES["bf16"], 2, 4).astype(np.uint64)
    begin, bytes_ = t["out"], t["n"].astype(np.uint64) * size
    writes = np.ones(len(t), dtype=bool)
    if given:  # (a gradient that is its own out counts once)
        other = t["grad"] != t["out"]
        begin = np.concatenate([begin, t["grad"][other]])
        bytes_ = np.concatenate([bytes_, bytes_[other]])
        writes = np.concatenate([writes, np.zeros(other.sum(), dtype=bool)])
    order = np.argsort(begin, kind="stable")
    begin, end, writes = begin[order], (begin + bytes_)[order], writes[order]
    # the farthest end of what lies before each, of all and of what is written
    far, far_written = np.maximum.accumulate(end), np.maximum.accumulate(np.where(writes, end, 0))
    if ((begin[1:] < far[:-1]) & writes[1:]).any() or (begin[1:] < far_written[:-1]).any():
        raise ValueError("tensors of the call overlap in memory that it writes")


__all__ = ["clip_grads", "grad_norm"]
