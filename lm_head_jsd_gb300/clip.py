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


def _checked(name, ts):
    """Their device; whole-list checks, for a call of many small tensors is bound by them."""
    require_cuda(f"{name}[0]", ts[0])
    dev = ts[0].device
    if (not set(map(_DTYPE, ts)) <= _DT.keys() or set(map(_DEVICE, ts)) != {dev.index}
            or not all(map(torch.Tensor.is_contiguous, ts))):
        raise ValueError(f"{name} must be contiguous, each of one dtype of {list(_DT)}, and on {dev}")
    return dev


def table(grads, outs=None):
    """fljsd_grad_tensor of each."""
    t = np.zeros(len(grads), dtype=_ENTRY)
    t["grad"] = list(map(torch.Tensor.data_ptr, grads))
    t["n"] = list(map(torch.Tensor.numel, grads))
    kinds = set(map(_DTYPE, grads))
    t["dtype"] = (_lib.DTYPES[_DT[kinds.pop()]] if len(kinds) == 1
                  else [_lib.DTYPES[_DT[g.dtype]] for g in grads])
    if outs is not None:
        t["out"] = t["grad"] if outs is grads else list(map(torch.Tensor.data_ptr, outs))
    return t


def workspace(count, device):
    return torch.empty(_lib.fljsd_grad_norm_workspace_bytes(count), dtype=torch.uint8, device=device)


def grad_norm(grads, *, norm_type=2.0, stream=None):
    """The norm of all gradients taken together, an fp32 scalar on their device (nothing is
    read back): the root of the sum of their squares, or with ``norm_type`` inf the largest
    magnitude. ``grads``: a tensor or a list of fp32 and bf16 tensors; None is left out."""
    kind, (_, live) = _kind(norm_type), _live(grads)
    dev = _checked("grads", live)
    t = table(live)
    with on(stream, dev):
        norm = torch.empty((), dtype=torch.float32, device=dev)
        _lib.fljsd_grad_norm(t.ctypes.data, len(t), kind, 0.0, None, norm, None,
                             workspace(len(t), dev))
    hand_over((norm,), stream, dev)
    return norm


def clip_grads(grads, max_norm, *, norm_type=2.0, out=None, stream=None):
    """Scales the gradients in place by min(1, max_norm / (norm + 1e-6)), and returns their
    norm before that (as :func:`grad_norm`). ``out``: tensors like the gradients that
    receive the scaled ones instead (None where the gradient is None). A norm of NaN makes
    every gradient NaN. No tensor may be given twice, or share memory with another."""
    kind, (every, live) = _kind(norm_type), _live(grads)
    check_max_norm(max_norm)
    dev = _checked("grads", live)
    outs = live
    if out is not None:
        out = [out] if isinstance(out, torch.Tensor) else list(out)
        if len(out) != len(every):
            raise ValueError(f"out has {len(out)} tensors, expected {len(every)}")
        outs = [o for o, g in zip(out, every) if g is not None]
        if not all(map(torch.is_tensor, outs)):
            raise ValueError("out has None where there is a gradient")
        require_cuda("out[0]", outs[0])
        if (list(map(_DTYPE, outs)) != list(map(_DTYPE, live)) or set(map(_DEVICE, outs)) != {dev.index}
                or list(map(torch.Tensor.numel, outs)) != list(map(torch.Tensor.numel, live))
                or not all(map(torch.Tensor.is_contiguous, outs))):
            raise ValueError(f"out must be contiguous, of the gradients' dtypes and sizes, on {dev}")
    t = table(live, outs)
    _apart(t, out is not None)
    with on(stream, dev):
        norm = torch.empty((), dtype=torch.float32, device=dev)
        _lib.fljsd_clip_grads(t.ctypes.data, len(t), kind, max_norm, norm, workspace(len(t), dev))
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
