"""Verification of drafted tokens against the target's probabilities (the C entry point
fljsd_verify). The formulas and the treatment of masked, empty and bad rows are in
include/fljsd.h."""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _lib
from ._streams import check_status, hand_over, on, report, require_cuda
from .api import _DT

_F32, _I64 = torch.float32, torch.int64


class Verified(NamedTuple):
    """tokens [requests, max_drafts + 1]: the accepted tokens, the drawn one, -1 behind;
    accepted [requests]: how many of the drafted tokens were; accept_prob [drafts]: the
    probability with which each drafted token is accepted, min(1, p / q)."""

    tokens: torch.Tensor
    accepted: torch.Tensor
    accept_prob: torch.Tensor


def _check_vector(name, t, dtype, n, device):
    if (not isinstance(t, torch.Tensor) or t.dtype != dtype or tuple(t.shape) != (n,)
            or not t.is_contiguous() or t.device != device):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor [{n}] on {device}")


def _check_logits(name, z, rows, v, dtype, device):
    if (not isinstance(z, torch.Tensor) or z.shape != (rows, v) or z.dtype != dtype
            or z.device != device):
        raise ValueError(f"{name} must be {dtype} [{rows}, {v}] on {device}")
    if z.stride(1) != 1 and v > 1 and rows > 0:
        raise ValueError(f"the rows of {name} must be contiguous")
    return z.stride(0) if rows > 1 else max(z.stride(0), v)


def verify_drafts(target_logits, draft_tokens, u_accept, u_draw, *, draft_logits=None, offsets=None,
                  max_drafts=None, temperature=1.0, status=None, stream=None) -> Verified:
    """Accepts or refuses drafted tokens [drafts] (int64) of a batch of requests, one request
    for each number of ``u_draw``, and draws the token that comes next, from given numbers in
    [0, 1) (fp32): ``u_accept`` one for each drafted token, ``u_draw`` one for each request.

    ``offsets`` [requests + 1] (int64, on the device): request b drafted
    draft_tokens[offsets[b]:offsets[b + 1]], at most ``max_drafts`` of them (requests that
    offsets describe wrongly, and all from the first that fall on, are refused); None: all as
    many. ``target_logits`` [drafts + requests, v], fp32 or bf16: request b's rows from
    offsets[b] + b on, one in front of each drafted token and one behind the last;
    ``draft_logits`` [drafts, v]: what each was drafted from (None: they have no
    probabilities). ``temperature``: a number, or fp32 [requests] on the device; 0: greedy.

    The tokens follow the target's probabilities. They depend on a request's own logits
    and numbers alone, not on the batch or on how the work is split. Carries no gradient.
    ``status``: an int32 on the device that receives the call's status word (0,
    FLJSD_ERR_INVALID_ARG where a drafted token, an offset or a temperature is out of
    range, or FLJSD_ERR_TIMEOUT)."""
    z = target_logits
    if not isinstance(z, torch.Tensor) or z.dim() != 2 or z.dtype not in _DT:
        raise ValueError(f"target_logits must be a matrix of one of {list(_DT)}")
    require_cuda("target_logits", z)
    dev, v = z.device, z.shape[1]
    if not isinstance(u_draw, torch.Tensor) or u_draw.dim() != 1 or not u_draw.numel():
        raise ValueError("u_draw must have a number for each request")
    if not isinstance(draft_tokens, torch.Tensor) or draft_tokens.dim() != 1:
        raise ValueError("draft_tokens must be a vector")
    b, n = u_draw.shape[0], draft_tokens.shape[0]
    if offsets is None:
        if n % b or (max_drafts is not None and max_drafts * b != n):
            raise ValueError(f"{n} drafted tokens of {b} requests need offsets")
        max_drafts = n // b
    else:
        _check_vector("offsets", offsets, _I64, b + 1, dev)
        if max_drafts is None or max_drafts < 0:
            raise ValueError("offsets need max_drafts, the most that a request may draft")
    # (in one expression: a call of few requests is bound by what is looked at)
    if not (isinstance(u_accept, torch.Tensor) and draft_tokens.dtype == _I64 and u_accept.dtype == _F32
            and u_draw.dtype == _F32 and u_accept.shape == (n,) and draft_tokens.is_contiguous()
            and u_accept.is_contiguous() and u_draw.is_contiguous() and draft_tokens.device == dev
            and u_accept.device == dev and u_draw.device == dev):
        _check_vector("draft_tokens", draft_tokens, _I64, n, dev)
        _check_vector("u_accept", u_accept, _F32, n, dev)
        _check_vector("u_draw", u_draw, _F32, b, dev)
    ld = _check_logits("target_logits", z, n + b, v, z.dtype, dev)
    ldd = v
    if draft_logits is not None:
        ldd = _check_logits("draft_logits", draft_logits, n, v, z.dtype, dev)
    each = None
    if isinstance(temperature, torch.Tensor):
        _check_vector("temperature", temperature, _F32, b, dev)
        each, temperature = temperature, 1.0
    check_status(status, dev)
    with on(stream, dev):
        r = Verified(torch.empty((b, max_drafts + 1), dtype=_I64, device=dev),
                     torch.empty(b, dtype=_I64, device=dev), torch.empty(n, dtype=_F32, device=dev))
        size = _lib.lib.fljsd_verify_workspace_bytes(b, n)
        ws = torch.empty(size, dtype=torch.uint8, device=dev)
        _lib.call("fljsd_verify", b, n, v, max_drafts, _lib.DTYPES[_DT[z.dtype]], z.data_ptr(), ld,
                  draft_logits.data_ptr() if draft_logits is not None and n else None, ldd,
                  draft_tokens.data_ptr(), u_accept.data_ptr(), u_draw.data_ptr(),
                  offsets.data_ptr() if offsets is not None else None,
                  each.data_ptr() if each is not None else None, temperature, r.tokens.data_ptr(),
                  r.accepted.data_ptr(), r.accept_prob.data_ptr(), ws.data_ptr(), size)
        report(status, ws)
    hand_over(r, stream, dev)
    return r


__all__ = ["Verified", "verify_drafts"]
