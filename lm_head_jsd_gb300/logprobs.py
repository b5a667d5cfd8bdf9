"""Token log probabilities, entropies and most likely alternatives of an lm_head's
rows (the C entry points fljsd_lp_* and fljsd_logits_lp*), with allocation and
autograd. The formulas and the treatment of ignored, masked and empty rows are in
include/fljsd.h."""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch
from torch.autograd.graph import increment_version

from . import _lib
from ._streams import (Memory, capture_id, check_status, hand_over, on, report,
                       require_cuda)
from .api import _DT, _check


class Logprobs(NamedTuple):
    """Per row: log probability of the label (None without labels), entropy, log of
    the softmax denominator, the same in two parts for the backward pass (the largest
    logit, and log2 of the sum relative to it), and the top_k alternatives (None with
    top_k 0)."""

    logp: Optional[torch.Tensor]
    entropy: torch.Tensor
    lse: torch.Tensor
    norm: torch.Tensor
    top_logp: Optional[torch.Tensor]
    top_id: Optional[torch.Tensor]


def _results(rows, top_k, with_logp, device) -> Logprobs:
    f32 = lambda *shape: torch.empty(shape, dtype=torch.float32, device=device)  # noqa: E731
    return Logprobs(f32(rows) if with_logp else None, f32(rows), f32(rows), f32(rows, 2),
                    f32(rows, top_k) if top_k else None,
                    torch.empty((rows, top_k), dtype=torch.int64, device=device) if top_k else None)


def _check_result(r, rows, with_logp, device, top_k=None):
    """That a result is one of ``rows`` rows (and of ``top_k`` alternatives, to be written)."""
    need = [("logp", torch.float32, (rows,))] if with_logp else []
    need += [("entropy", torch.float32, (rows,)), ("norm", torch.float32, (rows, 2))]
    if top_k is not None:
        need.append(("lse", torch.float32, (rows,)))
        if top_k:
            need += [("top_logp", torch.float32, (rows, top_k)), ("top_id", torch.int64, (rows, top_k))]
    for name, dtype, shape in need:
        _check(f"the result's {name}", getattr(r, name), dtype, device, shape)


def _check_grad(name, t, rows, device):
    if t is not None:
        _check(name, t, torch.float32, device, (rows,))


class FusedLinearLogprobs:
    """Plans one problem shape and keeps its workspace for repeated calls.

    ``forward`` returns :class:`Logprobs` (``out``: a result to be written instead); with
    ``keep_for_backward`` the plan also serves ``backward``, which takes the upstream
    gradients of logp and entropy. A forward whose plan is one chunk leaves the
    probabilities (bt x v fp16) in the workspace for the first backward of its result; any
    other backward computes them again (so do captured calls, but for a backward in the
    capture of its forward, and eager ones of a plan that has been captured).
    """

    def __init__(self, bt, h, v, dtype=torch.bfloat16, *, top_k=0, temperature=1.0,
                 ignore_index=-100, chunk_rows=0, keep_for_backward=False, accum_fp32=False,
                 device="cuda", free_hbm_bytes=None):
        self.device = torch.device(device)
        require_cuda("the plan", self.device)
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        if dtype not in _DT:
            raise ValueError(f"dtype {dtype} is not one of {list(_DT)}")
        self.dtype = dtype
        self.problem = _lib.make_lp_problem(bt, h, v, _DT[dtype], top_k, temperature, ignore_index,
                                            chunk_rows, keep_for_backward, accum_fp32)
        if free_hbm_bytes is None:
            free_hbm_bytes = torch.cuda.mem_get_info(self.device)[0]
        self.plan = _lib.fljsd_lp_plan(self.problem, int(free_hbm_bytes))
        self.workspace = torch.empty(self.plan.workspace_bytes, dtype=torch.uint8,
                                     device=self.device)
        self._memory = Memory([self.workspace])
        # the result whose probabilities the workspace holds, and the capture it was made in
        self._kept, self._captured = (None, 0), False

    def forward(self, x, w, labels=None, out=None, stream=None) -> Logprobs:
        p = self.problem
        _check("x", x, self.dtype, self.device, (p.bt, p.h))
        _check("w", w, self.dtype, self.device, (p.v, p.h))
        if labels is not None:
            _check("labels", labels, torch.int64, self.device, (p.bt,))
        if out is not None:
            _check_result(out, p.bt, labels is not None, self.device, p.top_k)
        self._kept = None, 0
        with on(stream, self.device):
            self._memory.use()
            capture = capture_id()
            self._captured |= capture != 0
            r = _results(p.bt, p.top_k, labels is not None, self.device) if out is None else out
            _lib.fljsd_lp_forward(p, self.plan, x, w, labels, r.logp, r.entropy, r.lse, r.norm,
                                  r.top_logp, r.top_id, self.workspace)
        if out is None:
            hand_over(r, stream, self.device)
        else:  # autograd's own check of what it saved: these have changed
            increment_version([t for t in out if t is not None])
        if p.flags & _lib.FLJSD_LP_BACKWARD and self.plan.num_chunks == 1:
            self._kept = r, capture
        return r

    def report(self, status):
        """The status word of the calls so far (since the last forward) into an int32 on the
        device, on the current stream (None: nothing)."""
        check_status(status, self.device)
        report(status, self.workspace, self.plan.status_offset)

    def backward(self, x, w, labels, result, grad_logp=None, grad_entropy=None, out=None,
                 need=(True, True), stream=None):
        """(grad_input, grad_weight) for the upstream gradients of ``result``'s logp
        and entropy ([bt] fp32, None for zero); ``need`` skips one of them."""
        p = self.problem
        _check("x", x, self.dtype, self.device, (p.bt, p.h))
        _check("w", w, self.dtype, self.device, (p.v, p.h))
        if labels is not None:
            _check("labels", labels, torch.int64, self.device, (p.bt,))
        _check_grad("grad_logp", grad_logp, p.bt, self.device)
        _check_grad("grad_entropy", grad_entropy, p.bt, self.device)
        if out is not None:
            for name, t, like in zip(("grad_input", "grad_weight"), out, (x, w), strict=True):
                if t is not None:
                    _check(name, t, self.dtype, self.device, like.shape)
        (r, made), self._kept = self._kept, (None, 0)
        if r is not result:
            _check_result(result, p.bt, labels is not None, self.device)
        with on(stream, self.device):
            self._memory.use()
            capture = capture_id()
            # A captured backward runs once for each replay, and replays of a captured
            # forward or backward write the workspace unseen.
            kept = r is result and made == capture and (capture != 0 or not self._captured)
            self._captured |= capture != 0
            g = out if out is not None else (torch.empty_like(x) if need[0] else None,
                                             torch.empty_like(w) if need[1] else None)
            _lib.fljsd_lp_backward(p, self.plan, x, w, labels, result.logp, result.entropy,
                                   result.norm, grad_logp, grad_entropy, int(kept), g[0], g[1],
                                   self.workspace)
        if out is None:
            hand_over(g, stream, self.device)
        else:
            increment_version([t for t in out if t is not None])
        return g


def _outputs(ctx, r):
    """Views of a result as a Function's outputs: what backward keeps of the result
    must not refer to the graph. Only logp and entropy carry gradients."""
    out = tuple(None if t is None else t.view_as(t) for t in r)
    ctx.mark_non_differentiable(*(t for t in out[2:] if t is not None))
    return out


def _upstream(g):
    return None if g is None else g.detach().to(torch.float32).contiguous()


class _Once(torch.autograd.Function):
    """Gradients as functions of what they come from, whose derivative is not provided."""

    @staticmethod
    def forward(ctx, n, *tensors):
        return tuple(None if g is None else g.view_as(g) for g in tensors[:n])

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("token log probabilities are differentiable once: the derivative of "
                           "their gradient is not provided")


def _once(grads, of):
    """Under create_graph=True the gradients depend on ``of``; otherwise as they are."""
    return _Once.apply(len(grads), *grads, *of) if torch.is_grad_enabled() else grads


class _FusedLinearLogprobsFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, labels, top_k, temperature, ignore_index, chunk_rows, need, status):
        check_status(status, x.device)
        run = FusedLinearLogprobs(x.shape[0], x.shape[1], w.shape[0], x.dtype, top_k=top_k,
                                  temperature=temperature, ignore_index=ignore_index,
                                  chunk_rows=chunk_rows, keep_for_backward=need, device=x.device)
        r = run.forward(x, w, labels)
        run.report(status)
        ctx.set_materialize_grads(False)
        if need:
            ctx.run, ctx.result, ctx.status = run, r, status
            # (of the result, for the check that nothing has been written over it)
            ctx.save_for_backward(x, w, labels, r.logp, r.entropy, r.norm)
        return _outputs(ctx, r)

    @staticmethod
    def backward(ctx, g_logp, g_entropy, *_):
        if g_logp is None and g_entropy is None:
            return (None,) * 9
        x, w, labels, *_ = ctx.saved_tensors
        need = ctx.needs_input_grad[:2]
        gx, gw = ctx.run.backward(x, w, labels, ctx.result, _upstream(g_logp), _upstream(g_entropy),
                                  need=need)
        ctx.run.report(ctx.status)
        return *_once((gx, gw), (x, w, g_logp, g_entropy)), *(None,) * 7


def fused_linear_logprobs(x, w, labels=None, *, top_k=0, temperature=1.0, ignore_index=-100,
                          chunk_rows=0, status=None) -> Logprobs:
    """:class:`Logprobs` of the logits x.w^T without forming them, differentiable in x
    and w through logp and entropy, once. 2-D tensors on one CUDA device, fp32 or bf16.
    ``status``: an int32 on the device that receives the forward's status word, and again
    after a backward pass (0; FLJSD_ERR_INVALID_ARG for a label outside [0, V) other than
    ignore_index; FLJSD_ERR_TIMEOUT).

    To capture a backward pass into a CUDA graph, use :class:`FusedLinearLogprobs`, or
    leaves of its own (``x.detach().requires_grad_()``): autograd delivers a leaf's
    gradient on the stream of whatever eager graph of that leaf is still alive, which a
    capture forbids."""
    need = torch.is_grad_enabled() and (x.requires_grad or w.requires_grad)
    x, w = x.contiguous(), w.contiguous()
    labels = None if labels is None else labels.contiguous()
    return Logprobs(*_FusedLinearLogprobsFunction.apply(x, w, labels, int(top_k), float(temperature),
                                                        int(ignore_index), int(chunk_rows), need, status))


def _logits_check(logits, labels):
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("expected [rows x V] logits")
    if logits.dtype not in _DT:
        raise ValueError(f"logits have dtype {logits.dtype}, expected one of {list(_DT)}")
    if logits.stride(1) != 1 and logits.shape[1] > 1:
        raise ValueError("the rows of logits must be contiguous")
    require_cuda("logits", logits)
    if labels is not None:
        _check("labels", labels, torch.int64, logits.device, (logits.shape[0],))


def _row_stride(t):
    # a single row's stride may be anything, and an expanded tensor's rows are 0 apart
    return max(t.stride(0), t.shape[1]) if t.shape[0] == 1 else t.stride(0)


def logits_logprobs(logits, labels=None, *, top_k=0, temperature=1.0, ignore_index=-100,
                    status=None, stream=None) -> Logprobs:
    """:class:`Logprobs` of given logits [rows x V], fp32 or bf16 (rows may be any
    stride apart). For a differentiable form see :func:`token_logprobs`. ``status``: an
    int32 on the device that receives the call's status word (0, or FLJSD_ERR_INVALID_ARG
    for a label outside [0, V) other than ignore_index)."""
    _logits_check(logits, labels)
    (rows, v), dev = logits.shape, logits.device
    if status is not None:
        check_status(status, dev)
    with on(stream, dev):
        r = _results(rows, top_k, labels is not None, dev)
        ws = torch.empty(_lib.fljsd_logits_lp_workspace_bytes(rows, v, top_k), dtype=torch.uint8,
                         device=dev)
        _lib.fljsd_logits_lp(rows, v, _row_stride(logits), _DT[logits.dtype], top_k, temperature,
                             ignore_index, logits, labels, r.logp, r.entropy, r.lse, r.norm,
                             r.top_logp, r.top_id, ws)
        if status is not None:
            report(status, ws)
    if stream is not None:
        hand_over(r, stream, dev)
    return r


def logits_logprobs_backward(logits, labels, result, grad_logp=None, grad_entropy=None, *,
                             temperature=1.0, ignore_index=-100, out=None, stream=None):
    """The gradient in the logits for upstream gradients of ``result``'s logp and
    entropy ([rows] fp32, None for zero); ``out`` may be the logits themselves."""
    _logits_check(logits, labels)
    rows, v = logits.shape
    _check_grad("grad_logp", grad_logp, rows, logits.device)
    _check_grad("grad_entropy", grad_entropy, rows, logits.device)
    _check_result(result, rows, labels is not None, logits.device)
    if out is not None and (out.shape != logits.shape or out.dtype != logits.dtype or
                            out.device != logits.device or (out.stride(1) != 1 and v > 1)):
        raise ValueError("out must be like the logits, with contiguous rows")
    with on(stream, logits.device):
        g = out if out is not None else torch.empty((rows, v), dtype=logits.dtype,
                                                    device=logits.device)
        _lib.fljsd_logits_lp_backward(rows, v, _row_stride(logits), _row_stride(g),
                                      _DT[logits.dtype], temperature, ignore_index, logits, labels,
                                      result.logp, result.entropy, result.norm, grad_logp,
                                      grad_entropy, g)
    if out is None:
        hand_over((g,), stream, logits.device)
    else:
        increment_version(out)
    return g


class _TokenLogprobsFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, labels, top_k, temperature, ignore_index, status):
        r = logits_logprobs(logits, labels, top_k=top_k, temperature=temperature,
                            ignore_index=ignore_index, status=status)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(logits, labels, r.logp, r.entropy, r.norm)
        ctx.result, ctx.opts = r, (temperature, ignore_index)
        return _outputs(ctx, r)

    @staticmethod
    def backward(ctx, g_logp, g_entropy, *_):
        if g_logp is None and g_entropy is None:
            return (None,) * 6
        z, labels, *_ = ctx.saved_tensors
        g = logits_logprobs_backward(z, labels, ctx.result, _upstream(g_logp), _upstream(g_entropy),
                                     temperature=ctx.opts[0], ignore_index=ctx.opts[1])
        return *_once((g,), (z, g_logp, g_entropy)), *(None,) * 5


def token_logprobs(logits, labels=None, *, top_k=0, temperature=1.0, ignore_index=-100,
                   status=None) -> Logprobs:
    """:func:`logits_logprobs`, differentiable in the logits through logp and entropy, once."""
    if logits.dim() == 2 and (logits.stride(1) != 1 or logits.stride(0) < logits.shape[1]):
        logits = logits.contiguous()  # columns apart, or rows that share memory
    labels = None if labels is None else labels.contiguous()
    return Logprobs(*_TokenLogprobsFunction.apply(logits, labels, int(top_k), float(temperature),
                                                  int(ignore_index), status))


__all__ = ["FusedLinearLogprobs", "Logprobs", "fused_linear_logprobs", "logits_logprobs",
           "logits_logprobs_backward", "token_logprobs"]
