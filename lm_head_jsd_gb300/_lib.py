"""ctypes binding of libfljsd.so (argument marshalling only).

The functions carry the names of the C entry points in include/fljsd.h. Tensor
arguments are torch tensors whose device pointers are passed through; no
arithmetic of the loss happens in Python. If the shared library is missing the
import fails: there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfljsd.so")

FLJSD_OK = 0
STATUS_NAMES = {0: "FLJSD_OK", 1: "FLJSD_ERR_INVALID_ARG", 2: "FLJSD_ERR_UNSUPPORTED",
                3: "FLJSD_ERR_WORKSPACE", 4: "FLJSD_ERR_CUDA", 5: "FLJSD_ERR_TIMEOUT"}
DTYPES = {"fp32": 0, "bf16": 1}
REDUCTIONS = {"none": 0, "sum": 1, "mean": 2, "batchmean": 3}
KERNEL_KINDS = {"gemm_logits": 0, "jsd_rows": 1, "gemm_grad_input": 2,
                "gemm_grad_weight": 3, "small": 4}


class FljsdError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} "
                         f"({fljsd_status_string(status)})")


class fljsd_problem(ctypes.Structure):
    _fields_ = [("bt", ctypes.c_int64), ("h_s", ctypes.c_int64), ("h_t", ctypes.c_int64),
                ("v", ctypes.c_int64), ("dtype", ctypes.c_int32), ("reduction", ctypes.c_int32),
                ("beta", ctypes.c_float), ("temperature", ctypes.c_float),
                ("ignore_index", ctypes.c_int64), ("chunk_rows", ctypes.c_int64),
                ("flags", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class fljsd_ce_problem(ctypes.Structure):
    _fields_ = [("bt", ctypes.c_int64), ("h", ctypes.c_int64), ("v", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reduction", ctypes.c_int32),
                ("ignore_index", ctypes.c_int64), ("chunk_rows", ctypes.c_int64),
                ("label_smoothing", ctypes.c_float), ("lse_square_scale", ctypes.c_float),
                ("softcap", ctypes.c_float), ("flags", ctypes.c_int32)]


class fljsd_lp_problem(ctypes.Structure):
    _fields_ = [("bt", ctypes.c_int64), ("h", ctypes.c_int64), ("v", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("ignore_index", ctypes.c_int64), ("chunk_rows", ctypes.c_int64),
                ("temperature", ctypes.c_float), ("flags", ctypes.c_int32)]


class fljsd_adamw_tensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("grad", "param", "master", "exp_avg", "exp_avg_sq",
                                               "exp_avg_scale", "exp_avg_sq_scale")] + [
        ("n", ctypes.c_int64)]


class fljsd_adamw_options(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay")] + [
        ("step", ctypes.c_int64), ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
        ("state_bits", ctypes.c_int32), ("master", ctypes.c_int32)]


class fljsd_grad_tensor(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


FLJSD_NORM_MAX, FLJSD_NORM_2 = 0, 2
FLJSD_FLAG_T2 = 1
FLJSD_FLAG_ACCUM_FP32 = 2
FLJSD_LP_BACKWARD = 4


class fljsd_plan_t(ctypes.Structure):
    _fields_ = [("chunk_rows", ctypes.c_int64), ("num_chunks", ctypes.c_int64),
                ("ld", ctypes.c_int64), ("workspace_bytes", ctypes.c_size_t),
                ("logits_bytes", ctypes.c_size_t), ("stats_bytes", ctypes.c_size_t),
                ("status_offset", ctypes.c_size_t)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python lm_head_jsd_gb300/build.py` (there is no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    lib.fljsd_plan.argtypes = [ctypes.POINTER(fljsd_problem), ctypes.c_size_t,
                               ctypes.POINTER(fljsd_plan_t)]
    lib.fljsd_plan.restype = ctypes.c_int
    lib.fljsd_forward.argtypes = [ctypes.POINTER(fljsd_problem), ctypes.POINTER(fljsd_plan_t),
                                  P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.fljsd_forward.restype = ctypes.c_int
    lib.fljsd_forward_noalloc.argtypes = [ctypes.POINTER(fljsd_problem), P, P, P, P, P, P, P, P,
                                          P, P]
    lib.fljsd_forward_noalloc.restype = ctypes.c_int
    lib.fljsd_backward.argtypes = [ctypes.POINTER(fljsd_problem), P, P, P, P]
    lib.fljsd_backward.restype = ctypes.c_int
    lib.fljsd_workspace_status.argtypes = [ctypes.POINTER(fljsd_plan_t), P, P,
                                           ctypes.POINTER(ctypes.c_int32)]
    lib.fljsd_workspace_status.restype = ctypes.c_int
    lib.fljsd_gemm_bf16.argtypes = [P, ctypes.c_int64, ctypes.c_int32, P, ctypes.c_int64,
                                    ctypes.c_int32, P, ctypes.c_int64, ctypes.c_int64,
                                    ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, P,
                                    ctypes.c_int32, P]
    lib.fljsd_gemm_bf16.restype = ctypes.c_int
    lib.fljsd_rows_workspace_bytes.argtypes = [ctypes.c_int64]
    lib.fljsd_rows_workspace_bytes.restype = ctypes.c_size_t
    lib.fljsd_jsd_logspace.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                       ctypes.c_float, ctypes.c_int32, ctypes.c_int64, P, P, P,
                                       P, P, P, ctypes.c_size_t, P]
    lib.fljsd_jsd_logspace.restype = ctypes.c_int
    lib.fljsd_tvd.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                              ctypes.c_int64, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.fljsd_tvd.restype = ctypes.c_int
    lib.fljsd_scale.argtypes = [ctypes.c_int32, P, ctypes.c_int64, P, P]
    lib.fljsd_scale.restype = ctypes.c_int
    lib.fljsd_ce_plan.argtypes = [ctypes.POINTER(fljsd_ce_problem), ctypes.c_size_t,
                                  ctypes.POINTER(fljsd_plan_t)]
    lib.fljsd_ce_plan.restype = ctypes.c_int
    lib.fljsd_ce_forward.argtypes = [ctypes.POINTER(fljsd_ce_problem),
                                     ctypes.POINTER(fljsd_plan_t), P, P, P, P, P, P, P,
                                     ctypes.c_size_t, P]
    lib.fljsd_ce_forward.restype = ctypes.c_int
    i32, i64, f32, size = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.fljsd_lp_plan.argtypes = [ctypes.POINTER(fljsd_lp_problem), size,
                                  ctypes.POINTER(fljsd_plan_t)]
    lib.fljsd_lp_plan.restype = ctypes.c_int
    lib.fljsd_lp_forward.argtypes = [ctypes.POINTER(fljsd_lp_problem),
                                     ctypes.POINTER(fljsd_plan_t), *[P] * 10, size, P]
    lib.fljsd_lp_forward.restype = ctypes.c_int
    lib.fljsd_lp_backward.argtypes = [ctypes.POINTER(fljsd_lp_problem),
                                      ctypes.POINTER(fljsd_plan_t), *[P] * 8, i32, P, P, P, size, P]
    lib.fljsd_lp_backward.restype = ctypes.c_int
    lib.fljsd_logits_lp_workspace_bytes.argtypes = [i64, i64, i32]
    lib.fljsd_logits_lp_workspace_bytes.restype = size
    lib.fljsd_logits_lp.argtypes = [i64, i64, i64, i32, i32, f32, i64, *[P] * 9, size, P]
    lib.fljsd_logits_lp.restype = ctypes.c_int
    lib.fljsd_logits_lp_backward.argtypes = [i64, i64, i64, i64, i32, f32, i64, *[P] * 9]
    lib.fljsd_logits_lp_backward.restype = ctypes.c_int
    lib.fljsd_adamw_step.argtypes = [ctypes.POINTER(fljsd_adamw_options), P, i32, P, P]
    lib.fljsd_adamw_step.restype = ctypes.c_int
    lib.fljsd_adamw_step_each.argtypes = [ctypes.POINTER(fljsd_adamw_options), P, P, i32, P, P]
    lib.fljsd_adamw_step_each.restype = ctypes.c_int
    lib.fljsd_grad_norm_workspace_bytes.argtypes = [i32]
    lib.fljsd_grad_norm_workspace_bytes.restype = size
    lib.fljsd_grad_norm.argtypes = [P, i32, i32, f32, P, P, P, P, size, P]
    lib.fljsd_grad_norm.restype = ctypes.c_int
    lib.fljsd_clip_grads.argtypes = [P, i32, i32, f32, P, P, size, P]
    lib.fljsd_clip_grads.restype = ctypes.c_int
    lib.fljsd_verify_workspace_bytes.argtypes = [i64, i64]
    lib.fljsd_verify_workspace_bytes.restype = size
    lib.fljsd_verify.argtypes = [i64, i64, i64, i32, i32, P, i64, P, i64, *[P] * 5, f32, *[P] * 4, size, P]
    lib.fljsd_verify.restype = ctypes.c_int
    lib.fljsd_low_rank_workspace_bytes.argtypes = [i64, i32, i32]
    lib.fljsd_low_rank_workspace_bytes.restype = size
    lib.fljsd_low_rank_add.argtypes = [i64, i64, i64, i32, i32, P, i64, P, P, P, P, i32, P, i64, P, i64, P,
                                       size, P]
    lib.fljsd_low_rank_add.restype = ctypes.c_int
    lib.fljsd_fp8_quantize.argtypes = [i64, i64, i32, i32, P, i64, P, i64, P, P]
    lib.fljsd_fp8_quantize.restype = ctypes.c_int
    lib.fljsd_fp8_linear_workspace_bytes.argtypes = [i64, i64]
    lib.fljsd_fp8_linear_workspace_bytes.restype = size
    lib.fljsd_fp8_linear.argtypes = [i64, i64, i64, i32, P, i64, P, i64, P, i32, P, i64, P, size, P]
    lib.fljsd_fp8_linear.restype = ctypes.c_int
    lib.fljsd_status_string.argtypes = [ctypes.c_int]
    lib.fljsd_status_string.restype = ctypes.c_char_p
    lib.fljsd_capture_id.argtypes = [P]
    lib.fljsd_capture_id.restype = ctypes.c_uint64
    lib.fljsd_test_stall.argtypes = [ctypes.c_int32]
    lib.fljsd_test_stall.restype = None
    lib.fljsd_launch_count.argtypes = []
    lib.fljsd_launch_count.restype = ctypes.c_int64
    lib.fljsd_launch_count_reset.argtypes = []
    lib.fljsd_launch_count_reset.restype = None
    lib.fljsd_trace_enable.argtypes = [ctypes.c_int32]
    lib.fljsd_trace_enable.restype = ctypes.c_int
    lib.fljsd_trace_reset.argtypes = []
    lib.fljsd_trace_reset.restype = ctypes.c_int
    lib.fljsd_trace_read.argtypes = [ctypes.c_int32, ctypes.POINTER(ctypes.c_double),
                                     ctypes.POINTER(ctypes.c_int64)]
    lib.fljsd_trace_read.restype = ctypes.c_int
    return lib


lib = _load()


def _ptr(t) -> int | None:
    """Device (or host) address of a tensor, None for None; ints pass through."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch

        if not torch.cuda.is_initialized():  # (is_available() would ask the driver at every call)
            return None
        # the handle alone: a Stream object takes longer to make than a launch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def make_problem(bt, h_s, h_t, v, dtype="bf16", reduction="batchmean", beta=0.5,
                 temperature=1.0, ignore_index=-100, chunk_rows=0, t2_scale=False,
                 accum_fp32=False) -> fljsd_problem:
    flags = (FLJSD_FLAG_T2 if t2_scale else 0) | (FLJSD_FLAG_ACCUM_FP32 if accum_fp32 else 0)
    return fljsd_problem(bt, h_s, h_t, v, DTYPES[dtype] if isinstance(dtype, str) else dtype,
                         REDUCTIONS[reduction] if isinstance(reduction, str) else reduction,
                         beta, temperature, ignore_index, chunk_rows, flags, 0)


def fljsd_status_string(status: int) -> str:
    return lib.fljsd_status_string(status).decode()


def fljsd_plan(problem: fljsd_problem, free_hbm_bytes: int = 0) -> fljsd_plan_t:
    plan = fljsd_plan_t()
    st = lib.fljsd_plan(ctypes.byref(problem), free_hbm_bytes, ctypes.byref(plan))
    if st != FLJSD_OK:
        raise FljsdError(st, "fljsd_plan")
    return plan


def fljsd_forward(problem, plan, x_s, w_s, x_t, w_t, labels, row_grad, loss, grad_input,
                  grad_weight, workspace, workspace_bytes=None, stream=None, check=True) -> int:
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    st = lib.fljsd_forward(ctypes.byref(problem), ctypes.byref(plan), _ptr(x_s), _ptr(w_s),
                           _ptr(x_t), _ptr(w_t), _ptr(labels), _ptr(row_grad), _ptr(loss),
                           _ptr(grad_input), _ptr(grad_weight), _ptr(workspace),
                           workspace_bytes, _stream(stream))
    if check and st != FLJSD_OK:
        raise FljsdError(st, "fljsd_forward")
    return st


def fljsd_forward_noalloc(problem, x_s, w_s, x_t, w_t, labels, row_grad, loss, grad_input,
                          grad_weight, stream=None, check=True) -> int:
    """fljsd_forward with the library's fixed device scratch instead of a
    caller-provided workspace (for callers that cannot allocate)."""
    st = lib.fljsd_forward_noalloc(ctypes.byref(problem), _ptr(x_s), _ptr(w_s), _ptr(x_t),
                                   _ptr(w_t), _ptr(labels), _ptr(row_grad), _ptr(loss),
                                   _ptr(grad_input), _ptr(grad_weight), _stream(stream))
    if check and st != FLJSD_OK:
        raise FljsdError(st, "fljsd_forward_noalloc")
    return st


def fljsd_backward(problem, grad_output, grad_input, grad_weight, stream=None,
                   check=True) -> int:
    st = lib.fljsd_backward(ctypes.byref(problem), _ptr(grad_output), _ptr(grad_input),
                            _ptr(grad_weight), _stream(stream))
    if check and st != FLJSD_OK:
        raise FljsdError(st, "fljsd_backward")
    return st


def fljsd_workspace_status(plan, workspace, stream=None) -> int:
    out = ctypes.c_int32()
    st = lib.fljsd_workspace_status(ctypes.byref(plan), _ptr(workspace), _stream(stream),
                                    ctypes.byref(out))
    if st != FLJSD_OK:
        raise FljsdError(st, "fljsd_workspace_status")
    return out.value


FLJSD_GEMM_SINGLE_CTA = 1
FLJSD_GEMM_TEST_STALL = 2


def fljsd_gemm_bf16(a, lda, a_mn, b, ldb, b_mn, d, ldd, m, n, k, accumulate=0, status=None,
                    flags=0, stream=None, check=True) -> int:
    st = lib.fljsd_gemm_bf16(_ptr(a), lda, a_mn, _ptr(b), ldb, b_mn, _ptr(d), ldd, m, n, k,
                             accumulate, _ptr(status), flags, _stream(stream))
    if check and st != FLJSD_OK:
        raise FljsdError(st, "fljsd_gemm_bf16")
    return st


def _dt(dtype):
    return DTYPES[dtype] if isinstance(dtype, str) else int(dtype)


def _red(reduction):
    return REDUCTIONS[reduction] if isinstance(reduction, str) else int(reduction)


def fljsd_rows_workspace_bytes(rows: int) -> int:
    return lib.fljsd_rows_workspace_bytes(rows)


def fljsd_jsd_logspace(rows, v, dtype, beta, reduction, ignore_index, input, target, labels,
                       loss, grad_input, workspace, workspace_bytes=None, stream=None,
                       check=True) -> int:
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    st = lib.fljsd_jsd_logspace(rows, v, _dt(dtype), beta, _red(reduction), ignore_index,
                                _ptr(input), _ptr(target), _ptr(labels), _ptr(loss),
                                _ptr(grad_input), _ptr(workspace), workspace_bytes,
                                _stream(stream))
    if check and st != FLJSD_OK:
        raise FljsdError(st, "fljsd_jsd_logspace")
    return st


def fljsd_tvd(rows, v, dtype, reduction, ignore_index, p, q, labels, loss, grad_p, workspace,
              workspace_bytes=None, stream=None, check=True) -> int:
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    st = lib.fljsd_tvd(rows, v, _dt(dtype), _red(reduction), ignore_index, _ptr(p), _ptr(q),
                       _ptr(labels), _ptr(loss), _ptr(grad_p), _ptr(workspace), workspace_bytes,
                       _stream(stream))
    if check and st != FLJSD_OK:
        raise FljsdError(st, "fljsd_tvd")
    return st


def fljsd_scale(dtype, x, n, grad_output, stream=None, check=True) -> int:
    st = lib.fljsd_scale(_dt(dtype), _ptr(x), n, _ptr(grad_output), _stream(stream))
    if check and st != FLJSD_OK:
        raise FljsdError(st, "fljsd_scale")
    return st


def make_ce_problem(bt, h, v, dtype="bf16", reduction="mean", ignore_index=-100, chunk_rows=0,
                    label_smoothing=0.0, lse_square_scale=0.0, softcap=0.0,
                    accum_fp32=False) -> fljsd_ce_problem:
    return fljsd_ce_problem(bt, h, v, _dt(dtype), _red(reduction), ignore_index, chunk_rows,
                            label_smoothing, lse_square_scale, softcap,
                            FLJSD_FLAG_ACCUM_FP32 if accum_fp32 else 0)


def fljsd_ce_plan(problem, free_hbm_bytes: int = 0) -> fljsd_plan_t:
    plan = fljsd_plan_t()
    st = lib.fljsd_ce_plan(ctypes.byref(problem), free_hbm_bytes, ctypes.byref(plan))
    if st != FLJSD_OK:
        raise FljsdError(st, "fljsd_ce_plan")
    return plan


def fljsd_ce_forward(problem, plan, x, w, labels, loss, grad_input, grad_weight, workspace,
                     workspace_bytes=None, stream=None, check=True) -> int:
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    st = lib.fljsd_ce_forward(ctypes.byref(problem), ctypes.byref(plan), _ptr(x), _ptr(w),
                              _ptr(labels), _ptr(loss), _ptr(grad_input), _ptr(grad_weight),
                              _ptr(workspace), workspace_bytes, _stream(stream))
    if check and st != FLJSD_OK:
        raise FljsdError(st, "fljsd_ce_forward")
    return st


def make_lp_problem(bt, h, v, dtype="bf16", top_k=0, temperature=1.0, ignore_index=-100,
                    chunk_rows=0, backward=False, accum_fp32=False) -> fljsd_lp_problem:
    flags = (FLJSD_LP_BACKWARD if backward else 0) | (FLJSD_FLAG_ACCUM_FP32 if accum_fp32 else 0)
    return fljsd_lp_problem(bt, h, v, _dt(dtype), top_k, ignore_index, chunk_rows, temperature,
                            flags)


def fljsd_lp_plan(problem, free_hbm_bytes: int = 0) -> fljsd_plan_t:
    plan = fljsd_plan_t()
    st = lib.fljsd_lp_plan(ctypes.byref(problem), free_hbm_bytes, ctypes.byref(plan))
    if st != FLJSD_OK:
        raise FljsdError(st, "fljsd_lp_plan")
    return plan


def fljsd_lp_forward(problem, plan, x, w, labels, logp, entropy, lse, norm, top_logp, top_id, workspace,
                     workspace_bytes=None, stream=None, check=True) -> int:
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    st = lib.fljsd_lp_forward(ctypes.byref(problem), ctypes.byref(plan), _ptr(x), _ptr(w),
                              _ptr(labels), _ptr(logp), _ptr(entropy), _ptr(lse), _ptr(norm),
                              _ptr(top_logp), _ptr(top_id), _ptr(workspace), workspace_bytes, _stream(stream))
    if check and st != FLJSD_OK:
        raise FljsdError(st, "fljsd_lp_forward")
    return st


def fljsd_lp_backward(problem, plan, x, w, labels, logp, entropy, norm, grad_logp, grad_entropy,
                      kept, grad_input, grad_weight, workspace, workspace_bytes=None, stream=None,
                      check=True) -> int:
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    st = lib.fljsd_lp_backward(ctypes.byref(problem), ctypes.byref(plan), _ptr(x), _ptr(w),
                               _ptr(labels), _ptr(logp), _ptr(entropy), _ptr(norm),
                               _ptr(grad_logp), _ptr(grad_entropy), kept, _ptr(grad_input),
                               _ptr(grad_weight), _ptr(workspace), workspace_bytes,
                               _stream(stream))
    if check and st != FLJSD_OK:
        raise FljsdError(st, "fljsd_lp_backward")
    return st


def fljsd_logits_lp_workspace_bytes(rows: int, v: int, top_k: int) -> int:
    return lib.fljsd_logits_lp_workspace_bytes(rows, v, top_k)


def fljsd_logits_lp(rows, v, ld, dtype, top_k, temperature, ignore_index, logits, labels, logp,
                    entropy, lse, norm, top_logp, top_id, workspace, workspace_bytes=None, stream=None,
                    check=True) -> int:
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    st = lib.fljsd_logits_lp(rows, v, ld, _dt(dtype), top_k, temperature, ignore_index,
                             _ptr(logits), _ptr(labels), _ptr(logp), _ptr(entropy), _ptr(lse), _ptr(norm),
                             _ptr(top_logp), _ptr(top_id), _ptr(workspace), workspace_bytes,
                             _stream(stream))
    if check and st != FLJSD_OK:
        raise FljsdError(st, "fljsd_logits_lp")
    return st


def fljsd_logits_lp_backward(rows, v, ld, ld_grad, dtype, temperature, ignore_index, logits,
                             labels, logp, entropy, norm, grad_logp, grad_entropy, grad_logits,
                             stream=None, check=True) -> int:
    st = lib.fljsd_logits_lp_backward(rows, v, ld, ld_grad, _dt(dtype), temperature, ignore_index,
                                      _ptr(logits), _ptr(labels), _ptr(logp), _ptr(entropy),
                                      _ptr(norm), _ptr(grad_logp), _ptr(grad_entropy),
                                      _ptr(grad_logits), _stream(stream))
    if check and st != FLJSD_OK:
        raise FljsdError(st, "fljsd_logits_lp_backward")
    return st


def make_adamw_options(lr, beta1, beta2, eps, weight_decay, step, param_dtype="bf16",
                       grad_dtype="bf16", state_bits=32, master=0) -> fljsd_adamw_options:
    return fljsd_adamw_options(lr, beta1, beta2, eps, weight_decay, step, _dt(param_dtype),
                               _dt(grad_dtype), state_bits, master)


def fljsd_adamw_step(options, tensors, count, grad_scale=None, stream=None, check=True) -> int:
    """``tensors``: address of ``count`` fljsd_adamw_tensor in host memory."""
    st = lib.fljsd_adamw_step(ctypes.byref(options), tensors, count, _ptr(grad_scale),
                              _stream(stream))
    if check and st != FLJSD_OK:
        raise FljsdError(st, "fljsd_adamw_step")
    return st


def fljsd_adamw_step_each(options, tensors, steps, count, grad_scale=None, stream=None,
                          check=True) -> int:
    """``tensors``, ``steps``: addresses of ``count`` fljsd_adamw_tensor and int64 in host
    memory."""
    st = lib.fljsd_adamw_step_each(ctypes.byref(options), tensors, steps, count, _ptr(grad_scale),
                                   _stream(stream))
    if check and st != FLJSD_OK:
        raise FljsdError(st, "fljsd_adamw_step_each")
    return st


def fljsd_grad_norm_workspace_bytes(count: int) -> int:
    return lib.fljsd_grad_norm_workspace_bytes(count)


def fljsd_grad_norm(tensors, count, kind, max_norm, grad_scale, norm, factor, workspace,
                    workspace_bytes=None, stream=None, check=True) -> int:
    """``tensors``: address of ``count`` fljsd_grad_tensor in host memory."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    st = lib.fljsd_grad_norm(tensors, count, kind, max_norm, _ptr(grad_scale), _ptr(norm),
                             _ptr(factor), _ptr(workspace), workspace_bytes, _stream(stream))
    if check and st != FLJSD_OK:
        raise FljsdError(st, "fljsd_grad_norm")
    return st


def fljsd_clip_grads(tensors, count, kind, max_norm, norm, workspace, workspace_bytes=None,
                     stream=None, check=True) -> int:
    """``tensors``: address of ``count`` fljsd_grad_tensor in host memory."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    st = lib.fljsd_clip_grads(tensors, count, kind, max_norm, _ptr(norm), _ptr(workspace),
                              workspace_bytes, _stream(stream))
    if check and st != FLJSD_OK:
        raise FljsdError(st, "fljsd_clip_grads")
    return st


def call(name, *args) -> None:
    """The C entry point with addresses as they are, on the current stream: for calls that are
    bound by the host, where converting a dozen arguments counts."""
    st = getattr(lib, name)(*args, _stream(None))
    if st != FLJSD_OK:
        raise FljsdError(st, name)


def fljsd_verify_workspace_bytes(requests: int, drafts: int) -> int:
    return lib.fljsd_verify_workspace_bytes(requests, drafts)


def fljsd_verify(requests, drafts, v, max_drafts, dtype, target, ld_target, draft, ld_draft, tokens,
                 u_accept, u_draw, offsets, temperatures, temperature, out, accepted, accept_prob,
                 workspace, workspace_bytes=None, stream=None, check=True) -> int:
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    st = lib.fljsd_verify(requests, drafts, v, max_drafts, _dt(dtype), _ptr(target), ld_target,
                          _ptr(draft), ld_draft, _ptr(tokens), _ptr(u_accept), _ptr(u_draw),
                          _ptr(offsets), _ptr(temperatures), temperature, _ptr(out), _ptr(accepted),
                          _ptr(accept_prob), _ptr(workspace), workspace_bytes, _stream(stream))
    if check and st != FLJSD_OK:
        raise FljsdError(st, "fljsd_verify")
    return st


def fljsd_low_rank_workspace_bytes(tokens: int, adapters: int, rank: int) -> int:
    return lib.fljsd_low_rank_workspace_bytes(tokens, adapters, rank)


def fljsd_low_rank_add(tokens, k, n, rank, adapters, x, ldx, a, b, index, scales, dtype, y, ldy, out, ldo,
                       workspace, workspace_bytes=None, stream=None, check=True) -> int:
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    st = lib.fljsd_low_rank_add(tokens, k, n, rank, adapters, _ptr(x), ldx, _ptr(a), _ptr(b), _ptr(index),
                                _ptr(scales), _dt(dtype), _ptr(y), ldy, _ptr(out), ldo, _ptr(workspace),
                                workspace_bytes, _stream(stream))
    if check and st != FLJSD_OK:
        raise FljsdError(st, "fljsd_low_rank_add")
    return st


def fljsd_fp8_quantize(rows, cols, dtype, block_rows, x, ldx, codes, ldq, scales, stream=None,
                       check=True) -> int:
    st = lib.fljsd_fp8_quantize(rows, cols, _dt(dtype), block_rows, _ptr(x), ldx, _ptr(codes), ldq,
                                _ptr(scales), _stream(stream))
    if check and st != FLJSD_OK:
        raise FljsdError(st, "fljsd_fp8_quantize")
    return st


def fljsd_fp8_linear_workspace_bytes(m: int, k: int) -> int:
    return lib.fljsd_fp8_linear_workspace_bytes(m, k)


def fljsd_fp8_linear(m, n, k, x_dtype, x, ldx, w_codes, ldw, w_scales, out_dtype, out, ldo,
                     workspace, workspace_bytes=None, stream=None, check=True) -> int:
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    st = lib.fljsd_fp8_linear(m, n, k, _dt(x_dtype), _ptr(x), ldx, _ptr(w_codes), ldw,
                              _ptr(w_scales), _dt(out_dtype), _ptr(out), ldo, _ptr(workspace),
                              workspace_bytes, _stream(stream))
    if check and st != FLJSD_OK:
        raise FljsdError(st, "fljsd_fp8_linear")
    return st


def fljsd_capture_id(stream=None) -> int:
    return lib.fljsd_capture_id(_stream(stream))


FLJSD_STALL_VERIFY, FLJSD_STALL_LOW_RANK_FIRST, FLJSD_STALL_LOW_RANK_SECOND, FLJSD_STALL_LOW_RANK_Y = 1, 2, 4, 8


def fljsd_test_stall(kernels: int) -> None:
    lib.fljsd_test_stall(kernels)


def fljsd_launch_count() -> int:
    return lib.fljsd_launch_count()


def fljsd_launch_count_reset() -> None:
    lib.fljsd_launch_count_reset()


def fljsd_trace_enable(max_launches: int) -> None:
    st = lib.fljsd_trace_enable(max_launches)
    if st != FLJSD_OK:
        raise FljsdError(st, "fljsd_trace_enable")


def fljsd_trace_reset() -> None:
    lib.fljsd_trace_reset()


def fljsd_trace_read(kind) -> tuple[float, int]:
    k = KERNEL_KINDS[kind] if isinstance(kind, str) else kind
    ms = ctypes.c_double()
    n = ctypes.c_int64()
    st = lib.fljsd_trace_read(k, ctypes.byref(ms), ctypes.byref(n))
    if st != FLJSD_OK:
        raise FljsdError(st, "fljsd_trace_read")
    return ms.value, n.value
