"""GB300 (sm_103a) fused-linear Jensen-Shannon distillation loss.

The compute path is libfljsd.so (CUDA kernels behind the C ABI declared in
include/fljsd.h). This package is its binding: ``_lib`` mirrors the C entry
points by name, ``api`` adds torch allocation and an autograd Function.
"""
from ._lib import (  # noqa: F401
    FljsdError,
    fljsd_backward,
    fljsd_ce_forward,
    fljsd_ce_plan,
    make_ce_problem,
    fljsd_forward,
    fljsd_forward_noalloc,
    fljsd_gemm_bf16,
    fljsd_jsd_logspace,
    fljsd_rows_workspace_bytes,
    fljsd_scale,
    fljsd_tvd,
    fljsd_adamw_step,
    fljsd_adamw_step_each,
    fljsd_fp8_linear,
    fljsd_fp8_linear_workspace_bytes,
    fljsd_fp8_quantize,
    fljsd_capture_id,
    fljsd_launch_count,
    fljsd_logits_lp,
    fljsd_logits_lp_backward,
    fljsd_logits_lp_workspace_bytes,
    fljsd_lp_backward,
    fljsd_lp_forward,
    fljsd_lp_plan,
    make_adamw_options,
    make_lp_problem,
    fljsd_launch_count_reset,
    fljsd_plan,
    fljsd_status_string,
    fljsd_trace_enable,
    fljsd_trace_read,
    fljsd_trace_reset,
    fljsd_workspace_status,
    make_problem,
)
from .api import (  # noqa: F401
    FusedLinearCrossEntropy,
    FusedLinearJSD,
    fused_linear_cross_entropy,
    fused_linear_jsd,
    jsd_logspace,
    tvd,
)
from .fp8 import fp8_linear, fp8_quantize  # noqa: F401
from .logprobs import (  # noqa: F401
    FusedLinearLogprobs,
    Logprobs,
    fused_linear_logprobs,
    logits_logprobs,
    logits_logprobs_backward,
    token_logprobs,
)
from .optim import AdamW  # noqa: F401

LIB_PATH = _lib.LIB_PATH
