/*
 * fljsd.h -- C ABI of the GB300 (sm_103a) fused-linear Jensen-Shannon
 * distillation loss.
 *
 * What the library computes (Liger-Kernel pull requests, cited by title):
 *
 *  - "[Perf] Fuse log-softmax into fused_linear_jsd kernel" (PR 1352),
 *    "Summary" and "Details": for a chunk of C rows, the student logits
 *    Z_s = X_s . W_s^T and the teacher logits Z_t = X_t . W_t^T are formed in
 *    the input dtype; the temperature-scaled log-softmaxes of both come from a
 *    three-pass online softmax over V (pass 1: running max m and denominator d
 *    for student and teacher together; pass 2: per-row loss and the
 *    cross-column term dX_sum; pass 3: the logit gradient dZ written in place
 *    over the student logits buffer). All math after the GEMM is fp32.
 *  - Same page, "Testing Done": beta == 0 is forward KL(P||Q), beta == 1 is
 *    reverse KL(Q||P), anything between is the generalized JSD
 *    beta*KL(P||M) + (1-beta)*KL(Q||M), M = beta*P + (1-beta)*Q, with P the
 *    teacher and Q the student distribution.
 *  - Same page, "Open questions" 2: the temperature divides the logits once.
 *  - "Fix TVD gradient at p == q" (PR 1374), "Summary": an element where the
 *    student and teacher log-probabilities tie contributes exactly zero.
 *  - "perf(flce): write the weight-gradient product directly into
 *    grad_weight" (PR 1429), "Summary" and "Changes": grad_input = dZ . W_s per
 *    chunk and grad_weight = sum over chunks of dZ^T . X_s, written straight
 *    into grad_weight; the first chunk overwrites (beta = 0), later chunks add
 *    the fp32 product to the stored value and round once; the outputs may be
 *    uninitialised (empty_like) because every element is written.
 *
 * Conventions for every entry point:
 *  - Matrices are dense, row-major, contiguous. Element type is given by
 *    fljsd_problem.dtype for X_s, W_s, X_t, W_t, grad_input and grad_weight.
 *  - Device pointers are caller-owned; the library allocates and frees no
 *    device memory. Every device pointer must be 16-byte aligned.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL is the legacy
 *    default stream). Argument checks are synchronous: on any error status
 *    nothing has been launched, except FLJSD_ERR_CUDA, which reports a launch
 *    failure after earlier launches of the same call may have been queued.
 *  - Not re-entrant across threads for the same workspace; distinct
 *    workspaces on distinct streams may run concurrently.
 */
#ifndef FLJSD_H
#define FLJSD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A cudaStream_t without pulling in the CUDA headers. */
typedef struct CUstream_st* fljsd_stream_t;

typedef enum {
  FLJSD_OK = 0,
  FLJSD_ERR_INVALID_ARG = 1, /* null pointer, bad size, beta or temperature, misalignment */
  FLJSD_ERR_UNSUPPORTED = 2, /* valid but beyond the kernels' size limits (stated per call) */
  FLJSD_ERR_WORKSPACE = 3,   /* workspace smaller than the plan requires */
  FLJSD_ERR_CUDA = 4,        /* a CUDA runtime call or kernel launch failed */
  FLJSD_ERR_TIMEOUT = 5      /* a bounded device-side wait expired */
} fljsd_status;

typedef enum { FLJSD_F32 = 0, FLJSD_BF16 = 1 } fljsd_dtype;

/* Reductions. The pages name four (PR 1374, "Details") and fix "batchmean"
 * as division by the number of rows (PR 1374, tie table). n = number of rows
 * whose label != ignore_index (BT when labels is NULL).
 *   NONE:      loss[r] = L_r (0 for ignored rows); gradients are those of
 *              sum_r row_grad[r] * L_r (row_grad NULL means all ones).
 *   SUM:       loss = sum_r L_r.
 *   MEAN:      loss = sum_r L_r / (n * V).
 *   BATCHMEAN: loss = sum_r L_r / n.
 * With n == 0 the loss and both gradients are 0. */
typedef enum {
  FLJSD_RED_NONE = 0,
  FLJSD_RED_SUM = 1,
  FLJSD_RED_MEAN = 2,
  FLJSD_RED_BATCHMEAN = 3
} fljsd_reduction;

typedef struct {
  int64_t bt;           /* rows (batch * sequence) */
  int64_t h_s;          /* student hidden size */
  int64_t h_t;          /* teacher hidden size */
  int64_t v;            /* vocabulary size */
  int32_t dtype;        /* fljsd_dtype of X_s, W_s, X_t, W_t and the gradients */
  int32_t reduction;    /* fljsd_reduction */
  float beta;           /* in [0, 1]; 0 and 1 select the KL endpoints exactly */
  float temperature;    /* > 0 and finite; logits are divided by it once */
  int64_t ignore_index; /* label value of rows that are skipped (Liger: -100) */
  int64_t chunk_rows;   /* rows per chunk; 0 lets fljsd_plan choose */
  int32_t flags;        /* FLJSD_FLAG_* bits, 0 for the pages' behaviour */
  int32_t reserved;     /* must be 0 */
} fljsd_problem;

/* Opt-in behaviours (none of them is the pages' default).
 * FLJSD_FLAG_T2: multiply the loss and both gradients by T^2 (Hinton et al.
 *   2015); the pages divide by T once and leave this to the caller
 *   ("[Perf] Fuse log-softmax into fused_linear_jsd kernel", Open questions 2).
 * FLJSD_FLAG_ACCUM_FP32: with bf16 inputs and more than one chunk, accumulate
 *   grad_weight across chunks in an fp32 buffer inside the workspace
 *   (V * h_s * 4 bytes) and round it to bf16 once after the last chunk, as
 *   the accum_dtype=float32 option of "perf(flce): write the weight-gradient
 *   product directly into grad_weight" (PR 1429) does; without it every chunk
 *   after the first rounds the running sum to bf16. */
#define FLJSD_FLAG_T2 1
#define FLJSD_FLAG_ACCUM_FP32 2

typedef struct {
  int64_t chunk_rows;     /* C: rows of one chunk */
  int64_t num_chunks;     /* ceil(bt / C) */
  int64_t ld;             /* row stride (elements) of the logits buffers, >= v */
  size_t workspace_bytes; /* device bytes fljsd_forward needs */
  size_t logits_bytes;    /* 2 * C * ld * sizeof(dtype): the two logits buffers */
  size_t stats_bytes;     /* per-row and per-tile statistics */
  size_t status_offset;   /* byte offset of the int32 device status word in the workspace */
} fljsd_plan_t;

/*
 * fljsd_plan -- choose the chunk geometry and size the workspace.
 *
 * If problem->chunk_rows > 0 it is used (clamped to bt). Otherwise the largest
 * chunk whose workspace fits in half of `free_hbm_bytes` is taken (a multiple
 * of 128 rows unless it is all of bt); free_hbm_bytes == 0 means "no limit",
 * i.e. one chunk. The pages found one chunk fastest and the fixed
 * cdiv(V, H) heuristic mis-tuned for JSD (PR 1352, "Open questions" 4); live
 * memory per chunk is the two logits tensors, 2 * C * V * s bytes (PR 1352,
 * "Details", memory table), plus O(C) statistics and the (BT,) loss vector.
 * Host only; launches nothing. Returns FLJSD_ERR_INVALID_ARG for a bad
 * problem, FLJSD_ERR_UNSUPPORTED for shapes the kernels do not handle (bt or
 * v above 2^30, h_s or h_t above 2^20), and FLJSD_ERR_WORKSPACE if not even
 * one row fits.
 */
fljsd_status fljsd_plan(const fljsd_problem* problem, size_t free_hbm_bytes,
                        fljsd_plan_t* out);

/*
 * fljsd_forward -- loss and both gradients (upstream gradient 1).
 *
 *   x_s [bt x h_s], w_s [v x h_s], x_t [bt x h_t], w_t [v x h_t]: inputs
 *       (device, dtype; never modified). The teacher is frozen: no teacher
 *       gradient is produced.
 *   labels [bt] int64 (device) or NULL: rows with label == ignore_index are
 *       skipped.
 *   row_grad [bt] fp32 (device) or NULL: upstream per-row gradient, used only
 *       with FLJSD_RED_NONE (NULL = ones).
 *   loss (device fp32): [1] for SUM, MEAN, BATCHMEAN; [bt] for NONE.
 *   grad_input [bt x h_s] (device, dtype): d loss / d x_s.
 *   grad_weight [v x h_s] (device, dtype): d loss / d w_s.
 *   workspace (device), workspace_bytes >= plan->workspace_bytes.
 *
 * Every element of loss, grad_input and grad_weight is written. `plan` must
 * come from fljsd_plan for the same problem.
 */
fljsd_status fljsd_forward(const fljsd_problem* problem, const fljsd_plan_t* plan,
                           const void* x_s, const void* w_s, const void* x_t,
                           const void* w_t, const int64_t* labels, const float* row_grad,
                           float* loss, void* grad_input, void* grad_weight,
                           void* workspace, size_t workspace_bytes, fljsd_stream_t stream);

/*
 * fljsd_forward_noalloc -- fljsd_forward for callers that cannot allocate
 * device memory (e.g. a plugin inside a host framework that owns every
 * device allocation and passes in only input and output buffers). The pages
 * have no counterpart of this entry point; it is an addition of this library.
 *
 * Arguments are those of fljsd_forward without plan and workspace: the
 * scratch lives in a fixed 64 MiB device array inside the library, which
 * every GPU that loads the library holds until the process exits.
 *   - The chunk rows are chosen to fit that array (problem->chunk_rows, if
 *     > 0, must fit it). A problem whose scratch does not fit even one row
 *     (2 * ceil8(v) * sizeof(dtype) bytes per row, plus 4 * bt bytes) returns
 *     FLJSD_ERR_WORKSPACE before anything is launched.
 *   - Every call shares the one array: calls whose work overlaps on the GPU
 *     (different streams, different host threads) race; serialise them.
 *     Nothing in the array has to start at zero: a call writes every byte it
 *     reads, so what the previous call left there does not matter.
 *   - The first call on a device (the current device) looks up the array's
 *     device address with the CUDA runtime and caches it; make that first
 *     call before any stream capture. It calls no cudaMalloc or cudaFree.
 * Returns what fljsd_forward returns, and FLJSD_ERR_CUDA if the address
 * lookup fails.
 */
fljsd_status fljsd_forward_noalloc(const fljsd_problem* problem, const void* x_s,
                                   const void* w_s, const void* x_t, const void* w_t,
                                   const int64_t* labels, const float* row_grad, float* loss,
                                   void* grad_input, void* grad_weight, fljsd_stream_t stream);

/*
 * fljsd_backward -- scale the gradients computed by fljsd_forward by the
 * upstream scalar gradient *grad_output (device fp32), in place, on `stream`.
 * The forward already holds the gradients for an upstream gradient of 1
 * (PR 1352, "Details": the gradient is written during the forward pass), so
 * this is one elementwise pass over grad_input [bt x h_s] and grad_weight
 * [v x h_s] that does nothing when *grad_output == 1.
 */
fljsd_status fljsd_backward(const fljsd_problem* problem, const float* grad_output,
                            void* grad_input, void* grad_weight, fljsd_stream_t stream);

/*
 * fljsd_workspace_status -- the device status word of the last fljsd_forward
 * that used `workspace` (FLJSD_OK, or FLJSD_ERR_TIMEOUT if a bounded wait
 * inside a kernel expired). Synchronises `stream`, then copies 4 bytes to
 * the host into *device_status. Returns FLJSD_ERR_CUDA if the copy fails.
 */
fljsd_status fljsd_workspace_status(const fljsd_plan_t* plan, const void* workspace,
                                    fljsd_stream_t stream, int32_t* device_status);

/*
 * fljsd_gemm_bf16 -- the tensor-core contraction used by the path, exposed
 * as a building block: D[m x n] = A . B^T (accumulate == 0) or
 * D = D + A . B^T (accumulate == 1; the stored value and the fp32 product
 * are added and rounded once, as for grad_weight in PR 1429, "Summary").
 *   a_mn == 0: A stored [m x k] row-major with row stride lda (k contiguous);
 *   a_mn == 1: A stored [k x m] row-major with row stride lda (m contiguous);
 *   b_mn == 0: B stored [n x k]; b_mn == 1: B stored [k x n] (stride ldb);
 *   D stored [m x ldd]. All bf16, device, 16-byte aligned; lda, ldb, ldd
 *   multiples of 8; m, n, k >= 1.
 * status: device int32 that receives FLJSD_ERR_TIMEOUT if a bounded wait
 * expires (may be NULL). flags: 0, FLJSD_GEMM_SINGLE_CTA or
 * FLJSD_GEMM_TEST_STALL (below).
 * Asynchronous on `stream`. FLJSD_ERR_INVALID_ARG for
 * shapes or alignments outside the above.
 */
fljsd_status fljsd_gemm_bf16(const void* a, int64_t lda, int32_t a_mn, const void* b,
                             int64_t ldb, int32_t b_mn, void* d, int64_t ldd, int64_t m,
                             int64_t n, int64_t k, int32_t accumulate, int32_t* status,
                             int32_t flags, fljsd_stream_t stream);
/* flags of fljsd_gemm_bf16: by default, for contractions at least 256 deep,
 * pairs of 128-row blocks of D run as CTA pairs (2-CTA clusters,
 * tcgen05.mma.cta_group::2) that compute a 256 x 256 tile together, each CTA
 * copying only its own rows of A and half of the B tile, unless the pairs
 * would need more than 12% more waves of tiles over the GPU than one CTA per
 * tile (an odd block count leaves a pair half empty; few tiles can add a
 * wave);
 * FLJSD_GEMM_SINGLE_CTA runs one CTA per 128 x 256 tile. The results are
 * identical. The environment variable FLJSD_GEMM_PAIR (read at each launch)
 * selects for every GEMM of the library: 0 one CTA per tile, 2 CTA pairs at
 * any contraction depth. */
#define FLJSD_GEMM_SINGLE_CTA 1
/* Test of the failure path: the kernel's copy warp issues nothing, so its
 * first bounded wait expires after 50 ms; *status then holds
 * FLJSD_ERR_TIMEOUT, D is not written, and the context stays usable. */
#define FLJSD_GEMM_TEST_STALL 2

/*
 * Distances over given distributions (no GEMM). Both take [rows x v] row-major
 * tensors of `dtype`, optional int64 labels [rows] (rows whose label equals
 * ignore_index give loss 0 and gradient 0; n = the other rows), a reduction
 * as for fljsd_forward (none / sum / mean = / (n v) / batchmean = / n), and a
 * device workspace of fljsd_rows_workspace_bytes(rows) bytes. They return the
 * gradient for an upstream gradient of 1 (fljsd_scale applies another).
 *
 * fljsd_jsd_logspace -- the generalized JSD on log-probabilities, the public
 * contract of Liger's _jsd_kernel ("[Perf] Fuse log-softmax into
 * fused_linear_jsd kernel", PR 1352, Open questions 3): input = X = log Q
 * (student), target = Y = log P (teacher); per element beta*P*(Y - log M) +
 * (1-beta)*Q*(X - log M) with M = beta*P + (1-beta)*Q, forward KL P*(Y - X) at
 * beta == 0, reverse KL Q*(X - Y) at beta == 1; ties (X == Y) contribute 0.
 * grad_input = d loss / d X element by element (inputs are not renormalised,
 * so no softmax Jacobian): (1-beta)*Q*(X - log M), -P at beta == 0,
 * Q*(X - Y + 1) at beta == 1, times the reduction weight. loss: [1], or [rows]
 * for reduction none.
 *
 * fljsd_tvd -- total variation distance with the tie fix of "Fix TVD
 * gradient at p == q" (PR 1374, Summary): per element 0.5*|p - q|, gradient
 * in p = 0.5 * sign(p - q) * (reduction weight) with sign(0) = 0. loss: [1],
 * or [rows x v] fp32 per element for reduction none.
 *
 * fljsd_scale -- x *= *grad_output in place (device fp32 scalar), skipped on
 * the device when it is 1: the backward of the two functions above.
 *
 * Errors (checked on the host before anything is launched):
 * FLJSD_ERR_INVALID_ARG for rows or v <= 0, an unknown dtype or reduction, beta
 * outside [0, 1], a null input, target, loss, gradient or workspace pointer, or
 * one not 16-byte aligned (loss: 4 bytes; labels, when given: 16 bytes);
 * FLJSD_ERR_UNSUPPORTED for rows or v above 2^31; FLJSD_ERR_WORKSPACE for a
 * workspace below fljsd_rows_workspace_bytes(rows); FLJSD_ERR_CUDA when a
 * launch fails. fljsd_scale: FLJSD_ERR_INVALID_ARG for an unknown dtype, n < 0,
 * or a null or unaligned pointer.
 */
size_t fljsd_rows_workspace_bytes(int64_t rows);
fljsd_status fljsd_jsd_logspace(int64_t rows, int64_t v, int32_t dtype, float beta,
                                int32_t reduction, int64_t ignore_index, const void* input,
                                const void* target, const int64_t* labels, float* loss,
                                void* grad_input, void* workspace, size_t workspace_bytes,
                                fljsd_stream_t stream);
fljsd_status fljsd_tvd(int64_t rows, int64_t v, int32_t dtype, int32_t reduction,
                       int64_t ignore_index, const void* p, const void* q, const int64_t* labels,
                       float* loss, void* grad_p, void* workspace, size_t workspace_bytes,
                       fljsd_stream_t stream);
fljsd_status fljsd_scale(int32_t dtype, void* x, int64_t n, const float* grad_output,
                         fljsd_stream_t stream);

/*
 * Fused linear cross-entropy (FLCE): loss = CE(x . w^T, labels) and its
 * gradients in x and w, on the same GEMMs, chunk planner and grad_weight
 * contract as fljsd_forward ("perf(flce): write the weight-gradient product
 * directly into grad_weight", PR 1429: first chunk overwrites, later chunks add
 * in fp32 and round once, or accumulate in fp32 with FLJSD_FLAG_ACCUM_FP32).
 * Per row with label y and logits z (c = softcap * tanh(z / softcap) when
 * softcap > 0, else c = z), lse = log sum_j e^{c_j}:
 *   L = lse - (1 - eps) c_y - (eps / V) sum_j c_j + lse_square_scale * lse^2
 * (eps = label_smoothing). Reductions: none -> [bt] per-row losses; sum;
 * mean and batchmean -> divided by the number of rows whose label is not
 * ignore_index. Labels are required (int64 [bt], device); a label outside
 * [0, v) that is not ignore_index makes its row contribute 0 and sets the
 * workspace status word to FLJSD_ERR_INVALID_ARG (fljsd_workspace_status).
 * x [bt x h], w [v x h], grad_input [bt x h], grad_weight [v x h] in dtype.
 * Gradients are for an upstream gradient of 1 (fljsd_scale applies another).
 *
 * fljsd_ce_plan / fljsd_ce_forward follow fljsd_plan / fljsd_forward: every
 * pointer is caller-owned device memory, 16-byte aligned (loss 4 bytes);
 * grad_input and grad_weight are written in full and may be uninitialised; the
 * workspace (plan->workspace_bytes, device, caller-owned) holds the logits of
 * one chunk and the per-row statistics; the forward is asynchronous on
 * `stream`. Errors, checked on the host before anything is launched:
 * FLJSD_ERR_INVALID_ARG for a dimension <= 0, an unknown dtype, reduction or
 * flag, label_smoothing outside [0, 1], a negative or non-finite
 * lse_square_scale or softcap, or a null or unaligned pointer;
 * FLJSD_ERR_UNSUPPORTED for bt or v above 2^30 or h above 2^20;
 * FLJSD_ERR_WORKSPACE when the workspace is smaller than the plan's (or, in
 * fljsd_ce_plan, when not even one row fits the budget); FLJSD_ERR_CUDA when a
 * launch fails.
 */
typedef struct {
  int64_t bt, h, v;
  int32_t dtype;          /* fljsd_dtype */
  int32_t reduction;      /* fljsd_reduction */
  int64_t ignore_index;
  int64_t chunk_rows;     /* 0 lets fljsd_ce_plan choose */
  float label_smoothing;  /* in [0, 1] */
  float lse_square_scale; /* z-loss coefficient, >= 0 */
  float softcap;          /* 0 disables the tanh cap */
  int32_t flags;          /* FLJSD_FLAG_ACCUM_FP32 or 0 */
} fljsd_ce_problem;

fljsd_status fljsd_ce_plan(const fljsd_ce_problem* problem, size_t free_hbm_bytes,
                           fljsd_plan_t* out);
fljsd_status fljsd_ce_forward(const fljsd_ce_problem* problem, const fljsd_plan_t* plan,
                              const void* x, const void* w, const int64_t* labels, float* loss,
                              void* grad_input, void* grad_weight, void* workspace,
                              size_t workspace_bytes, fljsd_stream_t stream);

/*
 * Token log probabilities: for every row of logits z (z = x . w^T of hidden
 * states and an lm_head weight, or given logits), with s = z / temperature and
 * p = softmax(s):
 *   lse = log sum_j e^{s_j},  logp = s_y - lse,  entropy = -sum_j p_j log p_j,
 *   the top_k largest logits as (column, log probability), in descending order,
 *   equal logits by the lower column.
 * Upstream gradients a (grad_logp) and b (grad_entropy), [bt] fp32 each, give
 *   dz_j = (a (1[j = y] - p_j) - b p_j (log p_j + entropy)) / temperature,
 *   grad_input = dz . w,  grad_weight = dz^T . x.
 * All of it is computed in fp32 from unrounded logits; the top alternatives carry
 * no gradient. The fused form returns no logits; its workspace holds, for each row of a
 * chunk, the alternatives' candidates (about v top_k / 16 bytes: with top_k 32 what bf16
 * logits take) and with FLJSD_LP_BACKWARD the kept values (2 v bytes); fp32 logits (4 v
 * bytes) of up to 16 rows with alternatives, and of what runs on the CUDA cores.
 *
 * Rows and values outside the ordinary:
 *  - a row whose label is ignore_index, or outside [0, v), has logp 0, entropy 0
 *    and gradient 0; its lse and alternatives are written all the same. A label
 *    outside [0, v) other than ignore_index also sets the status word to
 *    FLJSD_ERR_INVALID_ARG (fljsd_workspace_status; fljsd_logits_lp: the first
 *    int32 of the workspace).
 *  - a logit of -inf (a masked token) has probability 0 and is no alternative:
 *    where fewer than top_k remain, the rest is column -1 with -inf. A row of
 *    nothing else has lse -inf, logp -inf, entropy 0 and gradient 0.
 *  - a logit of NaN or +inf makes the row's lse, logp and entropy NaN; NaN is no
 *    alternative.
 *
 * fljsd_lp_plan / fljsd_lp_forward / fljsd_lp_backward follow fljsd_plan and
 * fljsd_forward: caller-owned device memory, asynchronous on `stream`, errors
 * found on the host before anything is launched. x [bt x h] and w [v x h] in
 * dtype, 16-byte aligned; labels [bt] int64 or NULL (then no logp); logp,
 * entropy, lse [bt] fp32; norm [bt x 2] fp32, for the backward pass (the row's
 * largest logit and log2 of the sum of e^{s_j} relative to it); top_logp
 * [bt x top_k] fp32 and top_id [bt x top_k] int64 (NULL with top_k 0). bf16 with h
 * a multiple of 8 runs on the tensor cores, everything else on the CUDA cores.
 *
 * FLJSD_LP_BACKWARD sizes the workspace for fljsd_lp_backward, and lets the
 * forward of a one-chunk plan leave there what the backward would otherwise
 * compute again: pass kept = 1 when the workspace is as the forward of the same
 * problem and inputs left it (a backward pass uses it up, at each replay where it
 * was captured), kept = 0 to compute it again. logp, entropy and norm are the
 * forward's results; grad_logp (needs labels) and grad_entropy may be NULL (zero).
 * grad_input and grad_weight are written in full, as by fljsd_forward; one of them
 * may be NULL and is left out.
 *
 * fljsd_logits_lp / fljsd_logits_lp_backward are the same of given logits
 * [rows x v] in dtype with row stride ld (elements, any alignment) and of their
 * gradient, written in dtype with row stride ld_grad; it may overwrite the
 * logits (same address and stride).
 *
 * Errors: FLJSD_ERR_INVALID_ARG for a dimension <= 0, a stride below v, an
 * unknown dtype or flag, top_k outside [0, v], a temperature that is not
 * positive and finite (with a finite log2(e) / temperature), grad_logp without labels, a null or unaligned pointer, or
 * kept = 1 with more than one chunk; FLJSD_ERR_UNSUPPORTED for top_k above 32,
 * bt, rows or v above 2^30 or h above 2^20; FLJSD_ERR_WORKSPACE for a workspace
 * below the plan's (or, in fljsd_lp_plan, when not even one row fits the
 * budget); FLJSD_ERR_CUDA when a launch fails.
 */
typedef struct {
  int64_t bt, h, v;
  int32_t dtype;         /* fljsd_dtype */
  int32_t top_k;         /* alternatives of each row, 0..32 */
  int64_t ignore_index;
  int64_t chunk_rows;    /* 0 lets fljsd_lp_plan choose */
  float temperature;     /* > 0 and finite */
  int32_t flags;         /* FLJSD_LP_BACKWARD, FLJSD_FLAG_ACCUM_FP32 */
} fljsd_lp_problem;
#define FLJSD_LP_BACKWARD 4

fljsd_status fljsd_lp_plan(const fljsd_lp_problem* problem, size_t free_hbm_bytes,
                           fljsd_plan_t* out);
fljsd_status fljsd_lp_forward(const fljsd_lp_problem* problem, const fljsd_plan_t* plan,
                              const void* x, const void* w, const int64_t* labels, float* logp,
                              float* entropy, float* lse, float* norm, float* top_logp, int64_t* top_id,
                              void* workspace, size_t workspace_bytes, fljsd_stream_t stream);
fljsd_status fljsd_lp_backward(const fljsd_lp_problem* problem, const fljsd_plan_t* plan,
                               const void* x, const void* w, const int64_t* labels,
                               const float* logp, const float* entropy, const float* norm,
                               const float* grad_logp, const float* grad_entropy, int32_t kept,
                               void* grad_input, void* grad_weight, void* workspace,
                               size_t workspace_bytes, fljsd_stream_t stream);
size_t fljsd_logits_lp_workspace_bytes(int64_t rows, int64_t v, int32_t top_k);
fljsd_status fljsd_logits_lp(int64_t rows, int64_t v, int64_t ld, int32_t dtype, int32_t top_k,
                             float temperature, int64_t ignore_index, const void* logits,
                             const int64_t* labels, float* logp, float* entropy, float* lse, float* norm,
                             float* top_logp, int64_t* top_id, void* workspace,
                             size_t workspace_bytes, fljsd_stream_t stream);
fljsd_status fljsd_logits_lp_backward(int64_t rows, int64_t v, int64_t ld, int64_t ld_grad,
                                      int32_t dtype, float temperature, int64_t ignore_index,
                                      const void* logits, const int64_t* labels,
                                      const float* logp, const float* entropy, const float* norm,
                                      const float* grad_logp, const float* grad_entropy,
                                      void* grad_logits, fljsd_stream_t stream);

/*
 * fljsd_adamw_step -- one AdamW step over `count` tensors, in place. Per element,
 * in fp32, each operation rounded once, t = options->step (the number of this
 * step, from 1, for all tensors of the call; fljsd_adamw_step_each: steps[i], host memory,
 * for tensor i):
 *   g = grad * grad_scale,  m = beta1 m + (1 - beta1) g,
 *   v = beta2 v + (1 - beta2) g^2,
 *   p = p (1 - lr weight_decay)
 *       - lr / (1 - beta1^t) m / (sqrt(v) / sqrt(1 - beta2^t) + eps).
 * param [n] in param_dtype, grad [n] in grad_dtype. With master = 1 (bf16 params)
 * the fp32 `master` [n] is what is stepped, and param receives it rounded.
 * state_bits 32: exp_avg and exp_avg_sq hold m and v, fp32 [n]. state_bits 8:
 * exp_avg and exp_avg_sq are e4m3 codes [n] of m and of sqrt(v), with one fp32
 * scale for every 128 consecutive elements ([ceil(n / 128)] each): value = code
 * * scale, scale = amax * (1 / 448) (amax of the block, not below 2^-100), code =
 * the nearest to value * (448 * (1 / amax)). States may start as zeros. There is no
 * floor under the codes: what is below about 2^-19 of its block's amax is held as 0,
 * and m and sqrt(v) have scales of their own, so that a sqrt(v) may be held as 0 whose
 * m is not. What that parameter's next step divides by is then its new gradient's part
 * of v and eps alone: choose eps so that lr m / eps is a step that may be taken.
 * grad_scale: device fp32 scalar or NULL (1), e.g. 1 / loss scale, or the factor
 * of a clipped gradient norm.
 * `tensors` is host memory, read before the call returns; the tensors' memory is
 * device memory, element-aligned (16 bytes, 8 for 8-bit states, is fastest), and
 * must not overlap. Tensors with n == 0 are left out (their pointers may be NULL).
 * Hyperparameters are taken at the call: a captured call repeats its step number.
 * Errors, found before anything is launched: FLJSD_ERR_INVALID_ARG for an unknown
 * dtype, state_bits other than 8 and 32, beta outside [0, 1), a negative or
 * non-finite eps, a non-finite lr or weight_decay, a step < 1, n < 0, a null or
 * misaligned pointer, master with fp32 params, a master pointer without master;
 * FLJSD_ERR_UNSUPPORTED for n above 2^40; FLJSD_ERR_CUDA when a launch fails.
 */
typedef struct {
  const void* grad;
  void* param;
  float* master;
  void* exp_avg;
  void* exp_avg_sq;
  float* exp_avg_scale;
  float* exp_avg_sq_scale;
  int64_t n;
} fljsd_adamw_tensor;

typedef struct {
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;        /* 1 for the first */
  int32_t param_dtype; /* fljsd_dtype */
  int32_t grad_dtype;
  int32_t state_bits;  /* 32 or 8 */
  int32_t master;      /* 0 or 1 */
} fljsd_adamw_options;

fljsd_status fljsd_adamw_step(const fljsd_adamw_options* options,
                              const fljsd_adamw_tensor* tensors, int32_t count,
                              const float* grad_scale, fljsd_stream_t stream);
fljsd_status fljsd_adamw_step_each(const fljsd_adamw_options* options,
                                   const fljsd_adamw_tensor* tensors, const int64_t* steps,
                                   int32_t count, const float* grad_scale,
                                   fljsd_stream_t stream);

/*
 * The norm of many tensors taken together, and clipping. Over the elements g of all
 * `count` tensors (fp32 and bf16 may be mixed):
 *   FLJSD_NORM_2: norm = sqrt(sum g^2); FLJSD_NORM_MAX: norm = max |g|;
 *   factor = min(1, max_norm / (norm + 1e-6)).
 * Sums are held in fp32 and joined in fp64, in one order: the same tensors have the same
 * norm in every call on a GPU. Every finite g counts, up to fp32's largest and down to its smallest; a norm
 * that fp32 does not hold is infinite. A NaN among the gradients makes the norm and the
 * factor NaN; an infinity makes the norm infinite and the factor 0. No tensors, or none
 * with elements: norm 0.
 *
 * fljsd_grad_norm -- the norm, and where factor is not NULL the factor (max_norm is not
 * looked at otherwise). grad_scale: device fp32 scalar or NULL (1) that every gradient
 * counts as multiplied by; the factor then includes it, so that it can be handed to
 * fljsd_adamw_step as its grad_scale. `out` is not looked at.
 *
 * fljsd_clip_grads -- the norm of `grad`, and out = grad * factor in the tensor's dtype,
 * rounded once. out may be the gradient itself (which is left as it is where the factor
 * is 1), but no other memory of the call's tensors.
 *
 * norm and factor: device fp32 scalars, 4-byte aligned. `tensors` is host memory, read
 * before the call returns; grad and out are element-aligned device memory (an out that
 * lies as its gradient does relative to 16 bytes is fastest). Tensors with n == 0 are
 * left out. workspace: fljsd_grad_norm_workspace_bytes(count) bytes, 16-byte aligned.
 * Errors, found before anything is launched: FLJSD_ERR_INVALID_ARG for an unknown dtype
 * or kind, n < 0, a null or misaligned pointer, a max_norm that is negative or NaN (where
 * it is looked at); FLJSD_ERR_UNSUPPORTED for n above 2^40; FLJSD_ERR_WORKSPACE;
 * FLJSD_ERR_CUDA when a launch fails.
 */
typedef enum { FLJSD_NORM_MAX = 0, FLJSD_NORM_2 = 2 } fljsd_norm_kind;

typedef struct {
  const void* grad;
  void* out;
  int64_t n;
  int32_t dtype; /* fljsd_dtype */
  int32_t reserved;
} fljsd_grad_tensor;

size_t fljsd_grad_norm_workspace_bytes(int32_t count);
fljsd_status fljsd_grad_norm(const fljsd_grad_tensor* tensors, int32_t count, int32_t kind,
                             float max_norm, const float* grad_scale, float* norm, float* factor,
                             void* workspace, size_t workspace_bytes, fljsd_stream_t stream);
fljsd_status fljsd_clip_grads(const fljsd_grad_tensor* tensors, int32_t count, int32_t kind,
                              float max_norm, float* norm, void* workspace, size_t workspace_bytes,
                              fljsd_stream_t stream);

/*
 * Product in 8-bit floating point with a scale for each block of 128, for a frozen
 * lm_head (a teacher's, or one that only scores): out = x . w^T with w [n x k]
 * held as e4m3 codes and one fp32 scale for each 128 x 128 block, and x [m x k]
 * quantised on the way with one scale for each 1 x 128. Sums inside a block are
 * exact products added in fp32, blocks are scaled and added in fp32, and the
 * result is rounded once to out_dtype.
 *
 * fljsd_fp8_quantize -- codes and scales of x [rows x cols] (dtype, row stride
 * ldx): per block of block_rows (1 or 128) x 128, amax = max |x|, not below
 * 2^-100; scale = amax * (1 / 448), code = the e4m3 nearest to x * (448 * (1 /
 * amax)). codes [rows x ldq], ldq a multiple of 16, 16-byte aligned (columns past
 * cols are written as zeros). scales: for 128 rows [ceil(rows / 128) x
 * ceil(cols / 128)], for one row [ceil(cols / 128) x rows]. A NaN keeps its place
 * (code NaN); an infinite amax makes its block NaN.
 *
 * fljsd_fp8_linear -- the product. x in x_dtype with row stride ldx; w_codes with
 * row stride ldw (a multiple of 16; 16-byte aligned), w_scales [ceil(n / 128) x
 * ceil(k / 128)]; out [m x n] in out_dtype with row stride ldo. workspace:
 * fljsd_fp8_linear_workspace_bytes(m, k) bytes, 16-byte aligned; its first int32
 * is a status word (FLJSD_ERR_TIMEOUT if a bounded device wait expired).
 *
 * Errors, found before anything is launched: FLJSD_ERR_INVALID_ARG for a dimension
 * <= 0, a stride below its row or not a multiple of 16 where one is asked for, an
 * unknown dtype, block_rows other than 1 and 128, a null or misaligned pointer;
 * FLJSD_ERR_UNSUPPORTED for m, n or rows above 2^30 or k or cols above 2^20;
 * FLJSD_ERR_WORKSPACE; FLJSD_ERR_CUDA when a launch fails.
 */
fljsd_status fljsd_fp8_quantize(int64_t rows, int64_t cols, int32_t dtype, int32_t block_rows,
                                const void* x, int64_t ldx, void* codes, int64_t ldq, float* scales,
                                fljsd_stream_t stream);
size_t fljsd_fp8_linear_workspace_bytes(int64_t m, int64_t k);
fljsd_status fljsd_fp8_linear(int64_t m, int64_t n, int64_t k, int32_t x_dtype, const void* x,
                              int64_t ldx, const void* w_codes, int64_t ldw, const float* w_scales,
                              int32_t out_dtype, void* out, int64_t ldo, void* workspace,
                              size_t workspace_bytes, fljsd_stream_t stream);

/*
 * fljsd_low_rank_add -- low-rank adapters of many requests on the output of a projection
 * that they share (serving; no gradient): for each of `tokens` rows, with a = index[t],
 *   out_t = y_t + scale_a B_a (A_a x_t);  a = -1: out_t = y_t.
 * a [adapters x rank x k] and b [adapters x n x rank] bf16, contiguous; scales [adapters]
 * fp32 or NULL (1); x [tokens x k] bf16 with row stride ldx; y and out [tokens x n] in
 * dtype with row strides ldy and ldo; out may be y (same address and stride; rows of
 * index -1 are then not touched), but no other memory of the call. The tokens' order is
 * free; those of one adapter need not be neighbours. The rank is a multiple of 8 (adapters
 * of smaller ranks are padded with zeros).
 * Products are added in fp32; A x, scaled, is carried on as the sum of two bf16 for y in
 * bf16 (2^-16 of it at most is lost) and of three for y in fp32 (2^-24); the result is added to y
 * in fp32 and rounded once to dtype. A row's result does not depend on the other rows.
 * An index that is neither -1 nor in [0, adapters) counts as -1 and sets the status word
 * (the workspace's first int32) to FLJSD_ERR_INVALID_ARG; FLJSD_ERR_TIMEOUT there: a
 * bounded device wait expired and out is not complete.
 * workspace: fljsd_low_rank_workspace_bytes(tokens, adapters, rank) bytes. b and the
 * workspace are 16-byte aligned, everything else element-aligned. (x and a are fastest on 16
 * bytes with ldx and k multiples of 8, y and out on 16 bytes with ldy, ldo and n multiples of 16
 * bytes: 8 bf16, 4 fp32. Other rows of y and out are added to one value at a time.)
 * Errors, found before anything is launched: FLJSD_ERR_INVALID_ARG for a dimension <= 0, a
 * stride below its row, a rank that is no multiple of 8, an unknown dtype, a null or
 * misaligned pointer, out at y's address with another stride; FLJSD_ERR_UNSUPPORTED for
 * tokens or k above 2^20, n above 2^26, rank above 128, adapters above 4096, adapters * n
 * of 2^31 and more;
 * FLJSD_ERR_WORKSPACE; FLJSD_ERR_CUDA when a launch fails.
 */
size_t fljsd_low_rank_workspace_bytes(int64_t tokens, int32_t adapters, int32_t rank);
fljsd_status fljsd_low_rank_add(int64_t tokens, int64_t k, int64_t n, int32_t rank, int32_t adapters,
                                const void* x, int64_t ldx, const void* a, const void* b,
                                const int64_t* index, const float* scales, int32_t dtype,
                                const void* y, int64_t ldy, void* out, int64_t ldo, void* workspace,
                                size_t workspace_bytes, fljsd_stream_t stream);

/*
 * fljsd_verify -- drafted tokens verified against a target's probabilities, from given
 * random numbers (speculative decoding). `requests` requests propose `drafts` tokens
 * together, request b tokens[offsets[b] .. offsets[b + 1]), at most max_drafts each;
 * offsets NULL: max_drafts each (drafts = requests * max_drafts). Row offsets[b] + b + i of
 * `target` [drafts + requests x v] holds the target's logits in front of its drafted token
 * i, the row after its last one those behind it; row offsets[b] + i of `draft` [drafts x v]
 * holds the logits that the token was drafted from (NULL: the tokens have no
 * probabilities, as those looked up in a prompt). With a temperature T for each request
 * (temperatures [requests], or `temperature` for all):
 *   p = softmax(target / T), q = softmax(draft / T), q = 1 at the drafted token without draft.
 * A request's tokens d are accepted in turn as long as u_accept q_d < p_d. The first that is
 * not gives way to a token drawn from max(p - q, 0) (from p where that is 0 everywhere);
 * where all are, one more is drawn from p. Drawn is the lowest column at which the running
 * sum of the weights exceeds u_draw [requests] times their sum. Over many random numbers,
 * uniform in [0, 1), the tokens follow p, whatever the drafts. T = 0: d is accepted where
 * it is the target's largest logit (of equal ones the lowest column), which is what is drawn.
 *   out [requests x (max_drafts + 1)]: the accepted tokens, the drawn one, -1 behind;
 *   accepted [requests]: how many of the drafted tokens were;
 *   accept_prob [drafts]: min(1, p_d / q_d) of every drafted token (T = 0: 1 or 0), fp32,
 *   whether or not an earlier one was refused.
 *
 * The weights are whole multiples of 2^-43 of the row's largest (of 1 for the difference),
 * so their sums have one value in any order: the tokens of a request depend on its own
 * logits and numbers alone, not on the batch or the launch. What is below 2^-44 is never
 * drawn. Tests are made in fp64.
 *
 * Rows and values outside the ordinary:
 *  - a logit of -inf has probability 0. A target row of nothing else, or with a NaN or
 *    +inf, accepts nothing; if a token is to be drawn from it, that is -1.
 *  - a token whose draft row is such a row is refused, and drawn from p alone.
 *  - a drafted token outside [0, v) is refused (accept_prob 0); a request whose offsets leave
 *    [0, drafts] or span more than max_drafts, every request from the first one on whose offsets
 *    fall, and a request whose temperature on the device is negative, infinite, NaN or so small
 *    that log2(e) / T is not finite, has accepted 0, -1s, and accept_prob 0 for its tokens. Both
 *    set the status word (the workspace's first int32) to FLJSD_ERR_INVALID_ARG.
 *  - FLJSD_ERR_TIMEOUT in the status word: a bounded device wait expired, the results are none
 *    (whatever else was wrong).
 *  - u_draw outside [0, 1) is taken to its nearer end, NaN as 0; u_accept of NaN refuses.
 *  - tokens of no request, as those before the first one's and behind the last one's, have
 *    accept_prob 0: a buffer may be longer than what a step fills. (offsets given; their rows are
 *    not read.)
 *
 * target and draft in dtype with row strides ld_target and ld_draft (elements, any
 * element alignment); tokens, offsets, out, accepted int64, u_accept [drafts], u_draw,
 * temperatures, accept_prob fp32. workspace: fljsd_verify_workspace_bytes bytes, 16-byte
 * aligned. Errors, found before anything is launched: FLJSD_ERR_INVALID_ARG for requests or
 * v <= 0, drafts or max_drafts < 0, drafts that are not requests * max_drafts without
 * offsets, a stride below v, an unknown dtype, a temperature that is negative, infinite, NaN
 * or so small that log2(e) / T is not finite, a null or misaligned pointer (tokens, u_accept and
 * accept_prob may be NULL with drafts 0); FLJSD_ERR_UNSUPPORTED for v of 2^20 and more,
 * requests above 2^20, drafts above 2^24, max_drafts above 1024, or requests *
 * (2 max_drafts + 1) of 2^27 and more; FLJSD_ERR_WORKSPACE; FLJSD_ERR_CUDA when a launch fails.
 */
size_t fljsd_verify_workspace_bytes(int64_t requests, int64_t drafts);
fljsd_status fljsd_verify(int64_t requests, int64_t drafts, int64_t v, int32_t max_drafts,
                          int32_t dtype, const void* target, int64_t ld_target, const void* draft,
                          int64_t ld_draft, const int64_t* tokens, const float* u_accept,
                          const float* u_draw, const int64_t* offsets, const float* temperatures,
                          float temperature, int64_t* out, int64_t* accepted, float* accept_prob,
                          void* workspace, size_t workspace_bytes, fljsd_stream_t stream);

/* Id of the capture into a CUDA graph that `stream` is in, unique in the process; 0 where
 * it is in none (or on an error). A caller that passes kept = 1 to fljsd_lp_backward needs
 * it: the two calls belong to one capture, or to none. */
uint64_t fljsd_capture_id(fljsd_stream_t stream);

/* Test of the failure paths of fljsd_verify and fljsd_low_rank_add: in calls made from now on the
 * kernels named by FLJSD_STALL_* bits wait for something that does not come, so that their
 * bounded waits expire, after 50 ms: the status word then holds FLJSD_ERR_TIMEOUT, and the context
 * stays usable. 0: as usual. Process-global. */
#define FLJSD_STALL_VERIFY 1          /* the copies of one CTA of each cluster */
#define FLJSD_STALL_LOW_RANK_FIRST 2  /* the products A x */
#define FLJSD_STALL_LOW_RANK_SECOND 4 /* the copies of B */
#define FLJSD_STALL_LOW_RANK_Y 8      /* the copies of y */
void fljsd_test_stall(int32_t kernels);

/* Static, human-readable name of a status code. Never NULL. */
const char* fljsd_status_string(fljsd_status status);

/*
 * Launch accounting and per-kernel timing (for benchmarks).
 *
 * fljsd_launch_count returns the number of kernels this library has launched
 * in the process (all devices, all streams) since load or the last
 * fljsd_launch_count_reset.
 *
 * fljsd_trace_enable(max_launches) turns on per-launch CUDA-event timing on
 * the launching stream for up to max_launches launches (events are created on
 * the current device); fljsd_trace_enable(0) turns it off and releases the
 * events. fljsd_trace_read synchronises the recorded events and returns, for
 * kernel class `kind` (FLJSD_KERNEL_*), the summed milliseconds and the number
 * of recorded launches; fljsd_trace_reset forgets the recorded launches.
 * These are process-global and not thread-safe.
 */
typedef enum {
  FLJSD_KERNEL_GEMM_LOGITS = 0,      /* Z = X . W^T, student and teacher */
  FLJSD_KERNEL_JSD_ROWS = 1,         /* the three passes over V */
  FLJSD_KERNEL_GEMM_GRAD_INPUT = 2,  /* dZ . W_s */
  FLJSD_KERNEL_GEMM_GRAD_WEIGHT = 3, /* dZ^T . X_s into grad_weight */
  FLJSD_KERNEL_SMALL = 4,            /* row count, loss reduction, scaling */
  FLJSD_KERNEL_NUM_KINDS = 5
} fljsd_kernel_kind;

int64_t fljsd_launch_count(void);
void fljsd_launch_count_reset(void);
fljsd_status fljsd_trace_enable(int32_t max_launches);
fljsd_status fljsd_trace_reset(void);
fljsd_status fljsd_trace_read(int32_t kind, double* total_ms, int64_t* launches);

#ifdef __cplusplus
}
#endif

#endif /* FLJSD_H */
