// Entry points of the token log probabilities: argument checks, workspace
// layout, chunk loop. Declarations and semantics are in include/fljsd.h, the
// formulas in lp.cuh.
#include "gemm_tc.cuh"
#include "lp.cuh"
#include "skinny_tc.cuh"

#include <cmath>

namespace fljsd {
namespace {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
inline size_t dsize(int dt) { return dt == FLJSD_BF16 ? 2 : 4; }
inline bool aligned(const void* q, uintptr_t a) { return ((uintptr_t)q & (a - 1)) == 0; }

// The tensor cores take bf16 operands whose rows are a whole number of 16-byte
// units; fp32 and the other bf16 shapes go through the CUDA-core product into
// fp32 logits and the row kernels.
bool on_tensor_cores(const fljsd_lp_problem& p) { return p.dtype == FLJSD_BF16 && p.h % 8 == 0; }

// How the logits of a plan's chunks are reduced.
//  kFused: in the product's epilogue.
//  kFew:   a forward of up to 16 rows, bound by reading w: in the epilogue of the
//          product for few rows (skinny_tc.cu), which writes the fp32 logits beside
//          where alternatives are asked for, 4 bytes for every 2 h of w.
//  kRows:  the CUDA-core product and the row kernels.
enum Path { kFused, kFew, kRows };
Path path_of(const fljsd_lp_problem& p) {
  if (!on_tensor_cores(p)) return kRows;
  return !(p.flags & FLJSD_LP_BACKWARD) && p.bt <= SK_ROWS ? kFew : kFused;
}

// Chunks of a row whose maxima the product of a few rows keeps.
int64_t few_chunks(int64_t v) { return (v + 127) / 128 * (128 / LP_FEW_COLS); }

struct LpLayout {
  Path path;
  bool tc, use_acc32;
  int64_t ld, parts, cap;
  // zeroed: status, count, gmax (in one piece, [zero, zero + zero_bytes))
  size_t zero, zero_bytes, status, count, gmax;
  int dump_blocks, bn;
  size_t part, zy, cand, cmax, dump, z, dz, acc32, splitk, splitk_bytes, total, logits_bytes, stats_bytes;
};

LpLayout lp_layout(const fljsd_lp_problem& p, int64_t c) {
  LpLayout L{};
  const bool bwd = (p.flags & FLJSD_LP_BACKWARD) != 0;
  L.tc = on_tensor_cores(p);
  L.path = path_of(p);
  const bool fused = L.path == kFused;
  L.ld = (p.v + 7) / 8 * 8;
  // (a backward pass reads parts of 128 columns)
  L.bn = fused && !bwd ? lp_head_tile_cols(c, p.v, p.h) : 2 * LP_PART_COLS;
  L.parts = fused             ? (p.v + L.bn / 2 - 1) / (L.bn / 2)
            : L.path == kFew ? few_chunks(p.v)  // (at most)
                             : lp_row_segs(p.v);
  L.cap = L.parts * p.top_k;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at += align_up(bytes);
    return r;
  };
  const size_t rows = (size_t)c;
  L.zero = L.status = take(sizeof(int));
  L.count = take(fused && p.top_k ? rows * sizeof(int) : 0);
  L.gmax = take(fused ? rows * p.top_k * sizeof(unsigned) : 0);
  L.zero_bytes = at - L.zero;
  L.part = take(rows * L.parts * sizeof(float4));
  L.zy = take(rows * sizeof(float));
  L.cand = take(fused ? rows * L.cap * sizeof(int2) : 0);
  L.cmax = take(fused || !p.top_k ? 0 : rows * L.parts * (L.path == kFew ? 1 : LP_CHUNKS) * sizeof(float));
  L.dump_blocks = fused ? lp_head_dump_blocks(c, p.v, p.h, p.top_k, L.bn) : 0;
  L.dump = take(rows * L.dump_blocks * 256 * sizeof(float));
  L.stats_bytes = at;
  // 2^t in fp16 that the backward pass turns into dz in place, or fp32 logits (and their
  // bf16 gradient beside them)
  const size_t zb = fused ? (bwd ? rows * L.ld * 2 : 0) : rows * L.ld * 4;
  L.z = take(zb);
  L.dz = L.z;
  if (bwd && !L.tc && p.dtype == FLJSD_BF16) L.dz = take(rows * L.ld * 2);
  L.logits_bytes = at - L.z;
  L.use_acc32 = bwd && (p.flags & FLJSD_FLAG_ACCUM_FP32) && p.dtype == FLJSD_BF16 && c < p.bt;
  L.acc32 = take(L.use_acc32 ? (size_t)p.v * p.h * sizeof(float) : 0);
  L.splitk_bytes = bwd && L.tc && c > 0 ? align_up(tc_splitk_bytes(c, p.h, p.v, TC_PLAN_CTAS)) : 0;
  L.splitk = take(L.splitk_bytes);
  L.total = at;
  return L;
}

float log2_scale(float temperature) {
  return (float)(1.4426950408889634 / (double)temperature);
}
// Positive, finite, and so is what the logits are multiplied by.
bool temperature_ok(float t) { return t > 0.f && std::isfinite(t) && std::isfinite(log2_scale(t)); }

fljsd_status lp_check(const fljsd_lp_problem* p) {
  if (!p) return FLJSD_ERR_INVALID_ARG;
  if (p->bt <= 0 || p->h <= 0 || p->v <= 0 || p->chunk_rows < 0) return FLJSD_ERR_INVALID_ARG;
  if (p->dtype != FLJSD_F32 && p->dtype != FLJSD_BF16) return FLJSD_ERR_INVALID_ARG;
  if (p->top_k < 0 || p->top_k > p->v) return FLJSD_ERR_INVALID_ARG;
  if (!temperature_ok(p->temperature)) return FLJSD_ERR_INVALID_ARG;
  if ((p->flags & ~(FLJSD_LP_BACKWARD | FLJSD_FLAG_ACCUM_FP32)) != 0) return FLJSD_ERR_INVALID_ARG;
  if (p->top_k > LP_MAX_TOP || p->v > (int64_t)1 << 30 || p->bt > (int64_t)1 << 30 ||
      p->h > (int64_t)1 << 20)
    return FLJSD_ERR_UNSUPPORTED;
  return FLJSD_OK;
}

// D[m x n] (+)= A . B^T in dtype, on the tensor cores where they take it.
cudaError_t lp_gemm(int kind, int dtype, bool tc, const void* a, int64_t lda, int a_mn,
                    const void* b, int64_t ldb, int b_mn, void* d, int64_t ldd, int64_t m,
                    int64_t n, int64_t k, int accumulate, float* d32, int finalize, int* status,
                    void* splitk, size_t splitk_bytes, cudaStream_t st) {
  cudaError_t e;
  trace_begin(kind, st);
  if (tc) {
    TcGemmArgs t{a, lda, a_mn, b, ldb, b_mn, d, ldd, m, n, k, accumulate,
                 1, status, nullptr, 0.f, d32, finalize};
    t.splitk_ws = static_cast<float*>(splitk);
    t.splitk_ws_bytes = splitk_bytes;
    e = launch_gemm_tc(t, st);
  } else {
    GemmArgs g{};
    g.a = a; g.sam = a_mn ? 1 : lda; g.sak = a_mn ? lda : 1;
    g.b = b; g.sbn = b_mn ? 1 : ldb; g.sbk = b_mn ? ldb : 1;
    g.c = d; g.ldc = ldd; g.m = m; g.n = n; g.k = k; g.accumulate = accumulate;
    g.c32 = d32; g.finalize = finalize;
    e = launch_gemm_simt(dtype, g, st);
  }
  trace_end(kind, st);
  return e;
}

// The parts of one chunk's rows (and, with `keep`, 2^t or the logits) into the
// workspace; `top` candidates of each row. zeroed: launch_zero came just before;
// first: the product of a few rows clears the status word.
cudaError_t lp_chunk(const fljsd_lp_problem& p, const LpLayout& L, const char* x, const void* w,
                     const int64_t* labels, int64_t rows, int top, bool keep, bool zeroed,
                     bool first, char* ws, cudaStream_t st) {
  const float c = log2_scale(p.temperature);
  if (L.path == kFused) {
    LpHeadArgs h{};
    h.x = x; h.ldx = p.h; h.w = w; h.ldw = p.h; h.m = rows; h.n = p.v; h.k = p.h; h.c = c;
    h.labels = labels;
    h.part = reinterpret_cast<float4*>(ws + L.part);
    h.parts = L.parts;
    h.zy = reinterpret_cast<float*>(ws + L.zy);
    h.top = top;
    h.gmax = reinterpret_cast<unsigned*>(ws + L.gmax);
    h.count = reinterpret_cast<int*>(ws + L.count);
    h.cand = reinterpret_cast<int2*>(ws + L.cand);
    h.dump = reinterpret_cast<float*>(ws + L.dump);
    h.dump_blocks = top ? L.dump_blocks : 0;
    h.bn = L.bn;
    h.e = keep ? ws + L.z : nullptr;
    h.lde = L.ld;
    h.status = reinterpret_cast<int*>(ws + L.status);
    h.own_zeros = zeroed;
    trace_begin(FLJSD_KERNEL_GEMM_LOGITS, st);
    const cudaError_t e = launch_lp_head(h, st);
    trace_end(FLJSD_KERNEL_GEMM_LOGITS, st);
    return e;
  }
  float* z = reinterpret_cast<float*>(ws + L.z);
  if (L.path == kFew) {
    SkinnyArgs k{};
    k.x = x; k.ldx = p.h; k.w = w; k.ldw = p.h; k.m = rows; k.n = p.v; k.k = p.h;
    k.out = top ? z : nullptr; k.ldo = L.ld;  // (alternatives are ranked from them)
    k.status = reinterpret_cast<int*>(ws + L.status);
    k.zero_status = first;
    k.part = reinterpret_cast<float4*>(ws + L.part);
    k.cmax = top ? reinterpret_cast<float*>(ws + L.cmax) : nullptr;
    k.c = c; k.labels = labels;
    k.zy = reinterpret_cast<float*>(ws + L.zy);
    trace_begin(FLJSD_KERNEL_GEMM_LOGITS, st);
    const cudaError_t e = launch_skinny(k, st);
    trace_end(FLJSD_KERNEL_GEMM_LOGITS, st);
    return e;
  }
  const cudaError_t e = lp_gemm(FLJSD_KERNEL_GEMM_LOGITS, p.dtype, false, x, p.h, 0, w, p.h, 0, z,
                                L.ld, rows, p.v, p.h, 0, z, 0, nullptr, nullptr, 0, st);
  if (e != cudaSuccess) return e;
  LpRowsArgs r{};
  r.z = z; r.ld = L.ld; r.v = p.v; r.rows = rows; r.c = c; r.labels = labels;
  r.part = reinterpret_cast<float4*>(ws + L.part);
  r.zy = reinterpret_cast<float*>(ws + L.zy);
  r.cmax = top ? reinterpret_cast<float*>(ws + L.cmax) : nullptr;
  r.own_logits = true;
  r.segs = (int)L.parts; r.group = 1;
  return launch_lp_rows(FLJSD_F32, r, st);
}

fljsd_status lp_plan_check(const fljsd_lp_problem* p, const fljsd_plan_t* plan,
                           size_t workspace_bytes, LpLayout* L) {
  const int64_t c = plan->chunk_rows;
  if (c <= 0 || c > p->bt) return FLJSD_ERR_INVALID_ARG;
  *L = lp_layout(*p, c);
  if (plan->ld != L->ld || plan->workspace_bytes != L->total ||
      plan->num_chunks != (p->bt + c - 1) / c)
    return FLJSD_ERR_INVALID_ARG;
  return workspace_bytes < L->total ? FLJSD_ERR_WORKSPACE : FLJSD_OK;
}

struct LogitsLayout {
  int64_t parts;
  size_t part, zy, cmax, total;
};
LogitsLayout logits_layout(int64_t rows, int64_t v, int k) {
  LogitsLayout L{};
  L.parts = lp_row_segs(v);
  L.part = kAlign;  // after the status word
  L.zy = L.part + align_up((size_t)rows * L.parts * sizeof(float4));
  L.cmax = L.zy + align_up((size_t)rows * sizeof(float));
  L.total = L.cmax + (k > 0 ? align_up((size_t)rows * L.parts * LP_CHUNKS * sizeof(float)) : 0);
  return L;
}

fljsd_status logits_check(int64_t rows, int64_t v, int64_t ld, int32_t dtype, int32_t top_k,
                          float temperature) {
  if (rows <= 0 || v <= 0 || ld < v) return FLJSD_ERR_INVALID_ARG;
  if (dtype != FLJSD_F32 && dtype != FLJSD_BF16) return FLJSD_ERR_INVALID_ARG;
  if (top_k < 0 || top_k > v) return FLJSD_ERR_INVALID_ARG;
  if (!temperature_ok(temperature)) return FLJSD_ERR_INVALID_ARG;
  if (top_k > LP_MAX_TOP || rows > (int64_t)1 << 30 || v > (int64_t)1 << 30)
    return FLJSD_ERR_UNSUPPORTED;
  return FLJSD_OK;
}

}  // namespace
}  // namespace fljsd

using namespace fljsd;

extern "C" {

fljsd_status fljsd_lp_plan(const fljsd_lp_problem* p, size_t free_hbm_bytes, fljsd_plan_t* out) {
  const fljsd_status st = lp_check(p);
  if (st != FLJSD_OK) return st;
  if (!out) return FLJSD_ERR_INVALID_ARG;
  int64_t c = p->chunk_rows > 0 && p->chunk_rows < p->bt ? p->chunk_rows : p->bt;
  if (p->chunk_rows == 0 && free_hbm_bytes != 0) {
    // the largest chunk within half of the free memory: all rows, or the first
    // of a falling series of multiples of 128 (then of single rows) that fits
    const size_t budget = free_hbm_bytes / 2;
    if (lp_layout(*p, c).total > budget) {
      int64_t lo = 0, hi = c;  // lo fits (no rows always do), hi does not
      while (hi - lo > 1) {
        const int64_t mid = lo + (hi - lo) / 2;
        (lp_layout(*p, mid).total <= budget ? lo : hi) = mid;
      }
      c = lo >= 128 ? lo / 128 * 128 : lo;
      // (the scratch of a split contraction does not grow evenly with the rows)
      while (c > 0 && lp_layout(*p, c).total > budget) c -= c > 128 ? 128 : 1;
      if (c <= 0) return FLJSD_ERR_WORKSPACE;
    }
  }
  const LpLayout L = lp_layout(*p, c);
  out->chunk_rows = c;
  out->num_chunks = (p->bt + c - 1) / c;
  out->ld = L.ld;
  out->workspace_bytes = L.total;
  out->logits_bytes = L.logits_bytes;
  out->stats_bytes = L.stats_bytes;
  out->status_offset = L.status;
  return FLJSD_OK;
}

fljsd_status fljsd_lp_forward(const fljsd_lp_problem* p, const fljsd_plan_t* plan, const void* x,
                              const void* w, const int64_t* labels, float* logp, float* entropy,
                              float* lse, float* norm, float* top_logp, int64_t* top_id,
                              void* workspace, size_t workspace_bytes, fljsd_stream_t stream_) {
  fljsd_status st = lp_check(p);
  if (st != FLJSD_OK) return st;
  if (!plan || !x || !w || !entropy || !lse || !norm || !workspace || (labels && !logp))
    return FLJSD_ERR_INVALID_ARG;
  if (p->top_k > 0 && (!top_logp || !top_id)) return FLJSD_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(workspace, 16) || !aligned(labels, 8) ||
      !aligned(logp, 4) || !aligned(entropy, 4) || !aligned(lse, 4) || !aligned(norm, 8) ||
      !aligned(top_logp, 4) || !aligned(top_id, 8))
    return FLJSD_ERR_INVALID_ARG;
  LpLayout L;
  st = lp_plan_check(p, plan, workspace_bytes, &L);
  if (st != FLJSD_OK) return st;
  const int64_t c = plan->chunk_rows;
  const bool keep = (p->flags & FLJSD_LP_BACKWARD) && c == p->bt;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  char* ws = static_cast<char*>(workspace);
  for (int64_t r0 = 0; r0 < p->bt; r0 += c) {
    const int64_t rows = p->bt - r0 < c ? p->bt - r0 : c;
    // the status word is reset once (by the product of a few rows itself), the counts and
    // thresholds for each chunk
    const size_t z0 = r0 == 0 ? L.zero : L.count, zb = L.zero + L.zero_bytes - z0;
    const bool zeros = L.path != kFew && zb > 0;
    if (zeros && launch_zero(ws + z0, zb, stream) != cudaSuccess) return FLJSD_ERR_CUDA;
    const char* xc = static_cast<const char*>(x) + (size_t)r0 * p->h * dsize(p->dtype);
    if (lp_chunk(*p, L, xc, w, labels ? labels + r0 : nullptr, rows, p->top_k, keep, zeros, r0 == 0,
                 ws, stream) != cudaSuccess)
      return FLJSD_ERR_CUDA;
    LpJoinArgs j{};
    j.rows = rows; j.row0 = r0; j.v = p->v;
    j.part = reinterpret_cast<const float4*>(ws + L.part);
    j.parts = L.parts;
    j.c = log2_scale(p->temperature);
    j.inv_t = 1.f / p->temperature;
    j.zy = reinterpret_cast<const float*>(ws + L.zy);
    j.labels = labels; j.ignore_index = p->ignore_index;
    j.status = reinterpret_cast<int*>(ws + L.status);
    j.logp = logp; j.entropy = entropy; j.lse = lse; j.norm = reinterpret_cast<float2*>(norm);
    j.k = p->top_k;
    if (L.path == kFused) {
      j.cand = reinterpret_cast<const int2*>(ws + L.cand);
      j.cap = L.cap;
      j.count = reinterpret_cast<const int*>(ws + L.count);
      j.gmax = reinterpret_cast<const unsigned*>(ws + L.gmax);
      j.dump = L.dump_blocks ? reinterpret_cast<const float*>(ws + L.dump) : nullptr;
      j.dump_cols = (int64_t)L.dump_blocks * 2 * LP_PART_COLS;
      j.part_cols = L.bn / 2;
    } else {
      j.z = ws + L.z; j.z_dtype = FLJSD_F32; j.ld = L.ld;
      j.cmax = reinterpret_cast<const float*>(ws + L.cmax);
      if (L.path == kFew) {
        j.parts = skinny_parts(p->v);
        j.few_chunks = few_chunks(p->v);
      } else {
        j.segs = L.parts;
      }
    }
    j.top_logp = top_logp; j.top_id = top_id;
    if (launch_lp_join(j, stream) != cudaSuccess) return FLJSD_ERR_CUDA;
  }
  return FLJSD_OK;
}

fljsd_status fljsd_lp_backward(const fljsd_lp_problem* p, const fljsd_plan_t* plan, const void* x,
                               const void* w, const int64_t* labels, const float* logp,
                               const float* entropy, const float* norm, const float* grad_logp,
                               const float* grad_entropy, int32_t kept, void* grad_input,
                               void* grad_weight, void* workspace, size_t workspace_bytes,
                               fljsd_stream_t stream_) {
  fljsd_status st = lp_check(p);
  if (st != FLJSD_OK) return st;
  if (!(p->flags & FLJSD_LP_BACKWARD) || (kept != 0 && kept != 1)) return FLJSD_ERR_INVALID_ARG;
  if (!plan || !x || !w || !entropy || !norm || !workspace || (!grad_input && !grad_weight))
    return FLJSD_ERR_INVALID_ARG;
  if ((labels && !logp) || (grad_logp && !labels)) return FLJSD_ERR_INVALID_ARG;
  const void* p16[] = {x, w, workspace, grad_input, grad_weight};
  for (const void* q : p16)
    if (!aligned(q, 16)) return FLJSD_ERR_INVALID_ARG;
  if (!aligned(labels, 8) || !aligned(logp, 4) || !aligned(entropy, 4) || !aligned(norm, 8) ||
      !aligned(grad_logp, 4) || !aligned(grad_entropy, 4))
    return FLJSD_ERR_INVALID_ARG;
  LpLayout L;
  st = lp_plan_check(p, plan, workspace_bytes, &L);
  if (st != FLJSD_OK) return st;
  const int64_t c = plan->chunk_rows;
  if (kept && c != p->bt) return FLJSD_ERR_INVALID_ARG;  // one chunk's values are kept at most
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  char* ws = static_cast<char*>(workspace);
  int* status = reinterpret_cast<int*>(ws + L.status);
  const size_t s = dsize(p->dtype);
  for (int64_t r0 = 0; r0 < p->bt; r0 += c) {
    const int64_t rows = p->bt - r0 < c ? p->bt - r0 : c;
    const char* xc = static_cast<const char*>(x) + (size_t)r0 * p->h * s;
    if (!kept &&
        lp_chunk(*p, L, xc, w, nullptr, rows, 0, true, false, false, ws, stream) != cudaSuccess)
      return FLJSD_ERR_CUDA;
    LpGradArgs g{};
    g.z = ws + L.z; g.ldz = L.ld;
    g.out = ws + L.dz; g.ldo = L.ld;
    g.v = p->v; g.rows = rows; g.row0 = r0;
    g.c = log2_scale(p->temperature);
    g.inv_t = 1.f / p->temperature;
    g.labels = labels; g.ignore_index = p->ignore_index;
    g.logp = logp; g.entropy = entropy; g.norm = reinterpret_cast<const float2*>(norm);
    g.grad_logp = grad_logp; g.grad_entropy = grad_entropy;
    g.part = reinterpret_cast<const float4*>(ws + L.part);
    g.parts = L.parts;
    if (launch_lp_grad(L.tc ? FLJSD_BF16 : FLJSD_F32, p->dtype, L.tc, g, stream) != cudaSuccess)
      return FLJSD_ERR_CUDA;
    if (grad_input &&
        lp_gemm(FLJSD_KERNEL_GEMM_GRAD_INPUT, p->dtype, L.tc, g.out, L.ld, 0, w, p->h, 1,
                static_cast<char*>(grad_input) + (size_t)r0 * p->h * s, p->h, rows, p->h, p->v, 0,
                nullptr, 0, status, ws + L.splitk, L.splitk_bytes, stream) != cudaSuccess)
      return FLJSD_ERR_CUDA;
    const bool last = r0 + rows >= p->bt;
    if (grad_weight &&
        lp_gemm(FLJSD_KERNEL_GEMM_GRAD_WEIGHT, p->dtype, L.tc, g.out, L.ld, 1, xc, p->h, 1,
                grad_weight, p->h, p->v, p->h, rows, r0 > 0 ? 1 : 0,
                L.use_acc32 ? reinterpret_cast<float*>(ws + L.acc32) : nullptr,
                L.use_acc32 && last ? 1 : 0, status, nullptr, 0, stream) != cudaSuccess)
      return FLJSD_ERR_CUDA;
  }
  return FLJSD_OK;
}

uint64_t fljsd_capture_id(fljsd_stream_t stream) {
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  unsigned long long id = 0;
  if (cudaStreamGetCaptureInfo(reinterpret_cast<cudaStream_t>(stream), &status, &id) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return status == cudaStreamCaptureStatusActive ? id : 0;
}

size_t fljsd_logits_lp_workspace_bytes(int64_t rows, int64_t v, int32_t top_k) {
  if (logits_check(rows, v, v, FLJSD_F32, top_k, 1.f) != FLJSD_OK) return 0;
  return logits_layout(rows, v, top_k).total;
}

fljsd_status fljsd_logits_lp(int64_t rows, int64_t v, int64_t ld, int32_t dtype, int32_t top_k,
                             float temperature, int64_t ignore_index, const void* logits,
                             const int64_t* labels, float* logp, float* entropy, float* lse,
                             float* norm, float* top_logp, int64_t* top_id, void* workspace,
                             size_t workspace_bytes, fljsd_stream_t stream_) {
  const fljsd_status st = logits_check(rows, v, ld, dtype, top_k, temperature);
  if (st != FLJSD_OK) return st;
  if (!logits || !entropy || !lse || !norm || !workspace || (labels && !logp))
    return FLJSD_ERR_INVALID_ARG;
  if (top_k > 0 && (!top_logp || !top_id)) return FLJSD_ERR_INVALID_ARG;
  if (!aligned(logits, dsize(dtype)) || !aligned(workspace, 16) || !aligned(labels, 8) ||
      !aligned(logp, 4) || !aligned(entropy, 4) || !aligned(lse, 4) || !aligned(norm, 8) ||
      !aligned(top_logp, 4) || !aligned(top_id, 8))
    return FLJSD_ERR_INVALID_ARG;
  const LogitsLayout L = logits_layout(rows, v, top_k);
  if (workspace_bytes < L.total) return FLJSD_ERR_WORKSPACE;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  char* ws = static_cast<char*>(workspace);
  LpRowsArgs r{};
  r.status = reinterpret_cast<int*>(ws);
  r.z = logits; r.ld = ld; r.v = v; r.rows = rows; r.c = log2_scale(temperature);
  r.labels = labels;
  r.part = reinterpret_cast<float4*>(ws + L.part);
  r.zy = reinterpret_cast<float*>(ws + L.zy);
  r.cmax = top_k > 0 ? reinterpret_cast<float*>(ws + L.cmax) : nullptr;
  r.segs = (int)L.parts; r.group = lp_row_group(dtype, rows, L.parts);
  if (launch_lp_rows(dtype, r, stream) != cudaSuccess) return FLJSD_ERR_CUDA;
  LpJoinArgs j{};
  j.rows = rows; j.v = v; j.part = r.part; j.segs = L.parts; j.c = r.c;
  j.parts = (r.segs + r.group - 1) / r.group; j.inv_t = 1.f / temperature;
  j.zy = r.zy;
  j.labels = labels; j.ignore_index = ignore_index;
  j.status = reinterpret_cast<int*>(ws);
  j.logp = logp; j.entropy = entropy; j.lse = lse; j.norm = reinterpret_cast<float2*>(norm);
  j.k = top_k; j.z = logits; j.z_dtype = dtype; j.ld = ld; j.cmax = r.cmax;
  j.top_logp = top_logp; j.top_id = top_id;
  return launch_lp_join(j, stream) == cudaSuccess ? FLJSD_OK : FLJSD_ERR_CUDA;
}

fljsd_status fljsd_logits_lp_backward(int64_t rows, int64_t v, int64_t ld, int64_t ld_grad,
                                      int32_t dtype, float temperature, int64_t ignore_index,
                                      const void* logits, const int64_t* labels,
                                      const float* logp, const float* entropy, const float* norm,
                                      const float* grad_logp, const float* grad_entropy,
                                      void* grad_logits, fljsd_stream_t stream_) {
  const fljsd_status st = logits_check(rows, v, ld, dtype, 0, temperature);
  if (st != FLJSD_OK) return st;
  if (!logits || !entropy || !norm || !grad_logits || ld_grad < v) return FLJSD_ERR_INVALID_ARG;
  if ((labels && !logp) || (grad_logp && !labels)) return FLJSD_ERR_INVALID_ARG;
  if (!aligned(logits, dsize(dtype)) || !aligned(grad_logits, dsize(dtype)) || !aligned(labels, 8) ||
      !aligned(logp, 4) || !aligned(entropy, 4) || !aligned(norm, 8) || !aligned(grad_logp, 4) ||
      !aligned(grad_entropy, 4))
    return FLJSD_ERR_INVALID_ARG;
  LpGradArgs g{};
  g.z = logits; g.ldz = ld; g.out = grad_logits; g.ldo = ld_grad; g.v = v; g.rows = rows;
  g.c = log2_scale(temperature);
  g.inv_t = 1.f / temperature;
  g.labels = labels; g.ignore_index = ignore_index;
  g.logp = logp; g.entropy = entropy; g.norm = reinterpret_cast<const float2*>(norm);
  g.grad_logp = grad_logp; g.grad_entropy = grad_entropy;
  return launch_lp_grad(dtype, dtype, false, g, reinterpret_cast<cudaStream_t>(stream_)) == cudaSuccess
             ? FLJSD_OK
             : FLJSD_ERR_CUDA;
}

}  // extern "C"
