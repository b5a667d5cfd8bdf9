// Token log probabilities: what the fused product (lp_head_tc.cu), the row
// kernels (lp_rows.cu) and the entry points (lp_api.cu) share.
//
// With z the logits of a row and c = log2(e) / T:
//   m = max z_j,  t_j = c (z_j - m),  d = sum 2^t_j,  s = sum 2^t_j t_j,
//   lse = m / T + ln2 log2 d,  log p_j = ln2 (t_j - log2 d),
//   entropy = -sum p_j log p_j = ln2 (log2 d - s / d).
// A row is cut into parts (up to 128 columns of a product's tile, what a warp sees of
// the product of a few rows, or up to four segments of given logits); each part writes
// (m, d, s), and k_lp_join combines them. For the k largest it has, from the product, at
// most k candidates of each part, and from logits that lie in memory the maximum of each
// 256 of them (32 from the product of a few rows): the k-th largest of those maxima
// says which few have to be read again. The entropy comes from
// sums centred on the maximum: lse - sum p_j s_j would cancel all digits of a
// peaked row. The difference z - m is taken before the scale, so that a row of
// the type's lowest value (a mask that leaves nothing) does not overflow, and
// (m, log2 d) are handed to the backward pass apart: their sum would lose the
// second beside a large first. All of it is held in fp32.
#pragma once

#include "internal.cuh"

namespace fljsd {

constexpr int LP_MAX_TOP = 32;
constexpr int LP_PART_COLS = 128;  // columns of a part of the fused product (at most)
constexpr int LP_FEW_COLS = 32;    // behind a kept maximum of the product of a few rows
constexpr int LP_SEG = 8192;       // elements of a segment of given logits
constexpr int LP_CHUNKS = 32;      // maxima kept of a segment: of 256 logits each
// Segments of a row of given logits: they are counted from the 16-byte boundary
// at or before the row, so a row that starts off one may need one more.
inline int64_t lp_row_segs(int64_t v) { return (v + 7 + LP_SEG - 1) / LP_SEG; }

struct LpJoinArgs {
  int64_t rows, row0, v;
  const float4* part;  // [rows x parts] (m, d, s, -); m = -inf: no finite logit
  int64_t parts;
  float c, inv_t;      // log2(e) / T, 1 / T
  const float* zy;     // [rows] logit of the label (written where it is in [0, v))
  const int64_t* labels;  // [bt] or null, indexed by row0 + row
  int64_t ignore_index;
  int* status;         // FLJSD_ERR_INVALID_ARG for a label outside [0, v)
  float *logp, *entropy, *lse;  // [bt]; logp null without labels
  float2* norm;        // [bt] (m, log2 d)
  int k;
  // from the product:
  const int2* cand;    // [rows x cap] (value bits, column)
  int64_t cap;
  const int* count;    // [rows] candidates of each row
  const unsigned* gmax;  // [k x rows] group maxima (see lp_head_tc.cu)
  const float* dump;   // [rows x dump_cols] logits of the first columns, or null: of each
  int64_t dump_cols;   // LP_PART_COLS the first part_cols, one part's
  int part_cols;
  // from given logits:
  const void* z;       // [rows x ld], or null
  int z_dtype;
  int64_t ld;
  int64_t segs;        // lp_row_segs
  const float* cmax;   // [rows x chunks]: segs * LP_CHUNKS, or few_chunks
  int64_t few_chunks;  // of LP_FEW_COLS columns, from the product of a few rows; else 0
  float* top_logp;     // [bt x k]
  int64_t* top_id;     // [bt x k]
};
cudaError_t launch_lp_join(const LpJoinArgs& a, cudaStream_t st);
// Zeros over whole 16-byte units, by a kernel that the next may be launched behind.
cudaError_t launch_zero(void* to, size_t bytes, cudaStream_t st);

struct LpRowsArgs {
  const void* z;       // [rows x ld]
  int64_t ld, v, rows, row0;
  float c;
  const int64_t* labels;
  int segs, group;     // lp_row_segs(v), and how many of them make a part
  float4* part;        // [rows x ceil(segs / group)]
  float* zy;
  float* cmax;         // [rows x segs * LP_CHUNKS], or null
  int* status;         // set to 0, or null
  bool own_logits;     // fp32, from the kernel launched just before
};
// How many of a row's segments one CTA reduces into a part.
int lp_row_group(int dtype, int64_t rows, int64_t segs);
cudaError_t launch_lp_rows(int dtype, const LpRowsArgs& a, cudaStream_t st);

// dz = (a (1[j = y] - p_j) - b p_j (log p_j + entropy)) / T from logits
// (z_dtype) into out (out_dtype); from_e: z holds 2^t_j in fp16, relative to
// the maximum of each part, and out may be the same memory.
struct LpGradArgs {
  const void* z;
  int64_t ldz;
  void* out;
  int64_t ldo, v, rows, row0;
  float c, inv_t;
  const int64_t* labels;
  int64_t ignore_index;
  const float *logp, *entropy, *grad_logp, *grad_entropy;  // [bt], by row0 + row; the last two or null
  const float2* norm;  // [bt]
  const float4* part;  // from_e
  int64_t parts;
};
cudaError_t launch_lp_grad(int z_dtype, int out_dtype, bool from_e, const LpGradArgs& a,
                           cudaStream_t st);

// The fused product (lp_head_tc.cu).
struct LpHeadArgs {
  const void* x; int64_t ldx;
  const void* w; int64_t ldw;
  int64_t m, n, k;     // rows, vocabulary, hidden size
  float c;
  const int64_t* labels;  // [m] or null (already offset to the first row)
  float4* part;
  int64_t parts;
  float* zy;
  int top;
  unsigned* gmax;      // [top x m], zeroed
  int* count;          // [m], zeroed
  int2* cand;          // [m x parts * top]
  int bn;              // columns of a tile (two parts): lp_head_tile_cols, or 256
  float* dump;         // [m x 256 dump_blocks] logits of the first tiles' columns (LpJoinArgs)
  int dump_blocks;
  void* e;             // [m x lde] fp16: 2^t_j relative to each part's maximum, or null
  int64_t lde;
  int* status;
  bool own_zeros;      // count, gmax and status were zeroed by the kernel launched just before
};
bool lp_head_supported(const LpHeadArgs& a);
// Columns of a tile, a multiple of 16 up to 256: as few as the rounds of tiles over the
// SMs allow, so that the last round is as full as the others.
int lp_head_tile_cols(int64_t m, int64_t n, int64_t k);
// Tiles in a row of them whose logits are best written out instead of listed.
int lp_head_dump_blocks(int64_t m, int64_t n, int64_t k, int top, int bn);
cudaError_t launch_lp_head(const LpHeadArgs& a, cudaStream_t st);

// Floats as integers in their order (0 is below every value); -0.0 becomes +0.0, its equal.
__host__ __device__ inline unsigned lp_key(float x) {
  x += 0.f;
#ifdef __CUDA_ARCH__
  const unsigned u = __float_as_uint(x);
#else
  unsigned u;
  __builtin_memcpy(&u, &x, 4);
#endif
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

}  // namespace fljsd
