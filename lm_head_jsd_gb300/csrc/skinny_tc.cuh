// Products of a few rows with a large weight (internal). See skinny_tc.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace fljsd {

constexpr int SK_ROWS = 16;  // rows of x at most

// out[i, j] = x[i] . w[j] for m <= SK_ROWS rows of x, w [n x k].
// bf16: x, w bf16, out fp32. e4m3: codes with scales sx [ceil(k / 128) x m] and
// sw [ceil(n / 128) x ceil(k / 128)] (fp8_gemm.cu), out fp32 or bf16.
struct SkinnyArgs {
  int e4m3;
  const void* x; int64_t ldx;
  const void* w; int64_t ldw;
  int64_t m, n, k;
  const float *sx, *sw;
  void* out; int64_t ldo;
  int out_bf16;
  int* status;
  // x and sx come from the kernel launched just before, which does not write w or sw:
  // w is on its way before that kernel has ended.
  bool own_x;
  bool zero_status;  // *status is set to 0 first
  // bf16: parts (m, d, s) as in lp.cuh, [m x skinny_parts(n)], with c = log2(e) / T; the
  // logit of each row's label; the maxima of 32 columns each, [m x 4 ceil(n / 128)], or
  // null. out may then be null.
  float4* part;
  float* cmax;
  float c;
  const int64_t* labels;
  float* zy;
};
// Whether the kernel takes the shape (alignment as for the tensor maps).
bool skinny_supported(const SkinnyArgs& a);
// Parts of a row: one for each epilogue warp.
int64_t skinny_parts(int64_t n);
cudaError_t launch_skinny(const SkinnyArgs& a, cudaStream_t st);

}  // namespace fljsd
