// Token log probabilities: parts of given logits, the join of a row's parts,
// and the gradient in the logits. The formulas are in lp.cuh.
//
// k_lp_rows cuts each row into segments of 8192 logits, one CTA each: the
// segment stays in registers (32 values a thread) between the maximum, the sums
// and the candidates, so logits are read once whatever k is, and a single row
// of 128256 still runs on 16 CTAs. k_lp_grad is elementwise. Both are bound by
// HBM.
#include "lp.cuh"
#include "jsd_math.cuh"

#include <cuda_fp16.h>

namespace fljsd {
namespace {

using namespace rowmath;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = LP_SEG / kThreads;  // logits a thread holds
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kJoinThreads = 128;
constexpr int kJoinCap = 1024;  // candidates ranked in shared memory

__device__ __forceinline__ float val(const float* p) { return *p; }
__device__ __forceinline__ float val(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float val(const __half* p) { return __half2float(*p); }

// Eight values, 16-byte aligned.
__device__ __forceinline__ void load8(const float* p, float (&o)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
  o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&o)[8]) {
  Vec<__nv_bfloat16>::load(p, o);
}
__device__ __forceinline__ void load8(const __half* p, float (&o)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    o[2 * i] = f.x;
    o[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void store8(float* p, const float (&o)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(o[0], o[1], o[2], o[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(o[4], o[5], o[6], o[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&o)[8]) {
  Vec<__nv_bfloat16>::store(p, o);
}

// Value first, then the lower column: one key for each candidate.
__device__ __forceinline__ unsigned long long cand_key(int2 c) {
  return c.y < 0 ? 0ull
                 : ((unsigned long long)lp_key(__int_as_float(c.x)) << 32) | (0xffffffffu - (unsigned)c.y);
}
__device__ __forceinline__ float key_value(unsigned long long key) {
  const unsigned k = (unsigned)(key >> 32);
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}
__device__ __forceinline__ int key_col(unsigned long long key) {
  return (int)(0xffffffffu - (unsigned)key);
}

template <int W>
__device__ __forceinline__ float block_max(float x, float* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
  __syncthreads();
  x = sh[0];
#pragma unroll
  for (int w = 1; w < W; ++w) x = fmaxf(x, sh[w]);
  __syncthreads();
  return x;
}
// Sums in a fixed order, so that results do not vary from run to run.
template <int W>
__device__ __forceinline__ float2 block_sum2(float2 x, float2* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    x.x += __shfl_xor_sync(0xffffffffu, x.x, o);
    x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
  }
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
  __syncthreads();
  x = sh[0];
#pragma unroll
  for (int w = 1; w < W; ++w) {
    x.x += sh[w].x;
    x.y += sh[w].y;
  }
  __syncthreads();
  return x;
}
template <int W>
__device__ __forceinline__ unsigned long long block_max64(unsigned long long x,
                                                          unsigned long long* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long y = __shfl_xor_sync(0xffffffffu, x, o);
    x = y > x ? y : x;
  }
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
  __syncthreads();
  x = sh[0];
#pragma unroll
  for (int w = 1; w < W; ++w) x = sh[w] > x ? sh[w] : x;
  __syncthreads();
  return x;
}

// Element offsets of one thread's values inside its segment: vectors of N
// elements, kThreads vectors apart. `lead` elements before the segment's first
// 16-byte boundary belong to a vector that starts before it and is read one
// element at a time, as is the vector that crosses the end.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_lp_rows(LpRowsArgs a, int64_t parts) {
  constexpr int N = Vec<T>::N;
  constexpr int V = kPer / N;
  __shared__ float shf[kWarps];
  __shared__ float2 sh2[kWarps];
  __shared__ unsigned long long sh64[kWarps];
  __shared__ float tmax[kThreads];
  __shared__ unsigned long long list[2 * kThreads];
  __shared__ int n_list;
  __shared__ float s_thr;
  const int tid = threadIdx.x;
  for (int64_t unit = blockIdx.x; unit < a.rows * parts; unit += gridDim.x) {
    const int64_t r = unit / parts, part = unit - r * parts;
    const T* zr = reinterpret_cast<const T*>(a.z) + r * a.ld;
    // segments start on a 16-byte boundary (counted from the row's first one)
    const int64_t lead = (((uintptr_t)zr) & 15u) / sizeof(T);
    const int64_t e0 = part * LP_SEG - lead;  // first element, may be before the row
    const int64_t e1 = e0 + LP_SEG < a.v ? e0 + LP_SEG : a.v;
    float z[kPer];
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int64_t j = e0 + (int64_t)(u * kThreads + tid) * N;
      if (j >= 0 && j + N <= e1) {
        float o[N];
        Vec<T>::load(zr + j, o);
#pragma unroll
        for (int e = 0; e < N; ++e) z[u * N + e] = o[e];
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
          z[u * N + e] = (j + e >= 0 && j + e < e1) ? val(zr + j + e) : -INFINITY;
      }
    }
    float mx = -INFINITY;  // (skips NaN)
#pragma unroll
    for (int i = 0; i < kPer; ++i) mx = fmaxf(mx, z[i]);
    const float tm = mx;
    mx = block_max<kWarps>(mx, shf);
    const float ref = mx == -INFINITY ? 0.f : mx;
    float2 ds = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float x = __fmul_rn(z[i] - ref, a.c);
      const float y = ex2(x);
      ds.x += y;
      ds.y = __fmaf_rn(y, fmaxf(x, -1024.f), ds.y);  // a logit of -inf adds 0, NaN stays
    }
    ds = block_sum2<kWarps>(ds, sh2);
    if (tid == 0) {
      a.part[r * parts + part] = make_float4(mx, ds.x, ds.y, 0.f);
      if (a.labels && part == 0) {
        const int64_t y = a.labels[a.row0 + r];
        if (y >= 0 && y < a.v) a.zy[r] = val(zr + y);
      }
    }
    if (a.k > 0) {
      // The k-th largest of the threads' maxima bounds the k-th largest logit
      // from below: what reaches it is listed and ranked. A list that
      // overflows (many equal logits) is replaced by k rounds of the largest
      // remaining key.
      tmax[tid] = tm;
      if (tid == 0) {
        n_list = 0;
        s_thr = -INFINITY;
      }
      __syncthreads();
      int rank = 0;
      for (int j = 0; j < kThreads; ++j) {
        const float o = tmax[j];
        rank += (o > tm || (o == tm && j < tid)) ? 1 : 0;
      }
      if (rank == a.k - 1) s_thr = tm;
      __syncthreads();
      const float thr = s_thr;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (z[i] >= thr && z[i] > -INFINITY) {
          const int at = atomicAdd(&n_list, 1);
          const int64_t col = e0 + (int64_t)((i / N) * kThreads + tid) * N + i % N;
          if (at < 2 * kThreads)
            list[at] = cand_key(make_int2(__float_as_int(z[i]), (int)col));
        }
      }
      __syncthreads();
      const int n = n_list;
      int2* out = a.cand + (r * parts + part) * a.k;
      if (n <= 2 * kThreads) {
        for (int i = tid; i < n; i += kThreads) {
          const unsigned long long key = list[i];
          int above = 0;
          for (int j = 0; j < n; ++j) above += list[j] > key ? 1 : 0;
          if (above < a.k) out[above] = make_int2(__float_as_int(key_value(key)), key_col(key));
        }
        for (int i = n + tid; i < a.k; i += kThreads) out[i] = make_int2(0, -1);
      } else {
        unsigned long long last = ~0ull;
        for (int q = 0; q < a.k; ++q) {
          unsigned long long best = 0;
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int64_t col = e0 + (int64_t)((i / N) * kThreads + tid) * N + i % N;
            const unsigned long long key =
                z[i] > -INFINITY ? cand_key(make_int2(__float_as_int(z[i]), (int)col)) : 0ull;
            best = key < last && key > best ? key : best;
          }
          best = block_max64<kWarps>(best, sh64);
          if (tid == 0)
            out[q] = best ? make_int2(__float_as_int(key_value(best)), key_col(best)) : make_int2(0, -1);
          last = best;
        }
      }
      __syncthreads();
    }
  }
}

// One CTA to a row: its parts into the row's results, its candidates into the
// k largest.
__global__ void __launch_bounds__(kJoinThreads) k_lp_join(LpJoinArgs a) {
  constexpr int W = kJoinThreads / 32;
  __shared__ float shf[W];
  __shared__ float2 sh2[W];
  __shared__ unsigned long long sh64[W];
  __shared__ unsigned long long list[kJoinCap];
  __shared__ int n_list;
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x, out = a.row0 + r;
  const float4* ps = a.part + r * a.parts;
  float m = -INFINITY;
  for (int64_t i = tid; i < a.parts; i += kJoinThreads) m = fmaxf(m, ps[i].x);
  m = block_max<W>(m, shf);
  float2 ds = make_float2(0.f, 0.f);
  for (int64_t i = tid; i < a.parts; i += kJoinThreads) {
    const float4 q = ps[i];
    // a part without a finite logit has d = s = 0 (NaN where it holds one)
    const float dm = q.x == -INFINITY ? 0.f : __fmul_rn(q.x - m, a.c);
    const float f = ex2(dm);
    ds.x = __fmaf_rn(q.y, f, ds.x);
    // 2^dm (s + d dm): both vanish where 2^dm does
    ds.y = __fmaf_rn(f, __fmaf_rn(q.y, fmaxf(dm, -1024.f), q.z), ds.y);
  }
  ds = block_sum2<W>(ds, sh2);
  // a row without a finite logit has d = 0: lse = -inf, entropy 0
  const bool empty = ds.x == 0.f;
  const float l2d = empty ? 0.f : log2f(ds.x);
  // not through log2 units, in which the type's lowest value overflows
  auto log_p = [&](float z) { return __fmaf_rn(z - m, a.inv_t, -kLn2 * l2d); };
  if (tid == 0) {
    a.lse[out] = empty ? -INFINITY : __fmaf_rn(m, a.inv_t, kLn2 * l2d);
    a.norm[out] = make_float2(empty ? -INFINITY : m, l2d);
    const int64_t y = a.labels ? a.labels[out] : 0;
    bool live = true;
    if (a.labels) {
      live = y != a.ignore_index;
      if (live && (y < 0 || y >= a.v)) {
        live = false;
        atomicExch(a.status, (int)FLJSD_ERR_INVALID_ARG);
      }
      float lp = 0.f;
      if (live) lp = empty ? -INFINITY : log_p(a.zy[r]);
      a.logp[out] = lp;
    }
    a.entropy[out] = live && !empty ? kLn2 * (l2d - ds.y / ds.x) : 0.f;
  }
  if (a.k == 0) return;
  // ---- the k largest candidates ----
  const int2* cand = a.cand + r * a.cap;
  const int64_t n_cand = a.count ? (int64_t)a.count[r] : a.cap;
  unsigned least = 0;
  if (a.gmax) {
    least = 0xffffffffu;
    for (int j = 0; j < a.k; ++j) least = min(least, a.gmax[r * a.k + j]);
  }
  if (tid == 0) n_list = 0;
  __syncthreads();
  for (int64_t i = tid; i < n_cand; i += kJoinThreads) {
    const unsigned long long key = cand_key(cand[i]);
    if (key != 0 && (unsigned)(key >> 32) >= least) {
      const int at = atomicAdd(&n_list, 1);
      if (at < kJoinCap) list[at] = key;
    }
  }
  __syncthreads();
  const int n = n_list;
  float* tl = a.top_logp + out * a.k;
  int64_t* ti = a.top_id + out * a.k;
  auto put = [&](int q, unsigned long long key) {
    tl[q] = key ? log_p(key_value(key)) : -INFINITY;
    ti[q] = key ? (int64_t)key_col(key) : -1;
  };
  if (n <= kJoinCap) {
    for (int i = tid; i < n; i += kJoinThreads) {
      const unsigned long long key = list[i];
      int above = 0;
      for (int j = 0; j < n; ++j) above += list[j] > key ? 1 : 0;
      if (above < a.k) put(above, key);
    }
    for (int i = n + tid; i < a.k; i += kJoinThreads) put(i, 0);
    return;
  }
  unsigned long long last = ~0ull;
  for (int q = 0; q < a.k; ++q) {
    unsigned long long best = 0;
    for (int64_t i = tid; i < n_cand; i += kJoinThreads) {
      const unsigned long long key = cand_key(cand[i]);
      best = key < last && key > best ? key : best;
    }
    best = block_max64<W>(best, sh64);
    if (tid == 0) put(q, best);
    last = best;
  }
}

struct GradRow {
  float a, b, ent, m, l2;  // log2 p = c (z - m) - l2
  int64_t y;
  float py;
  bool live;
};

// dz of one logit; lp2 = log2 p. -inf: p = 0 and p log p = 0.
__device__ __forceinline__ float grad_of(const GradRow& g, float lp2) {
  const float p = ex2(lp2);
  const float t = __fmaf_rn(g.b, __fmaf_rn(kLn2, fmaxf(lp2, -1024.f), g.ent), g.a);
  return -p * t;
}

template <typename TI, typename TO, bool FROM_E>
__global__ void __launch_bounds__(kThreads) k_lp_grad(LpGradArgs a, int64_t segs) {
  constexpr int N = 8;
  for (int64_t unit = blockIdx.x; unit < a.rows * segs; unit += gridDim.x) {
    const int64_t r = unit / segs, seg = unit - r * segs;
    const TI* zr = reinterpret_cast<const TI*>(a.z) + r * a.ldz;
    TO* orow = reinterpret_cast<TO*>(a.out) + r * a.ldo;
    const int64_t row = a.row0 + r;
    GradRow g;
    g.y = a.labels ? a.labels[row] : -1;
    g.live = !a.labels || (g.y != a.ignore_index && g.y >= 0 && g.y < a.v);
    const float2 norm = a.norm[row];
    g.m = norm.x;
    g.l2 = norm.y;
    g.live = g.live && !(g.m == -INFINITY && g.l2 == 0.f);  // (a row of NaN stays NaN)
    g.a = a.grad_logp && a.labels ? a.grad_logp[row] * a.inv_t : 0.f;
    g.b = a.grad_entropy ? a.grad_entropy[row] * a.inv_t : 0.f;
    g.ent = a.entropy[row];
    const bool has_y = g.live && a.labels;
    const float lpy = has_y ? a.logp[row] : 0.f;
    // the label's own element from its fp32 log probability: 1 - p_y would
    // lose its digits to a rounded p_y
    const float dzy =
        has_y ? __fmaf_rn(-ex2(lpy * (1.f / kLn2)),
                          __fmaf_rn(g.b, fmaxf(lpy, -1024.f) + g.ent, g.a), g.a)
              : 0.f;
    // vectors where both sides' addresses allow them (rows of odd length start
    // anywhere), else elements
    const bool vec = ((((uintptr_t)zr) | ((uintptr_t)orow)) & 15u) == 0;
    const int64_t j0 = seg * LP_SEG, j1 = j0 + LP_SEG < a.v ? j0 + LP_SEG : a.v;
    auto one = [&](float z, int64_t j, float ref) {
      const float lp2 = FROM_E ? lg2(z) + ref : __fmul_rn(z - g.m, a.c) - g.l2;
      float o = g.live ? grad_of(g, lp2) : 0.f;
      if (has_y && j == g.y) o = dzy;
      return o;
    };
    if (vec) {
      for (int64_t j = j0 + (int64_t)threadIdx.x * N; j < j1; j += (int64_t)kThreads * N) {
        const float ref = FROM_E ? __fmul_rn(a.part[r * a.parts + j / LP_PART_COLS].x - g.m, a.c) - g.l2 : 0.f;
        float z[N];
        if (j + N <= a.v) {
          load8(zr + j, z);
#pragma unroll
          for (int e = 0; e < N; ++e) z[e] = one(z[e], j + e, ref);
          store8(orow + j, z);
        } else {
          for (int e = 0; j + e < a.v; ++e) Vec<TO>::put(orow + j + e, one(val(zr + j + e), j + e, ref));
        }
      }
    } else {
      for (int64_t j = j0 + threadIdx.x; j < j1; j += kThreads) {
        const float ref = FROM_E ? __fmul_rn(a.part[r * a.parts + j / LP_PART_COLS].x - g.m, a.c) - g.l2 : 0.f;
        Vec<TO>::put(orow + j, one(val(zr + j), j, ref));
      }
    }
  }
}

int64_t units_grid(int64_t units, int per_sm) {
  const int64_t most = (int64_t)num_sms() * per_sm;
  return units < most ? units : most;
}

}  // namespace

cudaError_t launch_lp_join(const LpJoinArgs& a, cudaStream_t st) {
  if (a.rows <= 0) return cudaSuccess;
  trace_begin(FLJSD_KERNEL_SMALL, st);
  k_lp_join<<<(unsigned)a.rows, kJoinThreads, 0, st>>>(a);
  trace_end(FLJSD_KERNEL_SMALL, st);
  return cudaGetLastError();
}

cudaError_t launch_lp_rows(int dtype, const LpRowsArgs& a, cudaStream_t st) {
  if (a.rows <= 0) return cudaSuccess;
  const int64_t parts = lp_row_parts(a.v);
  const unsigned grid = (unsigned)units_grid(a.rows * parts, 32);
  trace_begin(FLJSD_KERNEL_JSD_ROWS, st);
  if (dtype == FLJSD_BF16)
    k_lp_rows<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a, parts);
  else
    k_lp_rows<float><<<grid, kThreads, 0, st>>>(a, parts);
  trace_end(FLJSD_KERNEL_JSD_ROWS, st);
  return cudaGetLastError();
}

cudaError_t launch_lp_grad(int z_dtype, int out_dtype, bool from_e, const LpGradArgs& a,
                           cudaStream_t st) {
  if (a.rows <= 0) return cudaSuccess;
  const int64_t segs = (a.v + LP_SEG - 1) / LP_SEG;
  const unsigned grid = (unsigned)units_grid(a.rows * segs, 32);
  using bf = __nv_bfloat16;
  trace_begin(FLJSD_KERNEL_JSD_ROWS, st);
  if (from_e)
    k_lp_grad<__half, bf, true><<<grid, kThreads, 0, st>>>(a, segs);
  else if (z_dtype == FLJSD_F32 && out_dtype == FLJSD_F32)
    k_lp_grad<float, float, false><<<grid, kThreads, 0, st>>>(a, segs);
  else if (z_dtype == FLJSD_F32)
    k_lp_grad<float, bf, false><<<grid, kThreads, 0, st>>>(a, segs);
  else
    k_lp_grad<bf, bf, false><<<grid, kThreads, 0, st>>>(a, segs);
  trace_end(FLJSD_KERNEL_JSD_ROWS, st);
  return cudaGetLastError();
}

}  // namespace fljsd
