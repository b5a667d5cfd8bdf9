// The norm of many tensors taken together, and their copies scaled so that it is at
// most max_norm.
//
//   norm = sqrt(sum g^2) or max |g|,  factor = min(1, max_norm / (norm + 1e-6))
//
// Both passes are bound by HBM: one reads every element, the other reads and writes it
// (525M bf16: 156 us = 6.7 TB/s, and with the copies 468 us for 3.15 GB).
// k_norm: every thread takes 64 bytes at a time, squares and adds them in fp32, and CTAs
// write one partial each; k_norm_finish adds the partials in a fixed order in fp64, so
// that a sum has one value whatever the SMs' order. Squares leave fp32's range beyond
// 2^64 and below 2^-63: a thread whose 64 bytes add up to less than 2^-100, or to 2^96 and
// more, takes them again in fp64, which holds the square of every fp32 and the sum of all.
// (2^96: a thread has fewer than 2^31 such sums in a launch, so theirs stays below 2^127.)
// That is rare, so the common path pays two comparisons for 16 or 32 elements.
// k_clip walks from the last chunk to the first: what k_norm has read last is still in L2.
#include "dependent.cuh"
#include "internal.cuh"

#include <cmath>

namespace fljsd {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;                           // 16-byte vectors a thread takes at a time
constexpr int kChunk = kThreads * kVecs * 16;      // bytes a CTA takes at a time
// CTAs of one or few chunks spread their accesses out evenly, as in an AdamW step, but each
// writes a partial sum (525M bf16: norm with 8, 16 and 32 an SM 173, 156 and 160 us, the
// clip's second pass 342, 332 and 312).
constexpr int kNormCtas = 16, kClipCtas = 32;
constexpr int kFew = 64, kMany = 800;              // tensors in a launch

struct Entry {
  const void* src;
  void* dst;
  int64_t n;
};
// Tensors [0, count): tensor i's chunks are numbered first[i] .. first[i + 1). A chunk
// starts on a 16-byte boundary, the first one at or before the tensor's start.
template <int CAP>
struct Table {
  Entry e[CAP];
  int64_t first[CAP + 1];
  unsigned char bf16[CAP];
  int count;
};
static_assert(sizeof(Table<kMany>) <= 32000, "kernel parameters");

// The last tensor that starts at or before chunk c.
template <int CAP>
__device__ __forceinline__ int find(const Table<CAP>& t, int64_t c) {
  int at = 0;
  for (int end = t.count; end - at > 1;) {
    const int mid = (at + end) / 2;
    if (c >= t.first[mid])
      at = mid;
    else
      end = mid;
  }
  return at;
}

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Elements [e0, e0 + 16 bytes) of a tensor of n, as they lie in memory; those outside of
// it read as zeros.
template <typename T>
__device__ __forceinline__ uint4 load16(const T* p, int64_t e0, int64_t n) {
  constexpr int N = 16 / sizeof(T);
  if (e0 >= 0 && e0 + N <= n) return *reinterpret_cast<const uint4*>(p + e0);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (e0 + i >= 0 && e0 + i < n) {
      if (sizeof(T) == 4)
        w[i] = reinterpret_cast<const uint32_t*>(p)[e0 + i];
      else
        w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[e0 + i] << (16 * (i & 1));
    }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The fp32 values of 16 bytes: four, or eight of bf16.
template <bool BF16>
__device__ __forceinline__ void values(const uint4& q, float (&x)[BF16 ? 8 : 4]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      x[2 * i] = lo16(w[i]);
      x[2 * i + 1] = hi16(w[i]);
    } else {
      x[i] = __uint_as_float(w[i]);
    }
  }
}

struct Acc {
  float sum;        // of squares
  double far;       // of squares that fp32 does not hold
  uint32_t top;     // the largest |g|, as its bits (a NaN is above infinity)
};

template <bool BF16, bool MAX>
__device__ __forceinline__ void take(const uint4 (&q)[kVecs], Acc& a) {
  constexpr int N = BF16 ? 8 : 4;
  if (MAX) {
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (BF16) m = max(m, max((w[i] << 16) & 0x7fffffffu, w[i] & 0x7fff0000u));
        else m = max(m, w[i] & 0x7fffffffu);
      }
    }
    a.top = max(a.top, m);
    return;
  }
  float2 s[2] = {};
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    float x[N];
    values<BF16>(q[u], x);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 v = make_float2(x[i], x[i + 1]);
      s[(i / 2) & 1] = __ffma2_rn(v, v, s[(i / 2) & 1]);
    }
  }
  const float c = (s[0].x + s[0].y) + (s[1].x + s[1].y);
  if (c >= 0x1p-100f && c < 0x1p96f) {  // (NaN is not)
    a.sum += c;
  } else {
#pragma unroll 1
    for (int u = 0; u < kVecs; ++u) {
      float x[N];
      values<BF16>(u == 0 ? q[0] : u == 1 ? q[1] : u == 2 ? q[2] : q[3], x);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (x[i] != 0.f) a.far = fma((double)x[i], (double)x[i], a.far);  // (NaN too)
    }
  }
}

template <bool MAX, int CAP>
__global__ void __launch_bounds__(kThreads) k_norm(const __grid_constant__ Table<CAP> t,
                                                   double* __restrict__ partial) {
  __shared__ double sh[kThreads / 32];
  let_next_launch();
  Acc a{0.f, 0.0, 0u};
  int at = 0;
  const int64_t chunks = t.first[t.count];
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    if (c >= t.first[at + 1]) at = find(t, c);
    const Entry& e = t.e[at];
    const int64_t chunk = c - t.first[at];
    uint4 q[kVecs];
    if (t.bf16[at]) {
      const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(e.src);
      const int64_t e0 = chunk * (kChunk / 2) - (int64_t)(((uintptr_t)p & 15u) / 2) + threadIdx.x * 8;
#pragma unroll
      for (int u = 0; u < kVecs; ++u) q[u] = load16(p, e0 + u * kThreads * 8, e.n);
      take<true, MAX>(q, a);
    } else {
      const float* p = reinterpret_cast<const float*>(e.src);
      const int64_t e0 = chunk * (kChunk / 4) - (int64_t)(((uintptr_t)p & 15u) / 4) + threadIdx.x * 4;
#pragma unroll
      for (int u = 0; u < kVecs; ++u) q[u] = load16(p, e0 + u * kThreads * 4, e.n);
      take<false, MAX>(q, a);
    }
  }
  double x = MAX ? (double)__uint_as_float(a.top) : (double)a.sum + a.far;
  auto join = [](double p, double q) {  // (a NaN stays)
    return MAX ? (p != p || p > q ? p : q) : p + q;
  };
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = join(x, __shfl_xor_sync(0xffffffffu, x, o));
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) x = join(x, sh[w]);
    partial[blockIdx.x] = x;
  }
}

constexpr int kFinish = 512;
template <bool MAX>
__global__ void __launch_bounds__(kFinish) k_norm_finish(const double* __restrict__ partial, int n,
                                                         const float* __restrict__ grad_scale,
                                                         float max_norm, float* __restrict__ norm,
                                                         float* __restrict__ factor) {
  __shared__ double sh[kFinish / 32];
  let_next_launch();
  wait_for_previous();
  auto join = [](double p, double q) { return MAX ? (p != p || p > q ? p : q) : p + q; };
  double x = 0.0;
  for (int i = threadIdx.x; i < n; i += kFinish) x = join(x, partial[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = join(x, __shfl_xor_sync(0xffffffffu, x, o));
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kFinish / 32; ++w) x = join(x, sh[w]);
    const float scale = grad_scale ? *grad_scale : 1.f;
    const float v = (float)((MAX ? x : sqrt(x)) * fabs((double)scale));
    *norm = v;
    if (factor) {
      const float f = max_norm / (v + 1e-6f);
      *factor = (f > 1.f ? 1.f : f) * scale;  // (NaN stays)
    }
  }
}

template <typename T>
__device__ __forceinline__ void clip_chunk(const Entry& e, int64_t chunk, float f) {
  constexpr int N = 16 / sizeof(T);
  const T* p = reinterpret_cast<const T*>(e.src);
  T* o = reinterpret_cast<T*>(e.dst);
  const int lead = (int)(((uintptr_t)p & 15u) / sizeof(T));
  const bool vec = (((uintptr_t)p ^ (uintptr_t)o) & 15u) == 0;
  const int64_t e0 = chunk * (kChunk / (int)sizeof(T)) - lead + threadIdx.x * N;
  uint4 q[kVecs];
#pragma unroll
  for (int u = 0; u < kVecs; ++u) q[u] = load16(p, e0 + u * kThreads * N, e.n);
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    const int64_t i0 = e0 + u * kThreads * N;
    float x[N];
    values<sizeof(T) == 2>(q[u], x);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __fmul_rn(x[i], f);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (sizeof(T) == 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[(2 * i) % N], x[(2 * i + 1) % N]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        w[i] = __float_as_uint(x[i]);
      }
    }
    if (vec && i0 >= 0 && i0 + N <= e.n) {
      *reinterpret_cast<uint4*>(o + i0) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i0 + i >= 0 && i0 + i < e.n) {
          if (sizeof(T) == 4)
            reinterpret_cast<uint32_t*>(o)[i0 + i] = w[i];
          else
            reinterpret_cast<uint16_t*>(o)[i0 + i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
        }
    }
  }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) k_clip(const __grid_constant__ Table<CAP> t,
                                                   const float* __restrict__ factor) {
  let_next_launch();
  wait_for_previous();
  const float f = *factor;
  const int64_t chunks = t.first[t.count];
  for (int64_t b = blockIdx.x; b < chunks; b += gridDim.x) {
    const int64_t c = chunks - 1 - b;
    const int at = find(t, c);
    const Entry& e = t.e[at];
    if (f == 1.f && e.src == e.dst) continue;  // as it is
    if (t.bf16[at])
      clip_chunk<__nv_bfloat16>(e, c - t.first[at], f);
    else
      clip_chunk<float>(e, c - t.first[at], f);
  }
}

int ctas(int64_t chunks, int per_sm) {
  const int64_t most = (int64_t)num_sms() * per_sm;
  return (int)(chunks < most ? chunks : most);
}

// Calls `f` with tables of up to CAP tensors each, the first ones first (or last).
template <int CAP, typename F>
cudaError_t each_table(const fljsd_grad_tensor* ts, int count, bool backwards, const F& f) {
  Table<CAP> t;
  const int tables = (count + CAP - 1) / CAP;
  for (int k = 0; k < tables; ++k) {
    const int at = (backwards ? tables - 1 - k : k) * CAP, end = at + CAP < count ? at + CAP : count;
    t.count = 0;
    t.first[0] = 0;
    for (int j = at; j < end; ++j) {
      const fljsd_grad_tensor& x = ts[j];
      if (x.n == 0) continue;
      const int i = t.count++;
      const int64_t size = x.dtype == FLJSD_BF16 ? 2 : 4;
      t.e[i] = Entry{x.grad, x.out, x.n};
      t.bf16[i] = x.dtype == FLJSD_BF16;
      t.first[i + 1] = t.first[i] + (x.n * size + (int64_t)((uintptr_t)x.grad & 15u) + kChunk - 1) / kChunk;
    }
    if (t.count == 0) continue;
    const cudaError_t e = f(t);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <bool MAX, int CAP>
cudaError_t norm_of(const fljsd_grad_tensor* ts, int count, const float* grad_scale, float max_norm,
                    float* norm, float* factor, double* partial, cudaStream_t st) {
  int n = 0;
  cudaError_t e = each_table<CAP>(ts, count, false, [&](const Table<CAP>& t) {
    const int grid = ctas(t.first[t.count], kNormCtas);
    trace_begin(FLJSD_KERNEL_SMALL, st);
    k_norm<MAX, CAP><<<grid, kThreads, 0, st>>>(t, partial + n);
    trace_end(FLJSD_KERNEL_SMALL, st);
    n += grid;
    return cudaGetLastError();
  });
  if (e != cudaSuccess) return e;
  trace_begin(FLJSD_KERNEL_SMALL, st);
  if (n > 0)
    e = launch_dependent(k_norm_finish<MAX>, 1, kFinish, 0, st, (const double*)partial, n, grad_scale,
                         max_norm, norm, factor);
  else  // (nothing of this library before it)
    k_norm_finish<MAX><<<1, kFinish, 0, st>>>(partial, n, grad_scale, max_norm, norm, factor);
  trace_end(FLJSD_KERNEL_SMALL, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int CAP>
cudaError_t norm_any(const fljsd_grad_tensor* ts, int count, int kind, const float* grad_scale,
                     float max_norm, float* norm, float* factor, double* partial, cudaStream_t st) {
  return kind == FLJSD_NORM_MAX
             ? norm_of<true, CAP>(ts, count, grad_scale, max_norm, norm, factor, partial, st)
             : norm_of<false, CAP>(ts, count, grad_scale, max_norm, norm, factor, partial, st);
}

template <int CAP>
cudaError_t clip_all(const fljsd_grad_tensor* ts, int count, const float* factor, cudaStream_t st) {
  return each_table<CAP>(ts, count, true, [&](const Table<CAP>& t) {
    trace_begin(FLJSD_KERNEL_SMALL, st);
    const cudaError_t e =
        launch_dependent(k_clip<CAP>, ctas(t.first[t.count], kClipCtas), kThreads, 0, st, t, factor);
    trace_end(FLJSD_KERNEL_SMALL, st);
    return e;
  });
}

fljsd_status check(const fljsd_grad_tensor* ts, int32_t count, int32_t kind, const float* grad_scale,
                   const float* norm, const float* factor, const void* ws, size_t ws_bytes, bool out) {
  if (count < 0 || (count > 0 && !ts) || !norm || !ws) return FLJSD_ERR_INVALID_ARG;
  if (kind != FLJSD_NORM_2 && kind != FLJSD_NORM_MAX) return FLJSD_ERR_INVALID_ARG;
  if ((((uintptr_t)grad_scale | (uintptr_t)norm | (uintptr_t)factor) & 3u) || ((uintptr_t)ws & 15u))
    return FLJSD_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i) {
    const fljsd_grad_tensor& t = ts[i];
    if (t.n < 0 || (t.dtype != FLJSD_F32 && t.dtype != FLJSD_BF16)) return FLJSD_ERR_INVALID_ARG;
    if (t.n == 0) continue;
    const uintptr_t al = t.dtype == FLJSD_BF16 ? 1 : 3;
    if (!t.grad || ((uintptr_t)t.grad & al)) return FLJSD_ERR_INVALID_ARG;
    if (out && (!t.out || ((uintptr_t)t.out & al))) return FLJSD_ERR_INVALID_ARG;
    if (t.n > (int64_t)1 << 40) return FLJSD_ERR_UNSUPPORTED;
  }
  return ws_bytes < fljsd_grad_norm_workspace_bytes(count) ? FLJSD_ERR_WORKSPACE : FLJSD_OK;
}

constexpr size_t kFactorBytes = 16;  // in front of the partials

}  // namespace
}  // namespace fljsd

using namespace fljsd;

extern "C" size_t fljsd_grad_norm_workspace_bytes(int32_t count) {
  const size_t tables = count <= kFew ? 1 : (count + kMany - 1) / kMany;
  return kFactorBytes + tables * num_sms() * kNormCtas * sizeof(double);
}

extern "C" fljsd_status fljsd_grad_norm(const fljsd_grad_tensor* tensors, int32_t count, int32_t kind,
                                        float max_norm, const float* grad_scale, float* norm,
                                        float* factor, void* workspace, size_t workspace_bytes,
                                        fljsd_stream_t stream) {
  const fljsd_status s = check(tensors, count, kind, grad_scale, norm, factor, workspace,
                               workspace_bytes, false);
  if (s != FLJSD_OK) return s;
  if (factor && !(max_norm >= 0)) return FLJSD_ERR_INVALID_ARG;
  double* partial = reinterpret_cast<double*>(reinterpret_cast<char*>(workspace) + kFactorBytes);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      count <= kFew ? norm_any<kFew>(tensors, count, kind, grad_scale, max_norm, norm, factor, partial, st)
                    : norm_any<kMany>(tensors, count, kind, grad_scale, max_norm, norm, factor, partial, st);
  return e == cudaSuccess ? FLJSD_OK : FLJSD_ERR_CUDA;
}

extern "C" fljsd_status fljsd_clip_grads(const fljsd_grad_tensor* tensors, int32_t count, int32_t kind,
                                         float max_norm, float* norm, void* workspace,
                                         size_t workspace_bytes, fljsd_stream_t stream) {
  const fljsd_status s = check(tensors, count, kind, nullptr, norm, nullptr, workspace,
                               workspace_bytes, true);
  if (s != FLJSD_OK) return s;
  if (!(max_norm >= 0)) return FLJSD_ERR_INVALID_ARG;
  float* factor = reinterpret_cast<float*>(workspace);
  const fljsd_status n = fljsd_grad_norm(tensors, count, kind, max_norm, nullptr, norm, factor,
                                         workspace, workspace_bytes, stream);
  if (n != FLJSD_OK) return n;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = count <= kFew ? clip_all<kFew>(tensors, count, factor, st)
                                      : clip_all<kMany>(tensors, count, factor, st);
  return e == cudaSuccess ? FLJSD_OK : FLJSD_ERR_CUDA;
}
