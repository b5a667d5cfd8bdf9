// Token log probabilities: parts of given logits, the join of a row's parts,
// and the gradient in the logits. The formulas are in lp.cuh.
//
// k_lp_rows cuts each row into segments of 8192 logits, one CTA each, so that a
// single row of 128256 still runs on 16 CTAs (of many rows of bf16 a CTA takes up to
// four segments: k_lp_rows_many); the next segment is on its way while one is
// reduced. The k largest are left to k_lp_join, which reads again the few 256s whose
// maxima reach the k-th largest of them (2047 x 128255 bf16, 8 alternatives: 28 us).
// k_lp_grad is elementwise. HBM bounds both for fp32 (1023 x 128255: 80 us = 6.6 TB/s, the
// gradient 160 us = 6.5 TB/s, 0.97 of a copy's rate) and nearly so for bf16, with twice
// the elements to a byte (2047 x 128255: 84 us = 6.2 TB/s, the gradient 165 us = 6.3 TB/s).
#include "dependent.cuh"
#include "lp.cuh"
#include "lp_mds.cuh"
#include "jsd_math.cuh"

#include <cuda_fp16.h>

#include <type_traits>

namespace fljsd {
namespace {

using namespace rowmath;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = LP_SEG / kThreads;  // logits a thread holds
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kQuarters = LP_CHUNKS / kWarps;  // of a warp's vectors, a maximum for each
static_assert(kQuarters == 4, "one 16-byte store");
// Threads of a row's join: few rows are bound by one CTA's way through its loads (333
// fused rows, 20 alternatives: 512 threads 16 us, 256 threads 19), many by how many
// CTAs an SM holds (given logits, 8 alternatives: 2047 rows of 128255 with 64, 128 and
// 256 threads 26, 34 and 45 us, 1000 rows of 50001 21, 18 and 22).
constexpr int kJoinFew = 512, kJoinMany = 128;
constexpr int kJoinCap = 1024;  // candidates ranked in shared memory
// as they are; more are sifted first (2000 x 1003, 20 alternatives: 359 us, sifted 25)
constexpr int kJoinMost = 192;
static_assert(kJoinFew <= kJoinCap && kJoinMany >= LP_MAX_TOP, "the threads' largest");

__device__ __forceinline__ float val(const float* p) { return *p; }
__device__ __forceinline__ float val(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float val(const __half* p) { return __half2float(*p); }

// Eight values, 16-byte aligned.
__device__ __forceinline__ void store8(float* p, const float (&o)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(o[0], o[1], o[2], o[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(o[4], o[5], o[6], o[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&o)[8]) {
  Vec<__nv_bfloat16>::store(p, o);
}

// 16 bytes of logits as they lie in memory, and their values.
template <typename T>
struct Raw {
  uint4 w;
};
template <typename T>
__device__ __forceinline__ void values(const Raw<T>& q, float* z);
template <>
__device__ __forceinline__ void values(const Raw<float>& q, float* z) {
  z[0] = __uint_as_float(q.w.x);
  z[1] = __uint_as_float(q.w.y);
  z[2] = __uint_as_float(q.w.z);
  z[3] = __uint_as_float(q.w.w);
}
template <>
__device__ __forceinline__ void values(const Raw<__nv_bfloat16>& q, float* z) {
  const uint32_t w[4] = {q.w.x, q.w.y, q.w.z, q.w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    z[2 * i] = __uint_as_float(w[i] << 16);
    z[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void values(const Raw<__half>& q, float* z) {
  const uint32_t w[4] = {q.w.x, q.w.y, q.w.z, q.w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    z[2 * i] = f.x;
    z[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ uint32_t bits_of(const float* p) { return __float_as_uint(*p); }
__device__ __forceinline__ uint32_t bits_of(const __nv_bfloat16* p) {
  return *reinterpret_cast<const uint16_t*>(p);
}
__device__ __forceinline__ uint32_t bits_of(const __half* p) {
  return *reinterpret_cast<const uint16_t*>(p);
}
// The 16 bytes at element j of a segment whose elements [first, n) exist; the others
// read as `none` (the bits of one element).
template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* zs, int j, int first, int n, uint32_t none) {
  constexpr int N = 16 / sizeof(T);
  Raw<T> q;
  if (j >= first && j + N <= n) {
    q.w = *reinterpret_cast<const uint4*>(zs + j);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (sizeof(T) == 4) {
        w[i] = j + i >= first && j + i < n ? bits_of(zs + j + i) : none;
      } else {
        const int a = j + 2 * i, b = a + 1;
        w[i] = (a >= first && a < n ? bits_of(zs + a) : none) |
               ((b >= first && b < n ? bits_of(zs + b) : none) << 16);
      }
    }
    q.w = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return q;
}

// Where a segment of a row lies: elements [first, n) of zs, which starts on a 16-byte
// boundary (lead elements before the row in its first segment).
template <typename T>
struct Segment {
  const T* zs;
  int64_t e0;  // the row's element at zs
  int first, n;
  __device__ __forceinline__ Segment(const void* z, int64_t ld, int64_t r, int64_t v, int64_t part) {
    const T* zr = reinterpret_cast<const T*>(z) + r * ld;
    const int lead = (int)((((uintptr_t)zr) & 15u) / sizeof(T));
    e0 = part * LP_SEG - lead;
    n = (int)(v - e0 < LP_SEG ? (v > e0 ? v - e0 : 0) : LP_SEG);
    first = e0 < 0 ? lead : 0;
    zs = zr + e0;
  }
};

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

// The block's, in a fixed order (in every thread of the first warp).
template <int W>
__device__ __forceinline__ Mds block_mds(Mds x, float c, Mds* sh) {
  x = warp_mds(x, c);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
  __syncthreads();
  if (threadIdx.x < 32) {
    x = threadIdx.x < W ? sh[threadIdx.x] : Mds{-INFINITY, 0.f, 0.f};
    x = warp_mds(x, c);
  }
  return x;
}

// The largest of a thread's logits (NaN passed over) and, where `keep` is set, the warp's
// largest of each quarter of them.
__device__ __forceinline__ float largest(const float (&z)[kPer], float* keep) {
  float m[kQuarters];
#pragma unroll
  for (int q = 0; q < kQuarters; ++q) {
    m[q] = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPer / kQuarters; ++i) m[q] = fmaxf(m[q], z[q * (kPer / kQuarters) + i]);
  }
  const float all = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
  if (keep) {
#pragma unroll
    for (int q = 0; q < kQuarters; ++q)
      asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m[q]) : "f"(m[q]));
    if ((threadIdx.x & 31) == 0) *reinterpret_cast<float4*>(keep) = make_float4(m[0], m[1], m[2], m[3]);
  }
  return all;
}

// {sum 2^t, sum 2^t t} of a thread's logits, t = c (z - m).
__device__ __forceinline__ float2 sums_of(const float (&z)[kPer], float m, float c) {
  // t = c z - c ref in one operation: c ref = hi + lo, hi rounded, and the sums
  // are put right for lo once (2^-lo, and s - lo d)
  const float ref = m == -INFINITY ? 0.f : m;
  const float hi = __fmul_rn(ref, c), lo = __fmaf_rn(ref, c, -hi);
  const float2 c2 = make_float2(c, c), nhi = make_float2(-hi, -hi);
  float2 d = make_float2(0.f, 0.f), t = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kPer; i += 2) {
    const float2 q = __ffma2_rn(make_float2(z[i], z[i + 1]), c2, nhi);
    const float2 y = make_float2(ex2(q.x), ex2(q.y));
    d = __fadd2_rn(d, y);
    t = __ffma2_rn(y, q, t);
  }
  const float f = ex2(-lo);
  float2 o = make_float2((d.x + d.y) * f, __fmaf_rn(-lo, d.x + d.y, t.x + t.y) * f);
  if (!(fabsf(o.y) < INFINITY && fabsf(lo) <= 64.f)) {
    // a logit of -inf or near the type's lowest (0 times -inf above), a maximum
    // that overflows c, a maximum so far out (2^30 and more) that 2^lo may vanish
    // beside a finite 2^-lo, or NaN, which stays: with the difference taken first
    o = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float q = __fmul_rn(z[i] - ref, c), y = ex2(q);
      o.x += y;
      o.y = __fmaf_rn(y, fmaxf(q, -1024.f), o.y);
    }
  }
  return o;
}

// A segment's logits, 32 to a thread: vectors of N elements, kThreads vectors
// apart, from a 16-byte boundary. The vector that starts before the row (whose
// first element may lie anywhere) and the one that crosses its end are read one
// element at a time. Sums are taken relative to each thread's own maximum, so
// that one reduction serves maximum and sums.
template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 3 : 4) k_lp_rows(LpRowsArgs a, int64_t parts) {
  constexpr int N = Vec<T>::N;
  constexpr int V = kPer / N;
  __shared__ Mds shm[kWarps];
  const int tid = threadIdx.x;
  const int64_t part = blockIdx.x;
  constexpr uint32_t kNone = sizeof(T) == 4 ? 0xff800000u : 0xff80u;  // -inf
  let_next_launch();
  wait_for_previous();
  if (a.status && part == 0 && blockIdx.y == 0 && tid == 0) *a.status = 0;
  Raw<T> raw[V];
  auto load = [&](int64_t r) {
    const Segment<T> g(a.z, a.ld, r, a.v, part);
    if (g.first == 0 && g.n == LP_SEG) {
#pragma unroll
      for (int u = 0; u < V; ++u)
        raw[u].w = *reinterpret_cast<const uint4*>(g.zs + (u * kThreads + tid) * N);
    } else {
#pragma unroll
      for (int u = 0; u < V; ++u)
        raw[u] = load_raw(g.zs, (u * kThreads + tid) * N, g.first, g.n, kNone);
    }
  };
  if (blockIdx.y < a.rows) load(blockIdx.y);
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    float z[kPer];
#pragma unroll
    for (int u = 0; u < V; ++u) values(raw[u], z + u * N);
    // the next row's segment is on its way while this one is reduced
    if (r + gridDim.y < a.rows) load(r + gridDim.y);
    float* keep = a.cmax ? a.cmax + ((r * parts + part) * kWarps + (tid >> 5)) * kQuarters : nullptr;
    Mds x{largest(z, keep), 0.f, 0.f};
    const float2 ds = sums_of(z, x.m, a.c);
    x.d = ds.x;
    x.s = ds.y;
    x = block_mds<kWarps>(x, a.c, shm);
    if (tid == 0) {
      a.part[r * parts + part] = make_float4(x.m, x.d, x.s, 0.f);
      if (a.labels && part == 0) {
        const int64_t y = a.labels[a.row0 + r];
        if (y >= 0 && y < a.v) a.zy[r] = val(reinterpret_cast<const T*>(a.z) + r * a.ld + y);
      }
    }
    __syncthreads();  // the shared results are written again by the next row
  }
}

// The same for many rows of bf16, where the block's reduction took a third of the
// instructions: a CTA takes `group` segments of a row into each thread's running sums and
// reduces them once (2047 x 128255: 84 us = 6.2 TB/s with four, 99.5 with a reduction for
// each; fp32, bound by HBM, 84 and 80). 64 registers a thread are all but full, and a few
// values that do not fit cost more than the reductions did: rows are counted in 32 bits.
__global__ void __launch_bounds__(kThreads, 4) k_lp_rows_many(LpRowsArgs a) {
  using T = __nv_bfloat16;
  constexpr int N = Vec<T>::N;
  constexpr int V = kPer / N;
  __shared__ Mds shm[kWarps];
  const int tid = threadIdx.x;
  const unsigned part = blockIdx.x;
  constexpr uint32_t kNone = 0xff80u;  // -inf
  let_next_launch();
  if (a.status && part == 0 && blockIdx.y == 0 && tid == 0) *a.status = 0;
  const int seg0 = part * a.group;
  const int count = seg0 + a.group < a.segs ? a.group : a.segs - seg0;
  // the next segment to ask for: its elements [lead, left) lie from zs on
  const int rows = (int)a.rows;
  int rl = blockIdx.y;
  const T* zs = nullptr;
  int lead = 0, left = 0, more = 0;
  Raw<T> raw[V];
  auto ask = [&]() {
    if (rl < rows) {
      if (more == 0) {
        const T* zr = reinterpret_cast<const T*>(a.z) + (int64_t)rl * a.ld;
        const int before = (int)((((uintptr_t)zr) & 15u) / sizeof(T));
        zs = zr - before + (int64_t)seg0 * LP_SEG;
        lead = seg0 == 0 ? before : 0;
        left = (int)a.v + before - seg0 * LP_SEG;
        more = count;
      }
      if (lead == 0 && left >= LP_SEG) {
#pragma unroll
        for (int u = 0; u < V; ++u)
          raw[u].w = *reinterpret_cast<const uint4*>(zs + (u * kThreads + tid) * N);
      } else {
#pragma unroll
        for (int u = 0; u < V; ++u)
          raw[u] = load_raw(zs, (u * kThreads + tid) * N, lead, left < LP_SEG ? left : LP_SEG, kNone);
      }
      zs += LP_SEG;
      left -= LP_SEG;
      lead = 0;
      if (--more == 0) rl += gridDim.y;
    }
  };
  ask();
  for (int r = blockIdx.y; r < rows; r += gridDim.y) {
    Mds x{-INFINITY, 0.f, 0.f};
    for (int seg = 0; seg < count; ++seg) {
      float z[kPer];
#pragma unroll
      for (int u = 0; u < V; ++u) values(raw[u], z + u * N);
      ask();
      float* keep = a.cmax ? a.cmax + (((int64_t)r * a.segs + seg0 + seg) * kWarps + (tid >> 5)) * kQuarters
                           : nullptr;
      float m = largest(z, keep);
      m = fmaxf(m, x.m);
      const float2 ds = sums_of(z, m, a.c);
      // the thread's sums so far, relative to the new maximum
      const float u = x.m == -INFINITY ? 0.f : __fmul_rn(x.m - m, a.c), fu = ex2(u);
      x = Mds{m, __fmaf_rn(x.d, fu, ds.x), __fmaf_rn(fu, __fmaf_rn(x.d, fmaxf(u, -1024.f), x.s), ds.y)};
      __syncwarp();  // (keeps the loads and conversions of the next one behind these sums)
    }
    x = block_mds<kWarps>(x, a.c, shm);
    if (tid == 0) {
      a.part[(int64_t)r * gridDim.x + part] = make_float4(x.m, x.d, x.s, 0.f);
      if (a.labels && part == 0) {
        const int64_t y = a.labels[a.row0 + r];
        if (y >= 0 && y < a.v) a.zy[r] = val(reinterpret_cast<const T*>(a.z) + (int64_t)r * a.ld + y);
      }
    }
    __syncthreads();  // the shared results are written again by the next row
  }
}

// CTAs an SM that the registers leave room for. The product's lists take 40 registers at
// no loss (333 rows, 20 alternatives: three CTAs of 512 threads 14 us, two 17; 4096 rows:
// twelve of 128 threads 29 us, eight 33); the loads from given logits would spill.
template <typename SRC, int THREADS>
constexpr int kJoinCtas = std::is_same<SRC, void>::value ? (THREADS == kJoinFew ? 3 : 12)
                                                         : (THREADS == kJoinFew ? 2 : 8);
// One CTA to a row: its parts into the row's results, its candidates into the
// k largest. SRC: where the candidates are; void: lists and written-out logits of
// the product, else given logits of that type.
template <typename SRC, int kJoinThreads>
__global__ void __launch_bounds__(kJoinThreads, (kJoinCtas<SRC, kJoinThreads>)) k_lp_join(LpJoinArgs a) {
  constexpr bool kRowsSrc = !std::is_same<SRC, void>::value;
  constexpr int W = kJoinThreads / 32;
  __shared__ Mds shm[W];
  __shared__ float2 sh_norm;
  __shared__ unsigned long long sh64[W];
  __shared__ unsigned long long list[kJoinCap];
  __shared__ unsigned keys[kJoinThreads];
  __shared__ int n_list;
  __shared__ unsigned sh_least;
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x, out = a.row0 + r;
  wait_for_previous();
  const float4* ps = a.part + r * a.parts;
  // four parts in flight a thread
  Mds x{-INFINITY, 0.f, 0.f};
  for (int64_t i0 = tid; i0 < a.parts; i0 += 4 * kJoinThreads) {
    float4 q[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t i = i0 + u * kJoinThreads;
      q[u] = i < a.parts ? ps[i] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) x = merge(x, Mds{q[u].x, q[u].y, q[u].z}, a.c);
  }
  if (tid == 0) n_list = 0;
  x = block_mds<W>(x, a.c, shm);
  const float m = x.m;  // (in the first warp)
  const float2 ds = make_float2(x.d, x.s);
  // a row without a finite logit has d = 0: lse = -inf, entropy 0
  const bool empty = ds.x == 0.f;
  const float l2d = empty ? 0.f : log2f(ds.x);
  // not through log2 units, in which the type's lowest value overflows
  auto log_p = [&](float z, float2 norm) {
    return __fmaf_rn(z - norm.x, a.inv_t, -kLn2 * norm.y);
  };
  if (tid == 0) {
    a.lse[out] = empty ? -INFINITY : __fmaf_rn(m, a.inv_t, kLn2 * l2d);
    a.norm[out] = sh_norm = make_float2(empty ? -INFINITY : m, l2d);
    const int64_t y = a.labels ? a.labels[out] : 0;
    bool live = true;
    if (a.labels) {
      live = y != a.ignore_index;
      if (live && (y < 0 || y >= a.v)) {
        live = false;
        atomicExch(a.status, (int)FLJSD_ERR_INVALID_ARG);
      }
      float lp = 0.f;
      if (live) lp = empty ? -INFINITY : log_p(a.zy[r], make_float2(m, l2d));
      a.logp[out] = lp;
    }
    a.entropy[out] = live && !empty ? kLn2 * (l2d - ds.y / ds.x) : 0.f;
  }
  if (a.k == 0) return;
  // ---- the k largest candidates ----
  // a value that at least k of the first n threads' values reach: the k-th largest of
  // them, or, of more than 128, of the largest of each four (0 if fewer are above 0)
  auto kth_of_threads = [&](unsigned mine, int n) {
    if (tid == 0) sh_least = 0;
    int gt = 0, ge = 0;
    if constexpr (kJoinThreads == kJoinFew) {
      if (n > kJoinFew / 4) {
        mine = max(mine, __shfl_xor_sync(0xffffffffu, mine, 1));
        mine = max(mine, __shfl_xor_sync(0xffffffffu, mine, 2));
        if ((tid & 3) == 0) keys[tid >> 2] = mine;
        n = (n + 3) / 4;
      } else if (tid < n) {
        keys[tid] = mine;
      }
      __syncthreads();
      // four threads to a value, each against a quarter of them
      if ((tid >> 2) < n) {
        const unsigned quad = 0xfu << (tid & 28), x = keys[tid >> 2];
#pragma unroll 8
        for (int j = tid & 3; j < n; j += 4) {
          gt += keys[j] > x ? 1 : 0;
          ge += keys[j] >= x ? 1 : 0;
        }
#pragma unroll
        for (int o = 2; o > 0; o >>= 1) {
          gt += __shfl_xor_sync(quad, gt, o);
          ge += __shfl_xor_sync(quad, ge, o);
        }
        if ((tid & 3) == 0 && gt < a.k && a.k <= ge) sh_least = x;  // (equal ones write the same)
      }
    } else {
      keys[tid] = mine;
      __syncthreads();
#pragma unroll 8
      for (int j = 0; j < n; ++j) {
        gt += keys[j] > mine ? 1 : 0;
        ge += keys[j] >= mine ? 1 : 0;
      }
      if (tid < n && gt < a.k && a.k <= ge) sh_least = mine;
    }
    __syncthreads();
    return sh_least;
  };
  unsigned least = 0;
  const bool few = kRowsSrc && a.few_chunks > 0;  // chunks: 32 columns of a product of few rows
  const int64_t chunks = few ? a.few_chunks : a.segs * LP_CHUNKS;
  const float* cmax = a.cmax + r * chunks;
  const int64_t n_cand = kRowsSrc ? 0 : (int64_t)a.count[r];
  const int2* cand = a.cand + r * a.cap;
  const float* dump = a.dump + r * a.dump_cols;
  const unsigned n_dump = !kRowsSrc && a.dump ? (unsigned)a.dump_cols : 0u;
  if (kRowsSrc) {
    unsigned mine = 0;
#pragma unroll 4
    for (int64_t i = tid; i < chunks; i += kJoinThreads) {
      const float m1 = cmax[i];
      if (m1 > -INFINITY) mine = max(mine, lp_key(m1));
    }
    least = kth_of_threads(mine, (int)(chunks < kJoinThreads ? chunks : kJoinThreads));
  } else {
    const int lane = tid & 31;  // (k is at most 32)
    least = __reduce_min_sync(0xffffffffu, lane < a.k ? a.gmax[lane * a.rows + r] : 0xffffffffu);
  }
  // every candidate's key that reaches `least`
  auto each = [&](auto&& f) {
    const float lo = least > 0x007fffffu ? key_value((unsigned long long)least << 32) : -INFINITY;
    auto give = [&](float z, int64_t col) {
      if (z >= lo && z > -INFINITY) f(cand_key(make_int2(__float_as_int(z), (int)col)));
    };
    if constexpr (kRowsSrc) {
      constexpr int N = 16 / sizeof(SRC);
      constexpr uint32_t kNone = sizeof(SRC) == 4 ? 0xff800000u : 0xff80u;  // -inf
      constexpr int V = kPer / N / kQuarters;  // vectors behind a kept maximum
      const SRC* zr = reinterpret_cast<const SRC*>(a.z) + r * a.ld;
      // every lane a chunk's maximum, the warp those chunks that reach it
      for (int64_t c0 = tid >> 5; c0 < chunks; c0 += 4 * 32 * W) {
        float m1[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int64_t c = c0 + (u * 32 + (tid & 31)) * W;
          m1[u] = c < chunks ? cmax[c] : -INFINITY;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          unsigned hit = __ballot_sync(0xffffffffu, m1[u] > -INFINITY && lp_key(m1[u]) >= least);
          for (; hit; hit &= hit - 1) {
            const int64_t c = c0 + (u * 32 + __ffs(hit) - 1) * W;
            if (few) {
              const int64_t col = c * LP_FEW_COLS + (tid & 31);
              if (col < a.v) give(val(zr + col), col);
              continue;
            }
            const Segment<SRC> g(a.z, a.ld, r, a.v, c / LP_CHUNKS);
            const int w = (int)(c % LP_CHUNKS);  // warp w / 4's vectors, quarter w % 4
            const int j0 = ((w % kQuarters) * V * kThreads + w / kQuarters * 32 + (tid & 31)) * N;
            Raw<SRC> raw[V];
#pragma unroll
            for (int v = 0; v < V; ++v)
              raw[v] = load_raw(g.zs, v * kThreads * N + j0, g.first, g.n, kNone);
#pragma unroll
            for (int v = 0; v < V; ++v) {
              float z[N];
              values(raw[v], z);
#pragma unroll
              for (int i = 0; i < N; ++i) give(z[i], g.e0 + v * kThreads * N + j0 + i);
            }
          }
        }
      }
    } else {
#pragma unroll 4
      for (int64_t i = tid; i < n_cand; i += kJoinThreads) {
        const int2 q = cand[i];
        give(__int_as_float(q.x), q.y);
      }
      // (columns past the part's or the vocabulary's hold nothing)
#pragma unroll 4
      for (unsigned i = tid * 4; i < n_dump; i += kJoinThreads * 4) {
        const float4 q = *reinterpret_cast<const float4*>(dump + i);
        const unsigned off = i % LP_PART_COLS, col = i / LP_PART_COLS * (unsigned)a.part_cols + off;
        if (off >= (unsigned)a.part_cols) continue;  // (a multiple of 8)
        if (col < a.v) give(q.x, col);
        if (col + 1 < a.v) give(q.y, col + 1);
        if (col + 2 < a.v) give(q.z, col + 2);
        if (col + 3 < a.v) give(q.w, col + 3);
      }
    }
  };
  auto gather = [&]() {
    each([&](unsigned long long key) {
      const int at = atomicAdd(&n_list, 1);
      if (at < kJoinCap) list[at] = key;
    });
  };
  gather();
  __syncthreads();
  if (n_list > kJoinCap) {
    // no threshold, or many equal logits: the k-th largest of the threads' own
    // largest bounds the k-th largest from below, ties apart
    unsigned long long mine = 0;
    each([&](unsigned long long key) { mine = key > mine ? key : mine; });
    __syncthreads();
    least = max(least, kth_of_threads((unsigned)(mine >> 32), kJoinThreads));
    if (tid == 0) n_list = 0;
    __syncthreads();
    gather();
    __syncthreads();
  }
  if (n_list > kJoinMost && n_list <= kJoinCap) {
    // ranking takes each against each: first leave out what cannot be among the k largest
    constexpr int PER = kJoinCap / kJoinThreads;
    const int have = n_list;
    unsigned long long mine[PER], best = 0;
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int i = u * kJoinThreads + tid;
      mine[u] = i < have ? list[i] : 0;
      best = mine[u] > best ? mine[u] : best;
    }
    const unsigned lo = kth_of_threads((unsigned)(best >> 32), have < kJoinThreads ? have : kJoinThreads);
    if (tid == 0) n_list = 0;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < PER; ++u)
      if (mine[u] != 0 && (unsigned)(mine[u] >> 32) >= lo) list[atomicAdd(&n_list, 1)] = mine[u];
    __syncthreads();
  }
  const int n = n_list;
  const float2 norm = sh_norm;
  float* tl = a.top_logp + out * a.k;
  int64_t* ti = a.top_id + out * a.k;
  auto put = [&](int q, unsigned long long key) {
    tl[q] = key ? log_p(key_value(key), norm) : -INFINITY;
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
    each([&](unsigned long long key) { best = key < last && key > best ? key : best; });
    best = block_max64<W>(best, sh64);
    if (tid == 0) put(q, best);
    last = best;
  }
}

// One CTA to a segment of a row, in vectors of eight where the logits and their
// gradient lie alike relative to a 16-byte boundary (rows of odd length start
// anywhere, but both at the same place), else one element at a time.
//   dz_j = -p (a + b (log p + entropy)) = -p (b ln2 log2 p + (a + b entropy))
// with log2 p = c (z - m) - log2 d, or, from 2^t, t + c (m of its part - m) - log2 d.
// All loads of a thread are issued before the first is used; four CTAs an SM keep
// enough of them in flight (the next row's loads before this one's arithmetic, with
// three CTAs: 190 us where this takes 167, 2047 x 128255 bf16, 0.93 of HBM).
template <typename TI, typename TO, bool FROM_E>
__global__ void __launch_bounds__(kThreads, 4) k_lp_grad(LpGradArgs a) {
  constexpr int N = 8, U = LP_SEG / (kThreads * N), R = N * sizeof(TI) / 16;
  const int tid = threadIdx.x;
  Raw<TI> raw[U][R];
  float top[U];  // (FROM_E) the maximum of the vector's part
  auto lies_alike = [&](int64_t r) {
    const TI* zr = reinterpret_cast<const TI*>(a.z) + r * a.ldz;
    const TO* orow = reinterpret_cast<const TO*>(a.out) + r * a.ldo;
    return ((uintptr_t)zr & 15u) / sizeof(TI) == ((uintptr_t)orow & 15u) / sizeof(TO);
  };
  auto load = [&](int64_t r) {
    if (!lies_alike(r)) return;
    const Segment<TI> g(a.z, a.ldz, r, a.v, blockIdx.x);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = (u * kThreads + tid) * N;
      if (g.first == 0 && g.n == LP_SEG) {
#pragma unroll
        for (int q = 0; q < R; ++q)
          raw[u][q].w = *reinterpret_cast<const uint4*>(g.zs + j + q * (N / R));
      } else {
#pragma unroll
        for (int q = 0; q < R; ++q) raw[u][q] = load_raw(g.zs, j + q * (N / R), g.first, g.n, 0u);
      }
      if (FROM_E) top[u] = j < g.n ? a.part[r * a.parts + (g.e0 + j) / LP_PART_COLS].x : 0.f;
    }
  };
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    load(r);
    TO* orow = reinterpret_cast<TO*>(a.out) + r * a.ldo;
    const int64_t row = a.row0 + r;
    const int64_t y = a.labels ? a.labels[row] : -1;
    const float2 norm = a.norm[row];
    // (a row of NaN is no empty row: its gradient is NaN)
    const bool live = (!a.labels || (y != a.ignore_index && y >= 0 && y < a.v)) &&
                      !(norm.x == -INFINITY && norm.y == 0.f);
    const float ga = a.grad_logp && a.labels ? a.grad_logp[row] * a.inv_t : 0.f;
    const float gb = a.grad_entropy ? a.grad_entropy[row] * a.inv_t : 0.f;
    const float ent = a.entropy[row];
    const float bl = -gb * kLn2, ab = -__fmaf_rn(gb, ent, ga);
    const bool alike = lies_alike(r);
    const Segment<TI> g(a.z, a.ldz, r, a.v, blockIdx.x);
    // (rows that do not lie alike: segments from the row's own start)
    const int64_t e0 = alike ? g.e0 : (int64_t)blockIdx.x * LP_SEG;
    const int n = alike ? g.n : (int)(a.v - e0 < LP_SEG ? (a.v > e0 ? a.v - e0 : 0) : LP_SEG);
    const int first = alike ? g.first : 0;
    TO* os = orow + e0;
    // two at a time; -inf: p = 0 and p log p = 0
    auto two = [&](float za, float zb, float ref) {
      float2 lp2;
      if (FROM_E)
        lp2 = __fadd2_rn(make_float2(lg2(za), lg2(zb)), make_float2(ref, ref));
      else
        lp2 = __ffma2_rn(__fadd2_rn(make_float2(za, zb), make_float2(-norm.x, -norm.x)),
                         make_float2(a.c, a.c), make_float2(-norm.y, -norm.y));
      const float2 t = __ffma2_rn(make_float2(fmaxf(lp2.x, -1024.f), fmaxf(lp2.y, -1024.f)),
                                  make_float2(bl, bl), make_float2(ab, ab));
      return __fmul2_rn(make_float2(ex2(lp2.x), ex2(lp2.y)), t);
    };
    if (alike) {
      float z[U][N], ref[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int q = 0; q < R; ++q) values(raw[u][q], z[u] + q * (N / R));
        ref[u] = FROM_E ? __fmul_rn(top[u] - norm.x, a.c) - norm.y : 0.f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = (u * kThreads + tid) * N;
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          const float2 o = live ? two(z[u][e], z[u][e + 1], ref[u]) : make_float2(0.f, 0.f);
          z[u][e] = o.x;
          z[u][e + 1] = o.y;
        }
        if (j >= first && j + N <= n) {
          store8(os + j, z[u]);
        } else {
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (j + e >= first && j + e < n) Vec<TO>::put(os + j + e, z[u][e]);
        }
      }
    } else {
      const TI* zs = reinterpret_cast<const TI*>(a.z) + r * a.ldz + e0;
      for (int j = tid; j < n; j += kThreads) {
        const float z = val(zs + j);
        Vec<TO>::put(os + j, live ? two(z, z, 0.f).x : 0.f);
      }
    }
    // The label's own element from its fp32 log probability (1 - p_y would lose its
    // digits to a rounded p_y), written over what the loop left there.
    if (live && a.labels && y >= e0 + first && y < e0 + n) {
      __syncthreads();
      if (tid == 0) {
        const float lp = a.logp[row];
        Vec<TO>::put(orow + y, __fmaf_rn(-ex2(lp * (1.f / kLn2)),
                                         __fmaf_rn(gb, fmaxf(lp, -1024.f) + ent, ga), ga));
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads) k_zero(uint4* to, int64_t n) {
  let_next_launch();
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads)
    to[i] = make_uint4(0u, 0u, 0u, 0u);
}

// x: segments of a row; y: rows, up to what keeps the GPU full (a CTA then walks on)
dim3 row_grid(int64_t segs, int64_t rows) {
  const int64_t most = ((int64_t)num_sms() * 32 + segs - 1) / segs;
  const int64_t y = rows < most ? rows : most;
  return dim3((unsigned)segs, (unsigned)(y < 65535 ? y : 65535));
}

template <int THREADS>
cudaError_t launch_join_t(const LpJoinArgs& a, cudaStream_t st) {
  const unsigned grid = (unsigned)a.rows;
  if (!a.z)
    return launch_dependent(k_lp_join<void, THREADS>, grid, THREADS, 0, st, a);
  if (a.z_dtype == FLJSD_BF16)
    return launch_dependent(k_lp_join<__nv_bfloat16, THREADS>, grid, THREADS, 0, st, a);
  return launch_dependent(k_lp_join<float, THREADS>, grid, THREADS, 0, st, a);
}

}  // namespace

cudaError_t launch_lp_join(const LpJoinArgs& a, cudaStream_t st) {
  if (a.rows <= 0) return cudaSuccess;
  trace_begin(FLJSD_KERNEL_SMALL, st);
  const cudaError_t e = a.rows <= num_sms() * 4 ? launch_join_t<kJoinFew>(a, st)  // 512 threads
                                                : launch_join_t<kJoinMany>(a, st);
  trace_end(FLJSD_KERNEL_SMALL, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_zero(void* to, size_t bytes, cudaStream_t st) {
  if (bytes == 0) return cudaSuccess;
  const int64_t n = (int64_t)(bytes / sizeof(uint4)), blocks = (n + kThreads - 1) / kThreads;
  k_zero<<<(unsigned)(blocks < num_sms() ? blocks : num_sms()), kThreads, 0, st>>>(
      static_cast<uint4*>(to), n);
  count_extra_launch();
  return cudaGetLastError();
}

int lp_row_group(int dtype, int64_t rows, int64_t segs) {
  if (dtype != FLJSD_BF16) return 1;
  const int64_t g = rows * segs / ((int64_t)num_sms() * 16);  // (16 parts for each SM are left)
  return g > 4 ? 4 : g > 1 ? (int)g : 1;
}

cudaError_t launch_lp_rows(int dtype, const LpRowsArgs& a, cudaStream_t st) {
  if (a.rows <= 0) return cudaSuccess;
  const int64_t parts = (a.segs + a.group - 1) / a.group;
  const dim3 grid = row_grid(parts, a.rows);
  trace_begin(FLJSD_KERNEL_JSD_ROWS, st);
  cudaError_t e = cudaSuccess;
  if (a.own_logits)  // (fp32)
    e = launch_dependent(k_lp_rows<float>, grid, kThreads, 0, st, a, parts);
  else if (a.group > 1)
    k_lp_rows_many<<<grid, kThreads, 0, st>>>(a);
  else if (dtype == FLJSD_BF16)
    k_lp_rows<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a, parts);
  else
    k_lp_rows<float><<<grid, kThreads, 0, st>>>(a, parts);
  trace_end(FLJSD_KERNEL_JSD_ROWS, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_lp_grad(int z_dtype, int out_dtype, bool from_e, const LpGradArgs& a,
                           cudaStream_t st) {
  if (a.rows <= 0) return cudaSuccess;
  const dim3 grid = row_grid(from_e ? (a.v + LP_SEG - 1) / LP_SEG : lp_row_segs(a.v), a.rows);
  using bf = __nv_bfloat16;
  trace_begin(FLJSD_KERNEL_JSD_ROWS, st);
  if (from_e)
    k_lp_grad<__half, bf, true><<<grid, kThreads, 0, st>>>(a);
  else if (z_dtype == FLJSD_F32 && out_dtype == FLJSD_F32)
    k_lp_grad<float, float, false><<<grid, kThreads, 0, st>>>(a);
  else if (z_dtype == FLJSD_F32)
    k_lp_grad<float, bf, false><<<grid, kThreads, 0, st>>>(a);
  else
    k_lp_grad<bf, bf, false><<<grid, kThreads, 0, st>>>(a);
  trace_end(FLJSD_KERNEL_JSD_ROWS, st);
  return cudaGetLastError();
}

}  // namespace fljsd
