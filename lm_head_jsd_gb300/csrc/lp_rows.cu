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
constexpr int kGroups = kThreads / 4;  // groups of threads whose maxima are ranked
constexpr int kList = 512;             // candidates of a segment ranked in shared memory
static_assert(LP_MAX_TOP <= kGroups, "the k-th of the groups' maxima");
constexpr int kJoinThreads = 256;
constexpr int kJoinCap = 1024;  // candidates ranked in shared memory
static_assert(kJoinThreads <= kJoinCap && kJoinThreads >= LP_MAX_TOP, "the threads' largest");

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

// (m, d, s) of two sets, each relative to its own maximum (lp.cuh); a set without a
// finite value has m = -inf and d = s = 0, or NaN where it holds one.
struct Mds {
  float m, d, s;
};
__device__ __forceinline__ Mds merge(const Mds& a, const Mds& b, float c) {
  const float m = fmaxf(a.m, b.m);
  const float ta = a.m == -INFINITY ? 0.f : __fmul_rn(a.m - m, c);
  const float tb = b.m == -INFINITY ? 0.f : __fmul_rn(b.m - m, c);
  const float fa = ex2(ta), fb = ex2(tb);
  // 2^t (s + d t): both vanish where 2^t does
  return Mds{m, __fmaf_rn(a.d, fa, b.d * fb),
             __fmaf_rn(fa, __fmaf_rn(a.d, fmaxf(ta, -1024.f), a.s),
                       fb * __fmaf_rn(b.d, fmaxf(tb, -1024.f), b.s))};
}
// The block's, in a fixed order (in every thread of the first warp).
template <int W>
__device__ __forceinline__ Mds block_mds(Mds x, float c, Mds* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    x = merge(x, Mds{__shfl_xor_sync(0xffffffffu, x.m, o), __shfl_xor_sync(0xffffffffu, x.d, o),
                     __shfl_xor_sync(0xffffffffu, x.s, o)}, c);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
  __syncthreads();
  if (threadIdx.x < 32) {
    x = threadIdx.x < W ? sh[threadIdx.x] : Mds{-INFINITY, 0.f, 0.f};
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1)
      x = merge(x, Mds{__shfl_xor_sync(0xffffffffu, x.m, o), __shfl_xor_sync(0xffffffffu, x.d, o),
                       __shfl_xor_sync(0xffffffffu, x.s, o)}, c);
  }
  return x;
}

// A segment's logits, 32 to a thread: vectors of N elements, kThreads vectors
// apart, from a 16-byte boundary. The vector that starts before the row (whose
// first element may lie anywhere) and the one that crosses its end are read one
// element at a time. Sums are taken relative to each thread's own maximum, so
// that one reduction serves maximum and sums.
template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads, TOP ? 3 : 4) k_lp_rows(LpRowsArgs a, int64_t parts) {
  constexpr int N = Vec<T>::N;
  constexpr int V = kPer / N;
  __shared__ Mds shm[kWarps];
  __shared__ unsigned long long sh64[kWarps];
  __shared__ float gmax[kGroups];
  __shared__ unsigned long long list[kList];
  __shared__ int n_list;
  __shared__ float s_thr;
  const int tid = threadIdx.x;
  const int64_t part = blockIdx.x;
  if (a.status && part == 0 && blockIdx.y == 0 && tid == 0) *a.status = 0;
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    const T* zr = reinterpret_cast<const T*>(a.z) + r * a.ld;
    const int lead = (int)((((uintptr_t)zr) & 15u) / sizeof(T));
    const int64_t e0 = part * LP_SEG - lead;  // first element, may be before the row
    const int n = (int)(a.v - e0 < LP_SEG ? (a.v > e0 ? a.v - e0 : 0) : LP_SEG);
    const int first = e0 < 0 ? lead : 0;      // elements [first, n) of the segment count
    const T* zs = zr + e0;
    float z[kPer];
#pragma unroll
    for (int u = 0; u < V; ++u) {
      const int j = (u * kThreads + tid) * N;
      if (j >= first && j + N <= n) {
        float o[N];
        Vec<T>::load(zs + j, o);
#pragma unroll
        for (int e = 0; e < N; ++e) z[u * N + e] = o[e];
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
          z[u * N + e] = (j + e >= first && j + e < n) ? val(zs + j + e) : -INFINITY;
      }
    }
    Mds x{-INFINITY, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kPer; ++i) x.m = fmaxf(x.m, z[i]);  // (skips NaN)
    {
      const float ref = x.m == -INFINITY ? 0.f : x.m;
      const float2 c2 = make_float2(a.c, a.c), nref = make_float2(-ref, -ref);
      float2 d = make_float2(0.f, 0.f), t = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kPer; i += 2) {
        const float2 q = __fmul2_rn(__fadd2_rn(make_float2(z[i], z[i + 1]), nref), c2);
        const float2 y = make_float2(ex2(q.x), ex2(q.y));
        d = __fadd2_rn(d, y);
        // a logit of -inf adds 0, NaN stays
        t = __ffma2_rn(y, make_float2(fmaxf(q.x, -1024.f), fmaxf(q.y, -1024.f)), t);
      }
      x.d = d.x + d.y;
      x.s = t.x + t.y;
    }
    const float tm = x.m;
    x = block_mds<kWarps>(x, a.c, shm);
    if (tid == 0) {
      a.part[r * parts + part] = make_float4(x.m, x.d, x.s, 0.f);
      if (a.labels && part == 0) {
        const int64_t y = a.labels[a.row0 + r];
        if (y >= 0 && y < a.v) a.zy[r] = val(zr + y);
      }
    }
    if (TOP) {
      // The k-th largest of 64 groups' maxima (four threads each) bounds the k-th
      // largest logit from below: what reaches it is listed and ranked. A list
      // that overflows (many equal logits) is replaced by k rounds of the largest
      // remaining key.
      float g = tm;
      g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 1));
      g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 2));
      if ((tid & 3) == 0) gmax[tid >> 2] = g;
      if (tid == 0) n_list = 0;
      __syncthreads();
      if (tid < kGroups) {
        const float o = gmax[tid];
        int rank = 0;
#pragma unroll 16
        for (int j = 0; j < kGroups; ++j) rank += (gmax[j] > o || (gmax[j] == o && j < tid)) ? 1 : 0;
        if (rank == a.k - 1) s_thr = o;
      }
      __syncthreads();
      const float thr = s_thr;
      if (tm >= thr) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (z[i] >= thr && z[i] > -INFINITY) {
            const int at = atomicAdd(&n_list, 1);
            const int col = (int)e0 + ((i / N) * kThreads + tid) * N + i % N;
            if (at < kList) list[at] = cand_key(make_int2(__float_as_int(z[i]), col));
          }
        }
      }
      __syncthreads();
      const int n_all = n_list;
      int2* out = a.cand + (r * parts + part) * a.k;
      if (n_all <= kList) {
        for (int i = tid; i < n_all; i += kThreads) {
          const unsigned long long key = list[i];
          int above = 0;
          for (int j = 0; j < n_all; ++j) above += list[j] > key ? 1 : 0;
          if (above < a.k) out[above] = make_int2(__float_as_int(key_value(key)), key_col(key));
        }
        for (int i = n_all + tid; i < a.k; i += kThreads) out[i] = make_int2(0, -1);
      } else {
        unsigned long long last = ~0ull;
        for (int q = 0; q < a.k; ++q) {
          unsigned long long best = 0;
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int col = (int)e0 + ((i / N) * kThreads + tid) * N + i % N;
            const unsigned long long key =
                z[i] > -INFINITY ? cand_key(make_int2(__float_as_int(z[i]), col)) : 0ull;
            best = key < last && key > best ? key : best;
          }
          best = block_max64<kWarps>(best, sh64);
          if (tid == 0)
            out[q] = best ? make_int2(__float_as_int(key_value(best)), key_col(best)) : make_int2(0, -1);
          last = best;
        }
      }
    }
    __syncthreads();  // the shared results are written again by the next row
  }
}

// One CTA to a row: its parts into the row's results, its candidates into the
// k largest.
__global__ void __launch_bounds__(kJoinThreads) k_lp_join(LpJoinArgs a) {
  constexpr int W = kJoinThreads / 32;
  __shared__ Mds shm[W];
  __shared__ float2 sh_norm;
  __shared__ unsigned long long sh64[W];
  __shared__ unsigned long long list[kJoinCap];
  __shared__ int n_list;
  __shared__ unsigned sh_least;
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x, out = a.row0 + r;
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
  const int2* cand = a.cand + r * a.cap;
  const int64_t n_cand = a.count ? (int64_t)a.count[r] : a.cap;
  unsigned least = 0;
  if (a.gmax) {
    least = 0xffffffffu;
    for (int j = 0; j < a.k; ++j) least = min(least, a.gmax[r * a.k + j]);
  }
  const float* dump = a.dump + r * a.dump_cols;
  const int64_t n_dump = a.dump ? (a.dump_cols < a.v ? a.dump_cols : a.v) : 0;
  auto dump_key = [&](int64_t i) {
    const float z = dump[i];
    return z > -INFINITY ? cand_key(make_int2(__float_as_int(z), (int)i)) : 0ull;
  };
  // every candidate's key, four loads in flight a thread
  auto each = [&](auto&& f) {
#pragma unroll 4
    for (int64_t i = tid; i < n_cand; i += kJoinThreads) f(cand_key(cand[i]));
#pragma unroll 4
    for (int64_t i = tid; i < n_dump; i += kJoinThreads) f(dump_key(i));
  };
  auto gather = [&]() {
    each([&](unsigned long long key) {
      if (key != 0 && (unsigned)(key >> 32) >= least) {
        const int at = atomicAdd(&n_list, 1);
        if (at < kJoinCap) list[at] = key;
      }
    });
  };
  gather();
  __syncthreads();
  if (n_list > kJoinCap) {
    // no threshold, or many equal logits: the k-th largest of the threads' own
    // largest keys bounds the k-th largest from below, ties apart
    unsigned long long mine = 0;
    each([&](unsigned long long key) { mine = key > mine ? key : mine; });
    __syncthreads();
    list[tid] = mine;
    __syncthreads();
    int rank = 0;
    for (int j = 0; j < kJoinThreads; ++j) rank += (list[j] > mine || (list[j] == mine && j < tid)) ? 1 : 0;
    if (rank == a.k - 1) sh_least = (unsigned)(mine >> 32);
    if (tid == 0) n_list = 0;
    __syncthreads();
    least = sh_least;
    gather();
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

// dz of one logit; lp2 = log2 p. -inf: p = 0 and p log p = 0.
//   -p (a + b (log p + entropy)) = -p (b ln2 log2 p + (a + b entropy))
__device__ __forceinline__ float grad_of(float lp2, float bl, float ab) {
  return -ex2(lp2) * __fmaf_rn(bl, fmaxf(lp2, -1024.f), ab);
}

// One CTA to a segment of a row, in vectors of eight where the logits and their
// gradient lie alike relative to a 16-byte boundary (rows of odd length start
// anywhere, but both at the same place), else one element at a time. All loads of
// a thread are issued before the first is used.
template <typename TI, typename TO, bool FROM_E>
__global__ void __launch_bounds__(kThreads) k_lp_grad(LpGradArgs a) {
  constexpr int N = 8, U = LP_SEG / (kThreads * N);
  const int tid = threadIdx.x;
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    const TI* zr = reinterpret_cast<const TI*>(a.z) + r * a.ldz;
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
    const float bl = gb * kLn2, ab = __fmaf_rn(gb, ent, ga);
    const bool same = ((uintptr_t)zr & 15u) / sizeof(TI) == ((uintptr_t)orow & 15u) / sizeof(TO);
    const int lead = same ? (int)(((uintptr_t)zr & 15u) / sizeof(TI)) : 0;
    const int64_t e0 = (int64_t)blockIdx.x * LP_SEG - lead;
    const int n = (int)(a.v - e0 < LP_SEG ? (a.v > e0 ? a.v - e0 : 0) : LP_SEG);
    const int first = e0 < 0 ? lead : 0;  // elements [first, n) of the segment count
    const TI* zs = zr + e0;
    TO* os = orow + e0;
    // log2 p = c (z - m) - log2 d; from 2^t, log2 p = t + c (m of its part - m) - log2 d
    auto one = [&](float z, float ref) {
      const float lp2 = FROM_E ? lg2(z) + ref : __fmul_rn(z - norm.x, a.c) - norm.y;
      return grad_of(lp2, bl, ab);
    };
    auto ref_of = [&](int j) {  // (FROM_E: lead is 0)
      return FROM_E ? __fmul_rn(a.part[r * a.parts + (e0 + j) / LP_PART_COLS].x - norm.x, a.c) - norm.y
                    : 0.f;
    };
    if (same) {
      float z[U][N], ref[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = (u * kThreads + tid) * N;
        ref[u] = 0.f;
        if (live && j >= first && j + N <= n) {
          load8(zs + j, z[u]);
          ref[u] = ref_of(j);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = (u * kThreads + tid) * N;
        if (j >= first && j + N <= n) {
#pragma unroll
          for (int e = 0; e < N; ++e) z[u][e] = live ? one(z[u][e], ref[u]) : 0.f;
          store8(os + j, z[u]);
        } else {
          for (int e = 0; e < N; ++e)
            if (j + e >= first && j + e < n)
              Vec<TO>::put(os + j + e, live ? one(val(zs + j + e), ref_of(j + e)) : 0.f);
        }
      }
    } else {
      for (int j = tid; j < n; j += kThreads)
        Vec<TO>::put(os + j, live ? one(val(zs + j), ref_of(j)) : 0.f);
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

// x: segments of a row; y: rows, up to what keeps the GPU full (a CTA then walks on)
dim3 row_grid(int64_t segs, int64_t rows) {
  const int64_t most = ((int64_t)num_sms() * 32 + segs - 1) / segs;
  const int64_t y = rows < most ? rows : most;
  return dim3((unsigned)segs, (unsigned)(y < 65535 ? y : 65535));
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
  const dim3 grid = row_grid(parts, a.rows);
  trace_begin(FLJSD_KERNEL_JSD_ROWS, st);
  if (dtype == FLJSD_BF16) {
    if (a.k > 0)
      k_lp_rows<__nv_bfloat16, true><<<grid, kThreads, 0, st>>>(a, parts);
    else
      k_lp_rows<__nv_bfloat16, false><<<grid, kThreads, 0, st>>>(a, parts);
  } else {
    if (a.k > 0)
      k_lp_rows<float, true><<<grid, kThreads, 0, st>>>(a, parts);
    else
      k_lp_rows<float, false><<<grid, kThreads, 0, st>>>(a, parts);
  }
  trace_end(FLJSD_KERNEL_JSD_ROWS, st);
  return cudaGetLastError();
}

cudaError_t launch_lp_grad(int z_dtype, int out_dtype, bool from_e, const LpGradArgs& a,
                           cudaStream_t st) {
  if (a.rows <= 0) return cudaSuccess;
  const dim3 grid = row_grid(from_e ? (a.v + LP_SEG - 1) / LP_SEG : lp_row_parts(a.v), a.rows);
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
