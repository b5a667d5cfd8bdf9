// Verification of drafted tokens against the target's probabilities, from given random
// numbers.
//
// With w_j = 2^((z_j - m) log2(e) / T) of a row (m its largest logit, w in fp32) and
// [x] = x as a whole number of 2^-43, the nearest:
//   total = sum_j [w_j],  p_j = w_j / total,
//   a drafted token d is accepted where u q_d < p_d (in fp64),
//   r_j = p_j, or p_j - q_j where that is more than 0 (fp32), and the token drawn is the
//   lowest one whose running sum of [r] exceeds floor(u sum_j [r_j]).
// Whole numbers add up to the same in any order: however a row is cut over threads, CTAs
// and launches, and whatever else is in the batch, the same logits and numbers give the
// same tokens. (With fp32 sums one draw in forty over 128256 columns goes another way when
// the order changes: every column's border moves by some 1e-7 of the whole.)
//
// A weight in [0, 1] becomes a whole number without a conversion (those take a slow
// unit): t = w + 12 rounds to 2^-20, and its bits minus 12's count them; w - (t - 12) is
// exact and, added to 1.5 2^-20, rounds to 2^-43 the same way. Both counts are summed as
// 32-bit integers, the constants taken off once.
//
// k_verify_rows: a cluster takes a row and keeps it in registers between finding its
// maximum and the sum, so that HBM is read once. k_verify_draw, one cluster for each
// request: the tests, then one pass over the row where a token is to be drawn (two rows
// after a refusal), each warp's vectors with a sum of their own; the one the number falls
// into is read again.
#include "dependent.cuh"
#include "internal.cuh"

#include <cmath>

namespace fljsd {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int64_t kMaxV = 1 << 20;  // sums of [w] stay below 2^63
constexpr double kUnit = 0x1p43;
constexpr float kC1 = 12.f, kC2 = 0x1.8p-20f;
constexpr uint32_t kBits1 = 0x41400000u, kBits2 = 0x35c00000u;
constexpr unsigned long long kNone = ~0ull;

enum { kRowOk = 0, kRowBad = 1 };  // bad: NaN, +inf, or nothing but -inf

struct RowStat {
  float m;    // largest logit
  float wd;   // the drafted token's weight
  unsigned long long total;
  int best;   // the first largest (greedy), -1: none
  int state;
};

struct Args {
  const void* target;
  const void* draft;  // or null
  int64_t ld_target, ld_draft;
  const int64_t* tokens;
  const float* u;
  const float* u_draw;
  const int64_t* offsets;  // [requests + 1] or null
  const float* temperature;  // [requests] or null
  float t;
  int64_t n, requests, v;
  int max_drafts, slots, cluster;
  int64_t* out;
  int64_t* accepted;
  float* prob;
  int* status;
  RowStat* stat_t;
  RowStat* stat_d;
};

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// Writes to the same shared variable of CTA `rank`.
__device__ __forceinline__ void put_remote(void* p, uint32_t rank, unsigned long long x) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p), r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(r), "l"(x) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

struct Request {
  int64_t start;
  int drafts;
  float c;  // log2(e) / T; 0: greedy
  bool ok;
};
__device__ __forceinline__ Request request(const Args& a, int64_t b) {
  Request r;
  int64_t end;
  if (a.offsets) {
    r.start = a.offsets[b];
    end = a.offsets[b + 1];
  } else {
    r.start = b * a.max_drafts;
    end = r.start + a.max_drafts;
  }
  const float t = a.temperature ? a.temperature[b] : a.t;
  r.c = t == 0.f ? 0.f : (float)(1.4426950408889634 / (double)t);
  r.ok = r.start >= 0 && r.start <= end && end <= a.n && end - r.start <= a.max_drafts && t >= 0.f &&
         t < INFINITY && r.c < INFINITY;
  r.drafts = r.ok ? (int)(end - r.start) : 0;
  return r;
}

template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  static constexpr uint32_t kMasked = sizeof(T) == 4 ? 0xff800000u : 0xff80u;  // -inf
};
template <typename T>
__device__ __forceinline__ uint32_t bits_at(const T* p) {
  return sizeof(T) == 4 ? *reinterpret_cast<const uint32_t*>(p)
                        : (uint32_t)*reinterpret_cast<const uint16_t*>(p);
}
template <typename T>
__device__ __forceinline__ float value_at(const T* p) {
  return __uint_as_float(sizeof(T) == 4 ? bits_at(p) : bits_at(p) << 16);
}
// Columns [j, j + N) of a row of v; those outside of it read as -inf. `whole`: j is on a
// 16-byte boundary.
template <typename T>
__device__ __forceinline__ uint4 load(const T* row, int64_t j, int64_t v, bool whole) {
  constexpr int N = Vec<T>::N;
  if (whole && j >= 0 && j + N <= v) return *reinterpret_cast<const uint4*>(row + j);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    auto at = [&](int64_t k) { return k >= 0 && k < v ? bits_at(row + k) : Vec<T>::kMasked; };
    w[i] = sizeof(T) == 4 ? at(j + i) : at(j + 2 * i) | (at(j + 2 * i + 1) << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ void values(const uint4& q, float2 (&z)[Vec<T>::N / 2]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if (sizeof(T) == 4) {
    z[0] = make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
    z[1] = make_float2(__uint_as_float(w[2]), __uint_as_float(w[3]));
  } else {
#pragma unroll
    for (int i = 0; i < Vec<T>::N / 2; ++i)
      z[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
}
// The largest of a vector; a NaN stays.
template <typename T>
__device__ __forceinline__ float largest(const uint4& q, float m) {
  float2 z[Vec<T>::N / 2];
  values<T>(q, z);
#pragma unroll
  for (int i = 0; i < Vec<T>::N / 2; ++i) m = max_nan(m, max_nan(z[i].x, z[i].y));
  return m;
}

// Two weights relative to m.
__device__ __forceinline__ float2 weights(float2 z, float m, float c) {
  const float2 d = __fadd2_rn(z, make_float2(-m, -m));
  const float2 x = __fmul2_rn(d, make_float2(c, c));
  return make_float2(ex2(x.x), ex2(x.y));
}

// Sums of whole numbers of 2^-43, of up to 511 values in [0, 1] each.
struct Count {
  uint32_t hi = 0, lo = 0;
  __device__ __forceinline__ void add(float2 w) {
    const float2 t = __fadd2_rn(w, make_float2(kC1, kC1));
    const float2 back = __ffma2_rn(t, make_float2(-1.f, -1.f), make_float2(kC1, kC1));  // exact
    const float2 s = __fadd2_rn(__fadd2_rn(w, back), make_float2(kC2, kC2));
    hi += __float_as_uint(t.x) + __float_as_uint(t.y);
    lo += __float_as_uint(s.x) + __float_as_uint(s.y);
  }
  __device__ __forceinline__ unsigned long long sum(uint32_t n) const {
    return ((unsigned long long)(hi - n * kBits1) << 23) + (long long)(int)(lo - n * kBits2);
  }
};

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// What a cluster's CTAs tell each other.
struct Shared {
  unsigned long long top[kMaxCluster];   // their maxima
  unsigned long long sum[kMaxCluster];
  unsigned long long best[kMaxCluster];
  unsigned long long warp[kWarps];
  float warp_top[kWarps];
};

// Where a row lies: vectors [first, last) of N columns, the first one from the 16-byte
// boundary at or before the row's start; column j of vector k is k N - lead.
template <typename T>
struct Cut {
  int lead, first, last;
  __device__ __forceinline__ Cut(const T* row, int64_t v, int cluster, int rank) {
    lead = (int)(((uintptr_t)row & 15u) / sizeof(T));
    const int all = (int)((v + lead + Vec<T>::N - 1) / Vec<T>::N);
    const int per = (all + cluster - 1) / cluster;
    first = min(rank * per, all);
    last = min(first + per, all);
  }
};

template <typename T>
constexpr int kept() {  // vectors a thread keeps: 32 columns
  return 32 / Vec<T>::N;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) k_verify_rows(const Args a) {
  constexpr int N = Vec<T>::N, R = kept<T>();
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cta_rank();
  const int64_t unit = blockIdx.x / a.cluster, b = unit / a.slots;
  const int slot = (int)(unit % a.slots);
  let_next_launch();
  if (blockIdx.x == 0 && tid == 0) *a.status = 0;
  const Request q = request(a, b);
  const bool is_draft = slot > a.max_drafts;
  const int j = is_draft ? slot - a.max_drafts - 1 : slot;
  if (!q.ok || j >= q.drafts + (is_draft ? 0 : 1) || (is_draft && q.c == 0.f)) return;
  if (a.cluster > 1) cluster_arrive();  // (none is written to before it has started)
  const int64_t at = q.start + j;
  const T* row = is_draft ? reinterpret_cast<const T*>(a.draft) + at * a.ld_draft
                          : reinterpret_cast<const T*>(a.target) + (at + b) * a.ld_target;
  const Cut<T> cut(row, a.v, a.cluster, rank);
  auto column = [&](int k) { return (int64_t)k * N - cut.lead; };
  uint4 raw[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int k = cut.first + r * kThreads + tid;
    raw[r] = load(row, k < cut.last ? column(k) : a.v, a.v, true);
  }
  float m = -INFINITY;
#pragma unroll
  for (int r = 0; r < R; ++r) m = largest<T>(raw[r], m);
  for (int k = cut.first + R * kThreads + tid; k < cut.last; k += kThreads)
    m = largest<T>(load(row, column(k), a.v, true), m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) sh.warp_top[warp] = m;
  __syncthreads();
  m = sh.warp_top[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) m = max_nan(m, sh.warp_top[w]);
  if (a.cluster > 1) {
    cluster_wait();
    if (tid < a.cluster) put_remote(&sh.top[rank], tid, (unsigned long long)__float_as_uint(m));
    cluster_sync();
    for (int i = 0; i < a.cluster; ++i) m = max_nan(m, __uint_as_float((uint32_t)sh.top[i]));
  }
  const bool bad = !(fabsf(m) < INFINITY);
  unsigned long long sum = 0, best = kNone;
  if (!bad && q.c != 0.f) {
    Count n;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 z[N / 2];
      values<T>(raw[r], z);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) n.add(weights(z[i], m, q.c));
    }
    sum = n.sum(R * N);
    for (int k = cut.first + R * kThreads + tid; k < cut.last; k += kThreads) {
      float2 z[N / 2];
      values<T>(load(row, column(k), a.v, true), z);
      Count more;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) more.add(weights(z[i], m, q.c));
      sum += more.sum(N);
    }
    sum = warp_sum(sum);
  } else if (!bad) {
    auto look = [&](const uint4& x, int64_t j0) {
      float2 z[N / 2];
      values<T>(x, z);
#pragma unroll
      for (int i = N / 2 - 1; i >= 0; --i) {
        if (z[i].y == m) best = min(best, (unsigned long long)(j0 + 2 * i + 1));
        if (z[i].x == m) best = min(best, (unsigned long long)(j0 + 2 * i));
      }
    };
#pragma unroll
    for (int r = 0; r < R; ++r) look(raw[r], column(cut.first + r * kThreads + tid));
    for (int k = cut.first + R * kThreads + tid; k < cut.last; k += kThreads)
      look(load(row, column(k), a.v, true), column(k));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = min(best, __shfl_xor_sync(0xffffffffu, best, o));
    sum = best;  // (what the warps hand over)
  }
  if (lane == 0) sh.warp[warp] = sum;
  __syncthreads();
  const bool greedy = q.c == 0.f;
  if (tid == 0) {
    sum = sh.warp[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) sum = greedy ? min(sum, sh.warp[w]) : sum + sh.warp[w];
    if (a.cluster > 1) put_remote(&sh.sum[rank], 0, sum);
  }
  if (a.cluster > 1) cluster_sync();
  if (rank == 0 && tid == 0) {
    if (a.cluster > 1) {
      sum = sh.sum[0];
      for (int i = 1; i < a.cluster; ++i) sum = greedy ? min(sum, sh.sum[i]) : sum + sh.sum[i];
    }
    RowStat s{m, 0.f, sum, -1, bad ? kRowBad : kRowOk};
    if (!bad && greedy) s.best = (int)sum;
    if (!bad && !greedy && j < q.drafts) {
      const int64_t d = a.tokens[at];
      if (d >= 0 && d < a.v) s.wd = ex2(__fmul_rn(__fsub_rn(value_at(row + d), m), q.c));
    }
    (is_draft ? a.stat_d[at] : a.stat_t[at + b]) = s;
  }
}

// The whole numbers of one vector of p, or of p - q.
template <typename T>
struct Residual {
  const T* p;
  const T* q;  // or null
  float mp, mq, c, ip, iq;
  int64_t v, without;  // a column whose q is 1, or -1
  bool q_whole;        // q lies to 16 bytes as p does
  __device__ __forceinline__ void get(int64_t j, float2 (&r)[Vec<T>::N / 2]) const {
    constexpr int N = Vec<T>::N;
    float2 z[N / 2], y[N / 2];
    values<T>(load(p, j, v, true), z);
    if (q) values<T>(load(q, j, v, q_whole), y);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      r[i] = __fmul2_rn(weights(z[i], mp, c), make_float2(ip, ip));
      if (q) {
        // (sums one by one: a packed product and a packed sum become one rounding)
        const float2 o = __fmul2_rn(weights(y[i], mq, c), make_float2(-iq, -iq));
        r[i].x = fmaxf(__fadd_rn(r[i].x, o.x), 0.f);
        r[i].y = fmaxf(__fadd_rn(r[i].y, o.y), 0.f);
      } else if (without >= 0) {  // p - 1 is at most 0
        if (j + 2 * i == without) r[i].x = 0.f;
        if (j + 2 * i + 1 == without) r[i].y = 0.f;
      }
    }
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) k_verify_draw(const Args a) {
  constexpr int N = Vec<T>::N;
  __shared__ Shared sh;
  __shared__ int s_accepted;
  extern __shared__ unsigned long long s_sums[];  // [iterations][kWarps]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cta_rank();
  const int64_t b = blockIdx.x / a.cluster;
  if (a.cluster > 1) cluster_arrive();  // (none is written to before it has started)
  wait_for_previous();
  const Request q = request(a, b);
  const bool greedy = q.c == 0.f;
  // the tests, a lane to each; every CTA of the cluster makes them
  if (warp == 0) {
    int accepted = 0;
    bool going = true, refuse = !q.ok;
    for (int j0 = 0; j0 < q.drafts; j0 += 32) {
      const int j = j0 + lane;
      bool hit = false;
      if (j < q.drafts) {
        const int64_t at = q.start + j, d = a.tokens[at];
        const RowStat st = a.stat_t[at + b];
        float prob = 0.f;
        const bool in = d >= 0 && d < a.v;
        refuse |= !in;
        if (in && st.state == kRowOk) {
          if (greedy) {
            hit = d == st.best;
            prob = hit ? 1.f : 0.f;
          } else {
            const double p = (double)st.wd / ((double)st.total / kUnit);
            double qd = 1.0;
            bool known = true;
            if (a.draft) {
              const RowStat sd = a.stat_d[at];
              known = sd.state == kRowOk;
              qd = known ? (double)sd.wd / ((double)sd.total / kUnit) : 1.0;
            }
            if (known) {
              hit = (double)a.u[at] * qd < p;
              const double x = qd > 0.0 ? p / qd : p > 0.0 ? 1.0 : 0.0;
              prob = (float)(x < 1.0 ? x : 1.0);
            }
          }
        }
        if (rank == 0) a.prob[at] = prob;
      }
      const uint32_t hits = __ballot_sync(0xffffffffu, hit);
      if (going) {
        const int run = hits == 0xffffffffu ? 32 : __ffs(~hits) - 1;
        accepted += run;
        going = run == 32;
      }
    }
    refuse = __any_sync(0xffffffffu, refuse);
    if (lane == 0) {
      s_accepted = accepted;
      if (refuse && rank == 0) atomicExch(a.status, (int)FLJSD_ERR_INVALID_ARG);
    }
  }
  __syncthreads();
  if (a.cluster > 1) cluster_wait();
  const int accepted = s_accepted;
  const int64_t at = q.start + accepted;
  RowStat sp{};
  if (q.ok) sp = a.stat_t[at + b];
  int64_t token = -1;
  if (rank == 0 && warp == 0) {  // drafts beyond the requests' are none
    if (b == 0 && a.offsets)
      for (int64_t i = lane; i < a.n && i < a.offsets[0]; i += 32) a.prob[i] = 0.f;
    if (b == a.requests - 1 && a.offsets)
      for (int64_t i = max((int64_t)0, a.offsets[b + 1]) + lane; i < a.n; i += 32) a.prob[i] = 0.f;
  }
  if (q.ok && greedy) {
    token = sp.best;
  } else if (q.ok && sp.state == kRowOk) {
    Residual<T> res{};
    res.p = reinterpret_cast<const T*>(a.target) + (at + b) * a.ld_target;
    res.mp = sp.m;
    res.c = q.c;
    res.ip = (float)(1.0 / ((double)sp.total / kUnit));
    res.v = a.v;
    res.without = -1;
    if (accepted < q.drafts) {
      if (a.draft) {
        const RowStat sd = a.stat_d[at];
        if (sd.state == kRowOk) {
          res.q = reinterpret_cast<const T*>(a.draft) + at * a.ld_draft;
          res.mq = sd.m;
          res.iq = (float)(1.0 / ((double)sd.total / kUnit));
          res.q_whole = (((uintptr_t)res.p ^ (uintptr_t)res.q) & 15u) == 0;
        }
      } else {
        res.without = a.tokens[at];
      }
    }
    const Cut<T> cut(res.p, a.v, a.cluster, rank);
    const int iters = (cut.last - cut.first + kThreads - 1) / kThreads;
    unsigned long long before = 0, total = 0, mine = 0;
    for (int turn = 0; turn < 2; ++turn) {
      mine = 0;
      for (int it = 0; it < iters; ++it) {
        const int k = cut.first + it * kThreads + tid;
        float2 r[N / 2];
        Count n;
        if (k < cut.last) {
          res.get((int64_t)k * N - cut.lead, r);
#pragma unroll
          for (int i = 0; i < N / 2; ++i) n.add(r[i]);
        }
        const unsigned long long s = warp_sum(k < cut.last ? n.sum(N) : 0ull);
        if (lane == 0) s_sums[it * kWarps + warp] = s;
        mine += s;
      }
      if (lane == 0) sh.warp[warp] = mine;
      __syncthreads();
      mine = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mine += sh.warp[w];
      if (a.cluster > 1) {
        if (tid < a.cluster) put_remote(&sh.sum[rank], tid, mine);
        cluster_sync();
        before = total = 0;
        for (int i = 0; i < a.cluster; ++i) {
          if (i < rank) before += sh.sum[i];
          total += sh.sum[i];
        }
      } else {
        total = mine;
      }
      if (total != 0) break;
      // p is nowhere above q: from p itself
      res.q = nullptr;
      res.without = -1;
      __syncthreads();  // (sh.warp is written again)
      if (a.cluster > 1) cluster_sync();
    }
    const double want = (double)a.u_draw[b] * (double)total;
    unsigned long long t = want > 0.0 ? want >= (double)total ? total - 1 : (unsigned long long)want : 0ull;
    t = min(t, total - 1);
    if (t >= before && t - before < mine && warp == 0) {
      t -= before;
      // the warp's vectors that hold it: the first of the sums whose running sum exceeds t
      unsigned long long run = 0;
      int found = 0;
      for (int i0 = 0; i0 < iters * kWarps; i0 += 32) {
        const int i = i0 + lane;
        unsigned long long x = i < iters * kWarps ? s_sums[i] : 0ull;
        const unsigned long long own = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const uint32_t over = __ballot_sync(0xffffffffu, run + x > t);
        if (over) {
          const int l = __ffs(over) - 1;
          found = i0 + l;
          run += __shfl_sync(0xffffffffu, x - own, l);
          break;
        }
        run += __shfl_sync(0xffffffffu, x, 31);
      }
      const int k = cut.first + (found / kWarps) * kThreads + (found % kWarps) * 32 + lane;
      const int64_t j0 = (int64_t)k * N - cut.lead;
      unsigned long long one[N], x = 0;
      float2 r[N / 2] = {};
      if (k < cut.last) res.get(j0, r);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        Count n;
        n.add(make_float2(r[i].x, 0.f));
        one[2 * i] = n.sum(2);
        Count o;
        o.add(make_float2(r[i].y, 0.f));
        one[2 * i + 1] = o.sum(2);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) x += one[i];
      const unsigned long long own = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const uint32_t over = __ballot_sync(0xffffffffu, run + x > t);
      if (over && lane == __ffs(over) - 1) {
        run += x - own;
        int i = 0;
#pragma unroll
        for (int e = 0; e < N - 1; ++e) {
          run += one[e];
          if (run <= t) i = e + 1;
        }
        a.out[b * (a.max_drafts + 1) + accepted] = j0 + i;
      }
    }
    token = -2;  // (written by the CTA that found it)
  }
  if (rank == 0) {
    for (int i = tid; i <= a.max_drafts; i += kThreads)
      if (i != accepted || token != -2)
        a.out[b * (a.max_drafts + 1) + i] = i < accepted ? a.tokens[q.start + i] : i == accepted ? token : -1;
    if (tid == 0) a.accepted[b] = accepted;
  }
  if (a.cluster > 1) cluster_sync();  // no CTA leaves while another writes to it
}

// CTAs to a row: enough that its threads hold it, more where there are few rows.
int cluster_for(int64_t v, int size, int64_t rows) {
  const int64_t per = (int64_t)kThreads * 32;  // columns a CTA keeps
  int c = 1;
  while (c < kMaxCluster && c * per < v + 16 / size) c *= 2;
  while (c < kMaxCluster && rows * c * 2 <= num_sms() && c * 4 * kThreads < v) c *= 2;
  return c;
}

template <typename T>
cudaError_t launch(Args a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  a.slots = a.max_drafts + 1 + (a.draft ? a.max_drafts : 0);
  a.cluster = cluster_for(a.v, sizeof(T), a.requests * a.slots);
  attr[0].val.clusterDim = {(unsigned)a.cluster, 1, 1};
  cfg.gridDim = dim3((unsigned)(a.requests * a.slots * a.cluster));
  cfg.numAttrs = 1;
  trace_begin(FLJSD_KERNEL_SMALL, st);
  cudaError_t e = cudaLaunchKernelEx(&cfg, k_verify_rows<T>, a);
  trace_end(FLJSD_KERNEL_SMALL, st);
  if (e != cudaSuccess) return e;
  a.cluster = cluster_for(a.v, sizeof(T), a.requests);
  attr[0].val.clusterDim = {(unsigned)a.cluster, 1, 1};
  cfg.gridDim = dim3((unsigned)(a.requests * a.cluster));
  const int64_t vecs = (a.v + 2 * Vec<T>::N - 2) / Vec<T>::N;
  const int64_t iters = ((vecs + a.cluster - 1) / a.cluster + kThreads - 1) / kThreads;
  cfg.dynamicSmemBytes = (size_t)(iters * kWarps * sizeof(unsigned long long));
  cfg.numAttrs = 2;
  trace_begin(FLJSD_KERNEL_SMALL, st);
  e = cudaLaunchKernelEx(&cfg, k_verify_draw<T>, a);
  trace_end(FLJSD_KERNEL_SMALL, st);
  return e;
}

constexpr size_t kStatusBytes = 16;

}  // namespace
}  // namespace fljsd

using namespace fljsd;

extern "C" size_t fljsd_verify_workspace_bytes(int64_t requests, int64_t drafts) {
  if (requests < 0 || drafts < 0) return 0;
  return kStatusBytes + (size_t)(requests + 2 * drafts) * sizeof(RowStat);
}

extern "C" fljsd_status fljsd_verify(int64_t requests, int64_t drafts, int64_t v, int32_t max_drafts,
                                     int32_t dtype, const void* target, int64_t ld_target,
                                     const void* draft, int64_t ld_draft, const int64_t* tokens,
                                     const float* u_accept, const float* u_draw,
                                     const int64_t* offsets, const float* temperatures,
                                     float temperature, int64_t* out, int64_t* accepted,
                                     float* accept_prob, void* workspace, size_t workspace_bytes,
                                     fljsd_stream_t stream) {
  if (requests <= 0 || drafts < 0 || v <= 0 || max_drafts < 0) return FLJSD_ERR_INVALID_ARG;
  if (dtype != FLJSD_F32 && dtype != FLJSD_BF16) return FLJSD_ERR_INVALID_ARG;
  const uintptr_t el = dtype == FLJSD_BF16 ? 1 : 3;
  if (!target || ((uintptr_t)target & el) || ((uintptr_t)draft & el) || ld_target < v ||
      (draft && ld_draft < v))
    return FLJSD_ERR_INVALID_ARG;
  if (!u_draw || !out || !accepted || !workspace || (drafts > 0 && (!tokens || !u_accept || !accept_prob)))
    return FLJSD_ERR_INVALID_ARG;
  if (((uintptr_t)tokens | (uintptr_t)offsets | (uintptr_t)out | (uintptr_t)accepted) & 7u)
    return FLJSD_ERR_INVALID_ARG;
  if (((uintptr_t)u_accept | (uintptr_t)u_draw | (uintptr_t)temperatures | (uintptr_t)accept_prob) & 3u)
    return FLJSD_ERR_INVALID_ARG;
  if ((uintptr_t)workspace & 15u) return FLJSD_ERR_INVALID_ARG;
  if (!offsets && drafts != requests * (int64_t)max_drafts) return FLJSD_ERR_INVALID_ARG;
  if (!temperatures && (!(temperature >= 0.f) || !std::isfinite(temperature) || (temperature > 0.f && !std::isfinite(
                                                      (float)(1.4426950408889634 / (double)temperature)))))
    return FLJSD_ERR_INVALID_ARG;
  if (v >= kMaxV || requests > (1 << 20) || drafts > (1 << 24) || max_drafts > 1024 ||
      requests * (2 * (int64_t)max_drafts + 1) * kMaxCluster > 0x7fffffffll)
    return FLJSD_ERR_UNSUPPORTED;
  if (workspace_bytes < fljsd_verify_workspace_bytes(requests, drafts)) return FLJSD_ERR_WORKSPACE;
  Args a{};
  a.target = target;
  a.draft = draft;
  a.ld_target = ld_target;
  a.ld_draft = ld_draft;
  a.tokens = tokens;
  a.u = u_accept;
  a.u_draw = u_draw;
  a.offsets = offsets;
  a.temperature = temperatures;
  a.t = temperature;
  a.n = drafts;
  a.requests = requests;
  a.v = v;
  a.max_drafts = max_drafts;
  a.out = out;
  a.accepted = accepted;
  a.prob = accept_prob;
  a.status = reinterpret_cast<int*>(workspace);
  a.stat_t = reinterpret_cast<RowStat*>(reinterpret_cast<char*>(workspace) + kStatusBytes);
  a.stat_d = a.stat_t + requests + drafts;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == FLJSD_BF16 ? launch<__nv_bfloat16>(a, st) : launch<float>(a, st);
  return e == cudaSuccess ? FLJSD_OK : FLJSD_ERR_CUDA;
}
