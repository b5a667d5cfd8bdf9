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
// same tokens. (Sums in fp32 move every column's border by some 1e-7 of the whole: over
// 128256 columns, most of them of less than that, one draw in forty would go another way.)
//
// A weight in [0, 1] becomes a whole number without a conversion (those take a slow
// unit): t = w + 12 rounds to 2^-20, and its bits minus 12's count them; w - (t - 12) is
// exact and, added to 1.5 2^-20, rounds to 2^-43 the same way. Both counts are summed as
// 32-bit integers, the constants taken off once.
//
// k_verify_rows: clusters take one row after the other and keep it in shared memory and
// registers between finding its maximum and the sum, so that HBM is read once. 256 requests of
// 4 drafts, V = 128256 bf16: 591 MB in 153 us = 3.9 TB/s. Neither HBM nor issue (55%) is full:
// of 10.3 instructions a column some six are its own (a thread's eight columns take 48), the
// others a warp's share of the row's exchange, of waits and maxima, which 64 columns a thread
// carry. Doubles are divided by one lane: with every thread dividing its own the two units for
// doubles of an SM took the kernels 442 and 132 us.
// Rows go to clusters by stride over all that a batch may have, so of ragged requests one
// cluster may take twice as many as the mean, and the kernel as long as that one.
// k_verify_draw, a cluster for each request: the tests, then one pass over the row where a
// token is to be drawn (two rows after a refusal), each warp's vectors with a sum of their
// own; those the number falls into are read again (the same requests: 39 us).
#include "dependent.cuh"
#include "internal.cuh"

#include <atomic>
#include <cmath>

namespace fljsd {
namespace {

constexpr int kThreads = 512;  // of k_verify_draw
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kRowCtas = 3;    // of k_verify_rows on an SM
constexpr int kRowThreads = 256, kRowWarps = kRowThreads / 32;
constexpr int kKept = 8;       // vectors of 16 bytes that one of them keeps of a row
constexpr int64_t kMaxV = 1 << 20;  // sums of [w] stay below 2^63
constexpr double kUnit = 0x1p43;
constexpr float kC1 = 12.f, kC2 = 0x1.8p-20f;
constexpr uint32_t kBits1 = 0x41400000u, kBits2 = 0x35c00000u;
constexpr unsigned long long kNone = ~0ull;
constexpr unsigned long long kWaitNs = 4ull * 1000 * 1000 * 1000;  // a wait's limit
constexpr double kLog2e = 1.4426950408889634;
constexpr int kNoFall = 0x7fffffff;
constexpr float kLeastT = 0x1.7154780000000p-128f;  // the least T with a finite log2(e) / T in fp32

enum { kRowOk = 0, kRowBad = 1 };  // bad: NaN, +inf, or nothing but -inf

struct RowStat {
  double p;   // of the drafted token
  float m;    // largest logit
  float inv;  // 1 / total
  float c;    // log2(e) / T
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
  float t, c;
  int64_t n, requests, v;
  int max_drafts, slots, cluster;
  int64_t* out;
  int64_t* accepted;
  float* prob;
  int* status;
  unsigned long long wait_ns;
  bool stall;  // (a test's) the last CTA of a cluster copies nothing
  int* fall;   // the first request whose offsets fall, or kNoFall (offsets given)
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

// A double is never divided here but by one lane: an SM has two units for doubles.
struct Request {
  int64_t start;
  int drafts;
  float t;
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
  r.t = a.temperature ? a.temperature[b] : a.t;
  r.ok = r.start >= 0 && r.start <= end && end <= a.n && end - r.start <= a.max_drafts &&
         (r.t == 0.f || (r.t >= kLeastT && r.t < INFINITY));
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
// The largest of a thread's vectors; a NaN stays. (bf16 two at a time, fp32 three.)
template <typename T>
struct Top;
template <>
struct Top<float> {
  float m = -INFINITY;
  __device__ __forceinline__ static float most(float a, float b, float c) {
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
  }
  __device__ __forceinline__ void add(const uint4& q) {
    m = most(m, __uint_as_float(q.x), __uint_as_float(q.y));
    m = most(m, __uint_as_float(q.z), __uint_as_float(q.w));
  }
  __device__ __forceinline__ float value() const { return m; }
};
template <>
struct Top<__nv_bfloat16> {
  uint32_t m = 0xff80ff80u;  // -inf, -inf
  __device__ __forceinline__ void add(const uint4& q) {
    auto two = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    const __nv_bfloat162 x = __hmax2_nan(
        two(m), __hmax2_nan(__hmax2_nan(two(q.x), two(q.y)), __hmax2_nan(two(q.z), two(q.w))));
    m = *reinterpret_cast<const uint32_t*>(&x);
  }
  __device__ __forceinline__ float value() const {
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
};

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
// The warp's, of counts of up to 64 values each: |hi| < 2^27, |lo| < 2^28 a thread.
__device__ __forceinline__ unsigned long long warp_sum(const Count& c, uint32_t n) {
  const int hi = (int)(c.hi - n * kBits1), lo = (int)(c.lo - n * kBits2);
  const int h = __reduce_add_sync(0xffffffffu, hi);
  const int l1 = __reduce_add_sync(0xffffffffu, lo >> 12), l0 = __reduce_add_sync(0xffffffffu, lo & 0xfff);
  return ((unsigned long long)(uint32_t)h << 23) + ((long long)l1 << 12) + l0;
}

// Where a row lies: vectors [first, last) of N columns, the first one from the 16-byte
// boundary at or before the row's start; column j of vector k is k N - lead.
template <typename T>
struct Cut {
  int lead, first, last;
  __device__ __forceinline__ Cut(const T* row, int64_t v, int cluster, int rank) {
    lead = (int)(((uintptr_t)row & 15u) / sizeof(T));
    const int all = (int)((v + lead + Vec<T>::N - 1) / Vec<T>::N);
    const int per = (all + cluster - 1) >> (31 - __clz(cluster));  // (a power of two)
    first = min(rank * per, all);
    last = min(first + per, all);
  }
};

// A row that k_verify_rows is to take.
struct Row {
  const void* z;  // null: none
  float c;        // 0: greedy
  int request;
  bool is_draft;
  int64_t stat;   // where the results go
  int64_t at;     // the drafted token in question, -1 behind the last
};
template <typename T>
__device__ __forceinline__ Row row_of(const Args& a, int64_t unit) {
  Row r{};
  const int b = (int)((uint32_t)unit / (uint32_t)a.slots);  // (fewer than 2^31)
  const int slot = (int)unit - b * a.slots;
  const Request q = request(a, b);
  r.request = b;
  r.is_draft = slot > a.max_drafts;
  const int j = r.is_draft ? slot - a.max_drafts - 1 : slot;
  if (!q.ok || j >= q.drafts + (r.is_draft ? 0 : 1) || (r.is_draft && q.t == 0.f)) return r;
  r.c = q.t == 0.f ? 0.f : a.temperature ? (float)(kLog2e / (double)q.t) : a.c;
  r.at = j < q.drafts ? q.start + j : -1;
  r.stat = r.is_draft ? q.start + j : q.start + j + b;
  r.z = r.is_draft ? reinterpret_cast<const T*>(a.draft) + r.stat * a.ld_draft
                   : reinterpret_cast<const T*>(a.target) + r.stat * a.ld_target;
  return r;
}

// A CTA's part of a row: n vectors, column j0 at its start.
struct Part {
  const void* z;  // the row, null: none
  int64_t j0;
  int n;
  float c;
};
constexpr int kRing = 4, kTopRing = 8;
struct RowsShared {  // by the row's number
  unsigned long long full[2], empty[2];       // a row's copy has landed; it has moved on to registers
  unsigned long long tops[kTopRing], sums[kRing];  // the cluster's have arrived
  unsigned long long sum[kRing][kMaxCluster * kRowWarps];  // (at the first CTA)
  float top[kTopRing][kMaxCluster * kRowWarps];            // of the cluster's warps
  Part part[kRing];
  struct {  // the control warp's
    Row row;
    float zd, m;  // the drafted token's logit, and the row's largest
  } own[kRing];
  unsigned long long fell;  // the column warps have looked for offsets that fall
  int fall[kRowWarps];      // the first that each has found, or kNoFall
  volatile int abort;
};

__device__ __forceinline__ uint32_t at_shared(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint32_t at_cta(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at_shared(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void bar_init(const void* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(at_shared(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(const void* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(at_shared(bar)) : "memory");
}
__device__ __forceinline__ void bar_expect(const void* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(at_shared(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ unsigned long long now() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __noinline__ void pause() {  // 100 us
  const unsigned long long t0 = now();
  while (now() - t0 < 100'000) __nanosleep(1000);
}
// With a limit, after which the CTA's waits all end and the call's status word says so. (Not
// inlined, as pause() is not: a kernel of few rows is a chain of first passes through its code,
// and with a copy of this at each wait the row kernel took 25.9 us of 64 ragged requests, without
// 25.0.)
__device__ __noinline__ bool bar_wait_long(uint32_t bar, uint32_t parity, volatile int* abort, int* status, unsigned long long ns) {
  unsigned long long t0 = 0;
  for (uint32_t it = 0;; ++it) {
    if (bar_try(bar, parity)) return true;
    if ((it & 255u) == 255u) {  // (reading the timer takes longer than most waits)
      if (*abort) return false;
      const unsigned long long t = now();
      if (!t0) t0 = t;
      if (t - t0 > ns) {
        *abort = 1;
        atomicExch(status, (int)FLJSD_ERR_TIMEOUT);
        return false;
      }
    }
  }
}
// (by whole warps: all go on, or none)
__device__ __forceinline__ bool bar_wait(const void* bar, uint32_t parity, volatile int* abort, const Args& a) {
  const uint32_t b = at_shared(bar);
  bool ok = bar_try(b, parity);
  if (!__all_sync(0xffffffffu, ok)) {
    if (!ok) ok = bar_wait_long(b, parity, abort, a.status, a.wait_ns);
    ok = __all_sync(0xffffffffu, ok) != 0;
  } else {
    ok = true;
  }
  return ok;
}
// Values to another CTA of the cluster, counted by a barrier there.
__device__ __forceinline__ void send(const float* to, const void* bar, uint32_t rank, float x) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(at_cta(to, rank)),
               "r"(__float_as_uint(x)), "r"(at_cta(bar, rank))
               : "memory");
}
__device__ __forceinline__ void send(const unsigned long long* to, const void* bar, uint32_t rank, unsigned long long x) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(at_cta(to, rank)),
               "l"(x), "r"(at_cta(bar, rank))
               : "memory");
}

// Clusters that stay, a row after the other. A warp of its own finds the rows and has their
// parts copied to shared memory, two ahead; row i moves on to registers before row i + 2
// takes its place. Every warp sends what it finds to all CTAs (its maximum) or to the first
// one (its sum); row i + 1's maximum is sent before row i's is waited for, so nobody waits
// for what is only just on its way.
// A place is written again when its last reader is done. Nobody sends row i's maximum
// without having those of row i - 2 from all CTAs, and none of these comes from a CTA whose
// control warp has not had that row copied. So by the time of row i + 8's maxima every
// control warp has had row i + 6 copied, two iterations after it has read row i's, and
// every other warp has read them before it sent row i + 2's; and by the time of row
// i + 4's sums the first CTA's control warp has had row i + 4 copied, after it has written
// row i's.
template <typename T>
__global__ void __launch_bounds__(kRowThreads + 32, kRowCtas) k_verify_rows(const Args a) {
  constexpr int N = Vec<T>::N;
  extern __shared__ __align__(128) uint4 s_rows[];  // [2][kKept * kRowThreads]
  __shared__ __align__(16) RowsShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cta_rank();
  let_next_launch();
  if (blockIdx.x == 0 && tid == 0) *a.status = 0;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(&sh.full[i], 1);
      bar_init(&sh.empty[i], kRowWarps);
    }
    for (int i = 0; i < kTopRing; ++i) bar_init(&sh.tops[i], 1);
    for (int i = 0; i < kRing; ++i) bar_init(&sh.sums[i], 1);
    bar_init(&sh.fell, kRowWarps);
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  cluster_sync();
  auto part_of = [&](int i) -> const Part& { return sh.part[i % kRing]; };
  auto top_of = [&](int i) {
    float m = -INFINITY;
    for (int e = lane; e < a.cluster * kRowWarps; e += 32) m = max_nan(m, sh.top[i % kTopRing][e]);
    asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(m));
    return m;
  };
  auto has_tops = [&](int i) { return bar_wait(&sh.tops[i % kTopRing], (i / kTopRing) & 1, &sh.abort, a); };
  if (warp == kRowWarps) {  // ---------------- control ----------------
    // Rows are looked for 32 units at a time, a lane to each.
    const uint32_t units = (uint32_t)(a.requests * a.slots), step = gridDim.x / a.cluster;
    uint32_t first_unit = blockIdx.x / a.cluster, found = 0;  // lanes whose row is still to come
    Row mine{};
    int64_t mine_j0 = 0;
    int mine_n = 0, src = 0;
    float mine_zd = -INFINITY;
    bool looked_up = false;
    auto look_up = [&]() {  // the drafted tokens' logits
      if (looked_up) return;
      if (rank == 0 && mine.z && mine.at >= 0) {
        const int64_t d = a.tokens[mine.at];
        if (d >= 0 && d < a.v) mine_zd = value_at(reinterpret_cast<const T*>(mine.z) + d);
      }
      looked_up = true;
    };
    auto keep_zd = [&](int j, int lane_of) {
      look_up();
      const float zd = __shfl_sync(0xffffffffu, mine_zd, lane_of);
      if (lane == 0) sh.own[j % kRing].zd = zd;
    };
    bool waiting = false;  // row 0's logit is not looked up yet: the first copies go before it
    int src_first = 0;
    auto catch_up = [&]() {
      if (waiting) keep_zd(0, src_first);
      waiting = false;
    };
    auto next_row = [&]() {
      while (!found && first_unit < units) {
        catch_up();
        const uint64_t unit = first_unit + (uint64_t)lane * step;
        mine = unit < units ? row_of<T>(a, (int64_t)unit) : Row{};
        if (mine.z) {
          const Cut<T> cut(reinterpret_cast<const T*>(mine.z), a.v, a.cluster, rank);
          mine_j0 = (int64_t)cut.first * N - cut.lead;
          mine_n = cut.last - cut.first;
        }
        mine_zd = -INFINITY;
        looked_up = false;
        found = __ballot_sync(0xffffffffu, mine.z != nullptr);
        const uint64_t on = first_unit + 32ull * step;
        first_unit = on < units ? (uint32_t)on : units;
      }
      if (!found) return false;
      src = __ffs(found) - 1;
      found &= found - 1;
      return true;
    };
    // row j into its place; false: there is none
    auto bring = [&](int j, bool& ok) {
      const bool there = next_row();
      // (where that wait ran out the place and its barriers are not touched)
      if (j >= 2 && !bar_wait(&sh.empty[j & 1], ((j >> 1) & 1) ^ 1, &sh.abort, a)) ok = false;
      if (!ok) return false;
      Part q{};
      if (there) {
        q.z = reinterpret_cast<const void*>(__shfl_sync(0xffffffffu, (unsigned long long)mine.z, src));
        q.j0 = __shfl_sync(0xffffffffu, mine_j0, src);
        q.n = __shfl_sync(0xffffffffu, mine_n, src);
        q.c = __shfl_sync(0xffffffffu, mine.c, src);
        const T* z = reinterpret_cast<const T*>(q.z);
        const int lo = q.n > 0 && q.j0 < 0 ? 1 : 0;
        const int most = kKept * kRowThreads;
        int hi = max(lo, q.n > 0 && q.j0 + (int64_t)q.n * N > a.v ? q.n - 1 : q.n);
        hi = min(hi, most);
        uint4* to = s_rows + (j & 1) * most;
        const uint32_t bytes = (uint32_t)(hi - lo) * 16;
        if (lane == 0 && bytes && !(a.stall && rank == a.cluster - 1)) {  // (counted below: the row is not there before that)
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          asm volatile(
              "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                  at_shared(to + lo)),
              "l"(z + q.j0 + (int64_t)lo * N), "r"(bytes), "r"(at_shared(&sh.full[j & 1]))
              : "memory");
        }
        // what is not copied whole: the vectors at the row's ends, and places that stay empty
        if (lane < lo) to[lane] = load(z, q.j0, a.v, false);
        constexpr uint32_t w = Vec<T>::kMasked | (sizeof(T) == 4 ? 0u : Vec<T>::kMasked << 16);
        for (int k = hi + lane; k < most; k += 32)
          to[k] = k < q.n ? load(z, q.j0 + (int64_t)k * N, a.v, false) : make_uint4(w, w, w, w);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          sh.part[j % kRing] = q;
          bar_expect(&sh.full[j & 1], bytes);
          bar_expect(&sh.tops[j % kTopRing], a.cluster * kRowWarps * 4);
          if (rank == 0) bar_expect(&sh.sums[j % kRing], a.cluster * kRowWarps * 8);
        }
        if (lane == src) sh.own[j % kRing].row = mine;
        if (j == 0) {
          src_first = src;
          waiting = true;
        } else {
          catch_up();
          keep_zd(j, src);
        }
      } else if (lane == 0) {
        sh.part[j % kRing] = q;
        bar_arrive(&sh.full[j & 1]);
      }
      __syncwarp();
      return there;
    };
    int fall = -1;  // as the other warps have found it
    auto first_fall = [&]() {
      if (fall < 0) {
        fall = kNoFall;
        if (a.offsets && bar_wait(&sh.fell, 0, &sh.abort, a))
          for (int w = 0; w < kRowWarps; ++w) fall = min(fall, sh.fall[w]);
      }
      return fall;
    };
    // what row i leaves to be written
    auto finish = [&](int i) {
      if (!bar_wait(&sh.sums[i % kRing], (i / kRing) & 1, &sh.abort, a)) return;
      const auto& own = sh.own[i % kRing];
      const bool greedy = own.row.c == 0.f;
      unsigned long long sum = greedy ? kNone : 0ull;
      for (int e = lane; e < a.cluster * kRowWarps; e += 32) {
        const unsigned long long x = sh.sum[i % kRing][e];
        sum = greedy ? min(sum, x) : sum + x;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long x = __shfl_xor_sync(0xffffffffu, sum, o);
        sum = greedy ? min(sum, x) : sum + x;
      }
      RowStat s{0.0, own.m, 0.f, own.row.c, -1, fabsf(own.m) < INFINITY ? kRowOk : kRowBad};
      if (s.state == kRowOk && greedy) s.best = (int)sum;
      if (s.state == kRowOk && !greedy) {
        // two quotients at once, a lane to each
        const double wd = (double)ex2(__fmul_rn(__fsub_rn(own.zd, own.m), own.row.c));
        const double q = (lane == 0 ? wd : 1.0) / ((double)sum / kUnit);
        s.p = q;
        s.inv = (float)__shfl_sync(0xffffffffu, q, 1);
      }
      const bool stands = own.row.request < first_fall();
      if (lane == 0 && stands) (own.row.is_draft ? a.stat_d : a.stat_t)[own.row.stat] = s;
    };
    bool ok = true;
    bool here = bring(0, ok), next = here && bring(1, ok);
    catch_up();
    int i = 0, brought = here ? 2 : 1;
    for (; here && ok; ++i) {
      const bool after = next && bring(i + 2, ok);
      brought += next && ok;
      if (rank == 0 && i > 0) finish(i - 1);
      ok = has_tops(i) && ok;
      const float m = top_of(i);
      if (lane == 0) sh.own[i % kRing].m = m;
      __syncwarp();
      here = next;
      next = after;
    }
    if (rank == 0 && i > 0) finish(i - 1);
    if (a.offsets && blockIdx.x == 0) {
      const int first = first_fall();
      if (lane == 0) *a.fall = first;
    }
    unsigned long long t0 = 0;
    for (int j = max(0, brought - 2); j < brought; ++j)  // no copy is under way at the end
      while (!bar_try(at_shared(&sh.full[j & 1]), (j >> 1) & 1)) {
        if (!t0) t0 = now();
        if (now() - t0 > a.wait_ns) break;
      }
  } else {  // ---------------- columns ----------------
    auto rest = [&](const Part& q, auto&& f) {  // vectors beyond those kept, read again
      for (int k = kKept * kRowThreads + tid; k < q.n; k += kRowThreads)
        f(load(reinterpret_cast<const T*>(q.z), q.j0 + (int64_t)k * N, a.v, true), k);
    };
    // whether there is a row i, whose maximum is sent
    auto send_top = [&](int i) {
      if (!bar_wait(&sh.full[i & 1], (i >> 1) & 1, &sh.abort, a)) return false;
      const Part& q = part_of(i);
      if (!q.z) return false;
      const uint4* mine = s_rows + (i & 1) * kKept * kRowThreads + tid;
      Top<T> top;
#pragma unroll
      for (int k = 0; k < kKept; ++k) top.add(mine[k * kRowThreads]);
      if (q.n > kKept * kRowThreads) rest(q, [&](const uint4& x, int) { top.add(x); });
      float m = top.value();
      asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(m));
      if (lane < a.cluster)
        send(&sh.top[i % kTopRing][rank * kRowWarps + warp], &sh.tops[i % kTopRing], lane, m);
      return true;
    };
    bool here = send_top(0);
    // While the first maxima are on their way:
    // What belongs to no request, or to one that is refused, is accepted with 0: k_verify_draw
    // writes the other requests' over it.
    if (a.offsets || a.temperature)
      for (int i = blockIdx.x * kRowThreads + tid; i < (int)a.n; i += gridDim.x * kRowThreads) a.prob[i] = 0.f;
    // From the first offsets that fall on, a request may claim rows that others have too: whose
    // statistics stood in the end would be chance. So theirs are not written.
    if (a.offsets && rank == 0) {
      int first = kNoFall;
      for (int b0 = tid; b0 < (int)a.requests && first == kNoFall; b0 += 4 * kRowThreads) {
#pragma unroll
        for (int i = 3; i >= 0; --i) {
          const int b = b0 + i * kRowThreads;
          if (b < (int)a.requests && a.offsets[b] > a.offsets[b + 1]) first = b;
        }
      }
      first = __reduce_min_sync(0xffffffffu, first);
      if (lane == 0) {
        sh.fall[warp] = first;
        bar_arrive(&sh.fell);
      }
      __syncwarp();
    }
    for (int i = 0; here; ++i) {
      uint4 raw[kKept];
#pragma unroll
      for (int k = 0; k < kKept; ++k) raw[k] = s_rows[((i & 1) * kKept + k) * kRowThreads + tid];
      __syncwarp();
      if (lane == 0) bar_arrive(&sh.empty[i & 1]);
      here = send_top(i + 1);
      if (!has_tops(i)) break;
      const float m = top_of(i), c = part_of(i).c;
      const int n_vecs = part_of(i).n;
      const bool bad = !(fabsf(m) < INFINITY);
      unsigned long long sum = 0;
      if (!bad && c != 0.f) {
        Count n;
#pragma unroll
        for (int k = 0; k < kKept; ++k) {
          float2 x[N / 2];
          values<T>(raw[k], x);
#pragma unroll
          for (int e = 0; e < N / 2; ++e) n.add(weights(x[e], m, c));
        }
        sum = warp_sum(n, kKept * N);
        if (n_vecs > kKept * kRowThreads) {
          unsigned long long more = 0;
          rest(part_of(i), [&](const uint4& q, int) {
            float2 x[N / 2];
            values<T>(q, x);
            Count n;
#pragma unroll
            for (int e = 0; e < N / 2; ++e) n.add(weights(x[e], m, c));
            more += n.sum(N);
          });
          sum += warp_sum(more);
        }
      } else if (!bad) {
        sum = kNone;
        const int64_t j0 = part_of(i).j0;
        auto look = [&](const uint4& q, int k) {
          float2 x[N / 2];
          values<T>(q, x);
#pragma unroll
          for (int e = 0; e < N / 2; ++e) {
            if (x[e].x == m) sum = min(sum, (unsigned long long)(j0 + (int64_t)k * N + 2 * e));
            if (x[e].y == m) sum = min(sum, (unsigned long long)(j0 + (int64_t)k * N + 2 * e + 1));
          }
        };
#pragma unroll
        for (int k = 0; k < kKept; ++k) look(raw[k], k * kRowThreads + tid);
        rest(part_of(i), look);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum = min(sum, __shfl_xor_sync(0xffffffffu, sum, o));
      }
      if (lane == 0) send(&sh.sum[i % kRing][rank * kRowWarps + warp], &sh.sums[i % kRing], 0, sum);
    }
  }
  // No CTA leaves while another sends to it. (Where a wait ran out, what was sent last has not
  // been waited for: a pause for what this CTA sent, and one for what others did.)
  const bool aborted = sh.abort != 0;
  if (aborted) pause();
  cluster_sync();
  if (aborted) pause();
}

// Columns [j, j + N) of a row that lies to 16 bytes otherwise than j does: from the two
// aligned vectors that hold them, where both lie within the row.
template <typename T>
__device__ __forceinline__ uint4 load_apart(const T* row, int64_t j, int64_t v) {
  constexpr int N = Vec<T>::N;
  if (j < N || j + 2 * N > v) return load(row, j, v, false);
  const uintptr_t at = (uintptr_t)(row + j);
  const uint4* q = reinterpret_cast<const uint4*>(at & ~(uintptr_t)15);
  const uint4 lo = q[0], hi = q[1];
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  const int words = (int)(at & 15u) / 4, bits = (int)(at & 3u) * 8;
  uint4 r;
  auto pick = [&](int o) {
    r.x = __funnelshift_r(w[o], w[o + 1], bits);
    r.y = __funnelshift_r(w[o + 1], w[o + 2], bits);
    r.z = __funnelshift_r(w[o + 2], w[o + 3], bits);
    r.w = __funnelshift_r(w[o + 3], w[o + 4 < 8 ? o + 4 : 7], bits);
  };
  switch (words) {  // (the same in the whole row)
    case 0: pick(0); break;
    case 1: pick(1); break;
    case 2: pick(2); break;
    default: pick(3); break;
  }
  return r;
}

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at_shared(dst)), "l"(src) : "memory");
}

// What the next token is drawn from: p, or p - q.
template <typename T>
struct Residual {
  const T* p;
  const T* q;  // or null
  float mp, mq, c, ip, iq;
  int64_t v, without;  // a column whose q is 1, or -1
  bool q_whole;        // q lies to 16 bytes as p does (or there is none)
  struct Raw {
    uint4 p, q;
  };
  __device__ __forceinline__ Raw fetch(int64_t j) const {
    Raw r;
    if (q_whole && j >= 0 && j + Vec<T>::N <= v) {
      r.p = *reinterpret_cast<const uint4*>(p + j);
      r.q = q ? *reinterpret_cast<const uint4*>(q + j) : r.p;
    } else {
      r.p = load(p, j, v, true);
      r.q = q ? q_whole ? load(q, j, v, true) : load_apart(q, j, v) : r.p;
    }
    return r;
  }
  __device__ __forceinline__ void get(const Raw& raw, int64_t j, float2 (&r)[Vec<T>::N / 2]) const {
    constexpr int N = Vec<T>::N;
    float2 z[N / 2], y[N / 2];
    values<T>(raw.p, z);
    values<T>(raw.q, y);
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

struct DrawShared {
  unsigned long long sum[kMaxCluster];
  unsigned long long warp[kWarps];
  int accepted;
};
constexpr int kAhead = 2;  // vectors of each row that a thread has in flight

// The first of n sums (a place of its own in each lane, 32 at a time) whose running sum
// exceeds t; `run`: the sum of those before it.
template <typename F>
__device__ __forceinline__ int find_sum(int n, unsigned long long t, unsigned long long& run, const F& sum_of) {
  const int lane = threadIdx.x & 31;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const unsigned long long own = i0 + lane < n ? sum_of(i0 + lane) : 0ull;
    unsigned long long x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const uint32_t over = __ballot_sync(0xffffffffu, run + x > t);
    if (over) {
      const int l = __ffs(over) - 1;
      run += __shfl_sync(0xffffffffu, x - own, l);
      return i0 + l;
    }
    run += __shfl_sync(0xffffffffu, x, 31);
  }
  return 0;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) k_verify_draw(const Args a) {
  constexpr int N = Vec<T>::N;
  __shared__ DrawShared sh;
  extern __shared__ uint4 s_raw[];  // [2][p, q][kAhead][kThreads]: a thread's own, a turn ahead
  unsigned long long* s_sums = reinterpret_cast<unsigned long long*>(s_raw + 4 * kAhead * kThreads);  // [turns][kWarps]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cta_rank();
  const int64_t b = blockIdx.x / a.cluster;
  if (a.cluster > 1) cluster_arrive();  // (none is written to before it has started)
  wait_for_previous();
  const int fall = a.offsets ? *a.fall : kNoFall;
  Request q = request(a, b);
  if (b >= fall) {
    q.ok = false;
    q.drafts = 0;
  }
  const bool greedy = q.t == 0.f;
  // the tests, a lane to each; every CTA of the cluster makes them
  double pd = 0.0, qd = -1.0;  // of this lane's last test; qd < 0: refused anyway
  int64_t mine_at = -1;
  auto tell = [&]() {  // the probability of that test's acceptance
    if (rank == 0 && mine_at >= 0)
      a.prob[mine_at] = qd < 0.0    ? 0.f
                        : qd == 0.0 ? (pd > 0.0 ? 1.f : 0.f)
                        : pd < qd   ? (float)(pd / qd)
                                    : 1.f;
  };
  if (warp == 0) {
    int accepted = 0;
    bool going = true, refuse = !q.ok;
    for (int j0 = 0; j0 < q.drafts; j0 += 32) {
      if (j0 > 0) tell();
      const int j = j0 + lane;
      bool hit = false;
      mine_at = -1;
      pd = 0.0;
      qd = -1.0;
      if (j < q.drafts) {
        const int64_t at = q.start + j, d = a.tokens[at];
        const RowStat st = a.stat_t[at + b];
        const bool drafted = a.draft && !greedy;
        const RowStat sd = drafted ? a.stat_d[at] : RowStat{1.0, 0.f, 0.f, 0.f, 0, kRowOk};
        const float u = a.u[at];
        mine_at = at;
        const bool in = d >= 0 && d < a.v;
        refuse |= !in;
        if (in && st.state == kRowOk && sd.state == kRowOk) {
          if (greedy) {
            hit = d == st.best;
            pd = qd = hit ? 1.0 : -1.0;
          } else {
            pd = st.p;
            qd = sd.p;  // (1 without draft)
            hit = (double)u * qd < pd;
          }
        }
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
      sh.accepted = accepted;
      // (a wait of k_verify_rows that ran out stays known: there are no results then)
      static_assert((int)FLJSD_ERR_TIMEOUT > (int)FLJSD_ERR_INVALID_ARG, "the greater one stays");
      if (refuse && rank == 0) atomicMax(a.status, (int)FLJSD_ERR_INVALID_ARG);
    }
  }
  __syncthreads();
  if (a.cluster > 1) cluster_wait();
  const int accepted = sh.accepted;
  const int64_t at = q.start + accepted;
  RowStat sp{};
  if (q.ok) sp = a.stat_t[at + b];
  int64_t token = -1;
  if (q.ok && greedy) {
    token = sp.best;
  } else if (q.ok && sp.state == kRowOk) {
    Residual<T> res{};
    res.p = reinterpret_cast<const T*>(a.target) + (at + b) * a.ld_target;
    res.mp = sp.m;
    res.c = sp.c;
    res.ip = sp.inv;
    res.v = a.v;
    res.without = -1;
    res.q_whole = true;
    if (accepted < q.drafts) {
      if (a.draft) {
        const RowStat sd = a.stat_d[at];
        if (sd.state == kRowOk) {
          res.q = reinterpret_cast<const T*>(a.draft) + at * a.ld_draft;
          res.mq = sd.m;
          res.iq = sd.inv;
          res.q_whole = (((uintptr_t)res.p ^ (uintptr_t)res.q) & 15u) == 0;
        }
      } else {
        res.without = a.tokens[at];
      }
    }
    const Cut<T> cut(res.p, a.v, a.cluster, rank);
    // a warp takes kAhead x 32 neighbouring vectors in a turn
    const int turns = (cut.last - cut.first + kThreads * kAhead - 1) / (kThreads * kAhead);
    auto column_of = [&](int t, int w, int i) {  // past the row where there is none
      const int k = cut.first + ((t * kWarps + w) * kAhead + i) * 32 + lane;
      return k < cut.last ? (int64_t)k * N - cut.lead : a.v;
    };
    auto column = [&](int it) { return column_of(it / kAhead, warp, it % kAhead); };
    unsigned long long before = 0, total = 0, mine = 0;
    for (int turn = 0; turn < 2; ++turn) {
      mine = 0;
      auto ask = [&](int t) {
        if (t < turns) {
          uint4* to = s_raw + (t & 1) * 2 * kAhead * kThreads + tid;
#pragma unroll
          for (int i = 0; i < kAhead; ++i, to += kThreads) {
            const int64_t j = column(t * kAhead + i);
            if (res.q_whole && j >= 0 && j + N <= a.v) {
              copy16(to, res.p + j);
              if (res.q) copy16(to + kAhead * kThreads, res.q + j);
            } else {
              const typename Residual<T>::Raw r = res.fetch(j);
              to[0] = r.p;
              to[kAhead * kThreads] = r.q;
            }
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      ask(0);
      for (int t = 0; t < turns; ++t) {
        ask(t + 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        typename Residual<T>::Raw raw[kAhead];
        const uint4* from = s_raw + (t & 1) * 2 * kAhead * kThreads + tid;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          raw[i].p = from[i * kThreads];
          raw[i].q = res.q ? from[(kAhead + i) * kThreads] : raw[i].p;
        }
        Count n;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          float2 r[N / 2];
          res.get(raw[i], column(t * kAhead + i), r);
#pragma unroll
          for (int e = 0; e < N / 2; ++e) n.add(r[e]);
        }
        const unsigned long long s = warp_sum(n, kAhead * N);
        if (lane == 0) s_sums[t * kWarps + warp] = s;
        mine += s;
      }
      if (lane == 0) sh.warp[warp] = mine;
      __syncthreads();
      mine = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mine += sh.warp[w];
      if (a.cluster > 1) {
        if (warp == 0) {
          if (lane < a.cluster) put_remote(&sh.sum[rank], lane, mine);
        }
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
    unsigned long long t = 0;
    if (warp == 0) {
      const double want = (double)a.u_draw[b] * (double)total;
      t = want > 0.0 ? want >= (double)total ? total - 1 : (unsigned long long)want : 0ull;
      t = min(t, total - 1);
    }
    if (warp == 0 && t >= before && t - before < mine) {
      t -= before;
      // the warp's vectors that hold it, the lane's, the column
      unsigned long long run = 0;
      const int found = find_sum(turns * kWarps, t, run, [&](int i) { return s_sums[i]; });
      // of its vectors the 32 that hold it, the lane's, the column
      float2 r[N / 2];
      int64_t j0 = 0;
#pragma unroll 1
      for (int i = 0; i < kAhead; ++i) {
        j0 = column_of(found / kWarps, found % kWarps, i);
        res.get(res.fetch(j0), j0, r);
        Count n;
#pragma unroll
        for (int e = 0; e < N / 2; ++e) n.add(r[e]);
        const unsigned long long s = warp_sum(n, N);
        if (run + s > t) break;
        run += s;
      }
      unsigned long long one[N], x = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        Count n;
        n.add(make_float2(i & 1 ? r[i / 2].y : r[i / 2].x, 0.f));
        one[i] = n.sum(2);
        x += one[i];
      }
      const int l = find_sum(32, t, run, [&](int) { return x; });
      if (lane == l) {
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
    if (warp == 0) tell();
  }
  if (a.cluster > 1) cluster_sync();  // no CTA leaves while another writes to it
}

// CTAs to a row of k_verify_rows: enough to keep all of it, more where there are few rows.
int cluster_of_rows(int64_t v, int size, int64_t rows) {
  const int64_t all = (v * size + 30) / 16;  // vectors, wherever the row starts
  int c = 1;
  while (c < kMaxCluster && (int64_t)c * kKept * kRowThreads < all) c *= 2;
  while (c < kMaxCluster && rows * c * 2 <= num_sms() && (int64_t)c * 512 < all) c *= 2;
  return c;
}
// CTAs to a request of k_verify_draw: as many as fill the SMs twice over, and have a vector
// for each thread. (256 requests, V = 128256: 8 CTAs 85 us, 1 CTA 49, before rows came a turn ahead.)
int cluster_of_draws(int64_t v, int size, int64_t requests) {
  const int64_t all = (v * size + 30) / 16;
  int c = 1;
  while (c < kMaxCluster && requests * c <= num_sms() && (int64_t)c * kThreads < all) c *= 2;
  return c;
}

// A kernel's launch in clusters, and how many of them the GPU holds at a time.
struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2] = {};
  Launch(int threads, int cluster, size_t smem, cudaStream_t st) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)cluster, 1, 1};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
};
// A kernel's attributes, set once on each device: clusters of 16, dynamic shared memory.
template <auto KERNEL>
cudaError_t allow(int smem) {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaGetDevice(&dev);
  const bool known = dev >= 0 && dev < 64;
  if (known && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && known) done[dev].store(true, std::memory_order_relaxed);
  return e;
}
template <typename T>
int resident(Launch& l, int cluster) {
  static std::atomic<int> cached[64][kMaxCluster + 1];
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  const bool known = dev >= 0 && dev < 64;
  if (known && (n = cached[dev][cluster].load(std::memory_order_relaxed)) > 0) return n;
  l.cfg.gridDim = dim3(cluster);
  if (cudaOccupancyMaxActiveClusters(&n, k_verify_rows<T>, &l.cfg) != cudaSuccess || n < 1) n = 1;
  if (known) cached[dev][cluster].store(n, std::memory_order_relaxed);
  return n;
}

template <typename T>
cudaError_t launch(Args a, cudaStream_t st) {
  a.slots = a.max_drafts + 1 + (a.draft ? a.max_drafts : 0);
  const int64_t rows = a.requests * a.slots;
  a.cluster = cluster_of_rows(a.v, sizeof(T), rows);
  constexpr int kRowsBytes = 2 * kKept * kRowThreads * 16, kDrawBytes = 128 * 1024;
  Launch l(kRowThreads + 32, a.cluster, kRowsBytes, st);
  cudaError_t e = allow<k_verify_rows<T>>(kRowsBytes);
  if (e != cudaSuccess) return e;
  const int64_t fit = resident<T>(l, a.cluster);
  l.cfg.gridDim = dim3((unsigned)((rows < fit ? rows : fit) * a.cluster));
  trace_begin(FLJSD_KERNEL_SMALL, st);
  e = cudaLaunchKernelEx(&l.cfg, k_verify_rows<T>, a);
  trace_end(FLJSD_KERNEL_SMALL, st);
  if (e != cudaSuccess) return e;
  a.cluster = cluster_of_draws(a.v, sizeof(T), a.requests);
  const int64_t vecs = (a.v * (int64_t)sizeof(T) + 30) / 16;
  const int64_t turns = ((vecs + a.cluster - 1) / a.cluster + kThreads * kAhead - 1) / (kThreads * kAhead);
  constexpr int kRawBytes = 4 * kAhead * kThreads * 16;
  static_assert((kMaxV * 4 + 30) / 16 / 32 / kAhead * 8 + kWarps * 8 + kRawBytes < kDrawBytes, "sums of one CTA's turns");
  Launch d(kThreads, a.cluster, kRawBytes + (size_t)(turns * kWarps * sizeof(unsigned long long)), st);
  d.cfg.gridDim = dim3((unsigned)(a.requests * a.cluster));
  d.cfg.numAttrs = 2;
  e = allow<k_verify_draw<T>>(kDrawBytes);
  if (e != cudaSuccess) return e;
  trace_begin(FLJSD_KERNEL_SMALL, st);
  e = cudaLaunchKernelEx(&d.cfg, k_verify_draw<T>, a);
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
  if (!temperatures && !(temperature == 0.f || (temperature >= kLeastT && std::isfinite(temperature))))
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
  a.c = temperature > 0.f ? (float)(kLog2e / (double)temperature) : 0.f;
  a.n = drafts;
  a.requests = requests;
  a.v = v;
  a.max_drafts = max_drafts;
  a.out = out;
  a.accepted = accepted;
  a.prob = accept_prob;
  a.status = reinterpret_cast<int*>(workspace);
  a.fall = a.status + 1;
  a.stall = (stalled() & FLJSD_STALL_VERIFY) != 0;
  a.wait_ns = a.stall ? kStallNs : kWaitNs;
  a.stat_t = reinterpret_cast<RowStat*>(reinterpret_cast<char*>(workspace) + kStatusBytes);
  a.stat_d = a.stat_t + requests + drafts;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == FLJSD_BF16 ? launch<__nv_bfloat16>(a, st) : launch<float>(a, st);
  return e == cudaSuccess ? FLJSD_OK : FLJSD_ERR_CUDA;
}
