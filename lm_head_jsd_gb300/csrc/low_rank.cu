// Low-rank adapters of many requests on the output of a projection that they share:
//   out_t = y_t + scale_a B_a (A_a x_t),  a = index[t]  (-1: out_t = y_t)
//
// Bound by reading and writing y (few tokens of many adapters: by reading their B). The
// tokens are first sorted by adapter and cut into tiles of up to 64 that share one
// (k_lr_plan); both products of a tile then run on the tensor cores with the adapter's
// rows as the instruction's 128 rows and the tokens as its columns, so that a tile of one
// token costs 16 columns and not 128 rows:
//  - k_lr_shrink: s = scale A x of a tile. A cluster of eight CTAs splits k and adds its
//    parts in shared memory, in one order. s is written as two bf16, the nearest and what
//    is left (2^-16 of s at most is lost): one would be 2^-8 off, as much as bf16's own rounding.
//  - k_lr_expand: y + B s for 256 columns at a time. Accumulator rows i of two products
//    hold columns 2 i and 2 i + 1, so that a thread reads and writes pairs and a warp 64
//    neighbouring columns of a token.
#include "dependent.cuh"
#include "elect.cuh"
#include "gemm_tc_kernel.cuh"

namespace fljsd {
namespace {

using namespace tcgemm;

constexpr int kTile = 64;       // tokens of a tile
constexpr int kCols = 256;      // columns of y that a block of k_lr_expand takes
constexpr int kMaxRank = 128;
constexpr int kMaxAdapters = 4096;
constexpr int kSplit = 8;       // CTAs of k_lr_shrink to a tile
constexpr int kOwn = kTile / kSplit;
constexpr int kThreads = 128;
constexpr int kPlanThreads = 1024;
constexpr int kStages = 4;
constexpr int kXStage = kTile * 128;  // 64 tokens x 64 of k
constexpr int kBlocks = 4;      // blocks of columns to a CTA of k_lr_expand

struct Tile {
  int adapter, first, count;  // tokens order[first .. first + count)
};

struct Args {
  int64_t tokens, k, n, ldx, ldy, ldo;
  int rank, rk, adapters, max_tiles;  // rk: rank up to a multiple of 16
  const __nv_bfloat16 *x, *a, *b;
  const int64_t* index;
  const float* scales;
  const void* y;
  void* out;
  bool vec_k, pairs, copy;
  int* status;
  int* num_tiles;
  Tile* tiles;
  int* order;
  char* s;  // a tile's s as it lies in shared memory: [nearest, rest] of kTile rows
};

// Operands lie in shared memory as 8 x 16-byte matrices, those of 8 rows side by side.
__host__ __device__ constexpr uint32_t place(int row, int piece, int pieces) {
  return (uint32_t)((row / 8) * pieces * 128 + piece * 128 + (row % 8) * 16);
}
// K-major, no swizzle: 128 bytes from one matrix to the next along k, `pieces` of them
// from 8 rows to the next 8.
__device__ __forceinline__ uint64_t desc(uint32_t addr, int pieces) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)(128 >> 4) << 16 |
         (uint64_t)((pieces * 128) >> 4) << 32 | (uint64_t)1 << 46;
}
// M = 128, fp32 accumulator, bf16 operands, n columns.
__device__ __forceinline__ uint32_t idesc_of(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  const int bytes = there ? 16 : 0;  // the rest is zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int KEEP>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(KEEP) : "memory");
}
// Eight elements of a row at k0, of any alignment.
__device__ __forceinline__ void copy8(uint32_t dst, const __nv_bfloat16* row, int64_t k0, int64_t k, bool vec,
                                      const void* any) {
  if (vec && k0 + 8 <= k) {
    copy16(dst, row + k0, true);
  } else if (k0 >= k) {
    copy16(dst, any, false);
  } else {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = (k0 + 2 * i < k ? p[k0 + 2 * i] : 0u) | ((k0 + 2 * i + 1 < k ? (uint32_t)p[k0 + 2 * i + 1] : 0u) << 16);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                 : "memory");
  }
}

// Waits with a limit (10 s), after which the call's status word says so.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = globaltimer();
  for (uint32_t it = 0;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 63u && globaltimer() - t0 > kTimeoutNs) {
      atomicExch(status, (int)FLJSD_ERR_TIMEOUT);
      return false;
    }
  }
}

// Sorts the tokens by adapter (those without one last, where they are to be copied) and
// cuts each adapter's into tiles. Which of an adapter's tokens comes first changes
// nothing in their results.
__global__ void __launch_bounds__(kPlanThreads) k_lr_plan(const Args a) {
  extern __shared__ int s_count[];  // [adapters + 1], then the places
  __shared__ int s_warp[2][kPlanThreads / 32];
  __shared__ int s_carry[2];
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int groups = a.adapters + 1;
  int* s_place = s_count + groups;
  let_next_launch();
  for (int i = tid; i < groups; i += kPlanThreads) s_count[i] = 0;
  if (tid == 0) s_carry[0] = s_carry[1] = s_bad = 0;
  __syncthreads();
  auto group = [&](int64_t t) {  // -1: left as it is
    const int64_t i = a.index[t];
    if (i >= 0 && i < a.adapters) return (int)i;
    if (i != -1) s_bad = 1;
    return a.copy ? a.adapters : -1;
  };
  for (int64_t t = tid; t < a.tokens; t += kPlanThreads) {
    const int g = group(t);
    if (g >= 0) atomicAdd(&s_count[g], 1);
  }
  __syncthreads();
  for (int g0 = 0; g0 < groups; g0 += kPlanThreads) {
    const int g = g0 + tid, n = g < groups ? s_count[g] : 0, tiles = (n + kTile - 1) / kTile;
    int sum = n, sum_t = tiles;  // running sums of tokens and tiles
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int p = __shfl_up_sync(0xffffffffu, sum, o), q = __shfl_up_sync(0xffffffffu, sum_t, o);
      if (lane >= o) {
        sum += p;
        sum_t += q;
      }
    }
    if (lane == 31) {
      s_warp[0][warp] = sum;
      s_warp[1][warp] = sum_t;
    }
    __syncthreads();
    int before = s_carry[0], before_t = s_carry[1];
    for (int w = 0; w < warp; ++w) {
      before += s_warp[0][w];
      before_t += s_warp[1][w];
    }
    before += sum - n;
    before_t += sum_t - tiles;
    if (g < groups) {
      s_place[g] = before;
      for (int i = 0; i < tiles; ++i)
        a.tiles[before_t + i] = Tile{g < a.adapters ? g : -1, before + i * kTile, min(kTile, n - i * kTile)};
    }
    __syncthreads();
    if (tid == kPlanThreads - 1) {
      s_carry[0] = before + n;
      s_carry[1] = before_t + tiles;
    }
    __syncthreads();
  }
  if (tid == 0) {
    *a.num_tiles = s_carry[1];
    *a.status = s_bad ? (int)FLJSD_ERR_INVALID_ARG : 0;
  }
  for (int64_t t = tid; t < a.tokens; t += kPlanThreads) {
    const int g = group(t);
    if (g >= 0) a.order[atomicAdd(&s_place[g], 1)] = (int)t;
  }
}

__global__ void __launch_bounds__(kThreads) k_lr_shrink(const Args a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ unsigned long long s_free[kStages];
  __shared__ uint32_t s_tmem;
  __shared__ int s_ok;
  __shared__ const __nv_bfloat16* s_row[kTile];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 127u) & ~127u;
  const int stage_bytes = kXStage + a.rank * 128;
  // (an instruction reads 128 rows of A; those past the rank are whatever lies there)
  float* parts = reinterpret_cast<float*>(smem_raw + (base - smem_u32(smem_raw)) + kStages * stage_bytes);
  const uint32_t rank_in_cluster = cluster_ctarank();
  // (none is written to before it has started)
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if (warp == 0) tmem_alloc<false>(smem_u32(&s_tmem), kTile);
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(&s_free[i]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s_ok = 1;
  }
  wait_for_previous();
  const int t = blockIdx.x / kSplit;
  const bool live = t < *a.num_tiles && a.tiles[t].adapter >= 0;
  const Tile tile = live ? a.tiles[t] : Tile{0, 0, 0};
  if (tid < tile.count) s_row[tid] = a.x + (int64_t)a.order[tile.first + tid] * a.ldx;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  let_next_launch();  // (with the tensor memory in hand)
  const uint32_t tmem = s_tmem;
  const int64_t chunks = (a.k + 63) / 64, per = (chunks + kSplit - 1) / kSplit;
  const int64_t c0 = min(rank_in_cluster * per, chunks), c1 = live ? min(c0 + per, chunks) : c0;
  const __nv_bfloat16* A = a.a + (int64_t)tile.adapter * a.rank * a.k;
  const int n16 = (tile.count + 15) / 16 * 16;
  auto ask = [&](int64_t c) {  // chunk c into its stage
    const uint32_t xs = base + (uint32_t)((c - c0) % kStages) * stage_bytes, as = xs + kXStage;
    for (int i = tid; i < tile.count * 8; i += kThreads)
      copy8(xs + place(i / 8, i % 8, 8), s_row[i / 8], c * 64 + (i % 8) * 8, a.k, a.vec_k, a.x);
    for (int i = tid; i < a.rank * 8; i += kThreads)
      copy8(as + place(i / 8, i % 8, 8), A + (int64_t)(i / 8) * a.k, c * 64 + (i % 8) * 8, a.k, a.vec_k, a.x);
  };
  bool ok = true;
  for (int i = 0; i < kStages - 1; ++i) {
    if (c0 + i < c1) ask(c0 + i);
    copies_commit();
  }
  for (int64_t c = c0; c < c1; ++c) {
    const int i = (int)(c - c0), stage = i % kStages;
    copies_wait<kStages - 2>();
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      const uint32_t xs = base + (uint32_t)stage * stage_bytes, as = xs + kXStage;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_bf16<false>(tmem, desc(as + kk * 256, 8), desc(xs + kk * 256, 8), idesc_of(n16), i + kk > 0);
      mma_commit<false>(smem_u32(&s_free[stage]));
    }
    __syncwarp();
    if (c + kStages - 1 < c1) {  // the stage before this one's is free once its products have run
      if (i > 0 && ok) ok = wait(smem_u32(&s_free[(i - 1) % kStages]), ((i - 1) / kStages) & 1, a.status);
      ask(c + kStages - 1);
    }
    copies_commit();
  }
  copies_wait<0>();
  const int used = (int)(c1 - c0);
  if (used > 0) ok = wait(smem_u32(&s_free[(used - 1) % kStages]), ((used - 1) / kStages) & 1, a.status) && ok;
  if (!ok) s_ok = 0;
  tc_fence_after();
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  // this CTA's part to the CTAs that add them: kOwn tokens to each
  if (live && warp * 32 < a.rank) {
    for (int j0 = 0; j0 < n16; j0 += 16) {
      float v[16];
      uint32_t r[16];
      asm volatile(
          "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
          "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
          : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
            "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
            "=r"(r[14]), "=r"(r[15])
          : "r"(tmem + ((uint32_t)(warp * 32) << 16) + j0));
      asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = used > 0 ? __uint_as_float(r[j]) : 0.f;
      const int rr = warp * 32 + lane;
      if (rr < a.rank) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int tok = j0 + j;
          if (tok < tile.count) {
            const uint32_t at = smem_u32(parts + ((int)rank_in_cluster * kOwn + tok % kOwn) * a.rank + rr);
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(map_to_cta(at, tok / kOwn)), "f"(v[j]) : "memory");
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 0) tmem_dealloc<false>(tmem, kTile);
  if (live) {
    const float scale = a.scales ? a.scales[tile.adapter] : 1.f;
    const int pieces = a.rk / 8, tok0 = (int)rank_in_cluster * kOwn;
    char* image = a.s + (int64_t)t * kTile * a.rk * 4;
    for (int i = tid; i < kOwn * a.rk; i += kThreads) {
      const int tok = i / a.rk, rr = i % a.rk;
      if (tok0 + tok >= tile.count) break;
      float s = 0.f;
      if (rr < a.rank) {
#pragma unroll
        for (int p = 0; p < kSplit; ++p) s += parts[(p * kOwn + tok) * a.rank + rr];
        s *= scale;
      }
      if (!s_ok) s = 0.f;
      const __nv_bfloat16 hi = __float2bfloat16_rn(s);
      // (an s that bf16 does not hold has nothing left)
      const float left = s - __bfloat162float(hi);
      const __nv_bfloat16 lo = __float2bfloat16_rn(fabsf(s) < INFINITY && fabsf(left) < INFINITY ? left : 0.f);
      const uint32_t at = place(tok0 + tok, rr / 8, pieces) + (rr % 8) * 2;
      *reinterpret_cast<__nv_bfloat16*>(image + at) = hi;
      *reinterpret_cast<__nv_bfloat16*>(image + (int64_t)kTile * a.rk * 2 + at) = lo;
    }
  }
}

template <typename T>
struct Pair;
template <>
struct Pair<float> {
  using V = float2;
  static constexpr int kTokens = 16;  // whose pairs a thread has in flight
};
template <>
struct Pair<__nv_bfloat16> {
  using V = uint32_t;
  static constexpr int kTokens = 32;
};
__device__ __forceinline__ float2 add_to(float2 y, float d0, float d1) { return make_float2(y.x + d0, y.y + d1); }
__device__ __forceinline__ uint32_t add_to(uint32_t y, float d0, float d1) {
  return pack_bf16(bf16_lo(y) + d0, bf16_hi(y) + d1);
}
__device__ __forceinline__ float2 join(float a, float b) { return make_float2(a, b); }
__device__ __forceinline__ uint32_t join(__nv_bfloat16 a, __nv_bfloat16 b) {
  return (uint32_t)__bfloat16_as_ushort(a) | ((uint32_t)__bfloat16_as_ushort(b) << 16);
}
__device__ __forceinline__ void split(float2 v, float& a, float& b) {
  a = v.x;
  b = v.y;
}
__device__ __forceinline__ void split(uint32_t v, __nv_bfloat16& a, __nv_bfloat16& b) {
  a = __ushort_as_bfloat16((unsigned short)(v & 0xffffu));
  b = __ushort_as_bfloat16((unsigned short)(v >> 16));
}

// 32 lanes x J columns of accumulators.
template <int J>
__device__ __forceinline__ void tmem_get(uint32_t taddr, float (&v)[J]) {
  static_assert(J == 16 || J == 32, "columns");
  if constexpr (J == 32) {
    tmem_ld32(taddr, v);
  } else {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) k_lr_expand(const Args a) {
  using V = typename Pair<T>::V;
  constexpr int J = Pair<T>::kTokens;
  extern __shared__ uint8_t smem_raw[];
  __shared__ unsigned long long s_done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_token[kTile];
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t base = (smem_u32(smem_raw) + 127u) & ~127u;
  const int pieces = a.rk / 8;
  const uint32_t s_at = base, s_half = (uint32_t)kTile * a.rk * 2;  // nearest, rest
  const uint32_t b_at = s_at + 2 * s_half, b_half = 128u * a.rk * 2;  // even columns, odd ones
  if (tid == 0) {
    mbar_init(smem_u32(&s_done), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  wait_for_previous();
  // (only now: what it waits for needs tensor memory too)
  if (warp == 0) tmem_alloc<false>(smem_u32(&s_tmem), 2 * kTile);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int t = blockIdx.x;
  if (t < *a.num_tiles) {
    const Tile tile = a.tiles[t];
    const bool adds = tile.adapter >= 0;
    if (tid < tile.count) s_token[tid] = a.order[tile.first + tid];
    if (adds) {
      const char* image = a.s + (int64_t)t * kTile * a.rk * 4;
      const int bytes16 = (int)(2 * s_half / 16);
      for (int i = tid; i < bytes16; i += kThreads) copy16(s_at + i * 16, image + i * 16, true);
    }
    __syncthreads();
    const __nv_bfloat16* B = a.b + (int64_t)(adds ? tile.adapter : 0) * a.n * a.rank;
    const int n16 = (tile.count + 15) / 16 * 16;
    const T* y = reinterpret_cast<const T*>(a.y);
    T* out = reinterpret_cast<T*>(a.out);
    int64_t block = (int64_t)blockIdx.y * kBlocks;
    bool ok = true;
    for (int it = 0; it < kBlocks && block * kCols < a.n; ++it, ++block) {
      const int64_t col0 = block * kCols;
      if (adds) {
        for (int i = tid; i < kCols * pieces; i += kThreads) {
          const int row = i / pieces, piece = i % pieces;
          const bool there = col0 + row < a.n && piece * 8 < a.rank;
          copy16(b_at + (row & 1) * b_half + place(row >> 1, piece, pieces),
                 there ? B + (col0 + row) * a.rank + piece * 8 : B, there);
        }
        copies_commit();
        copies_wait<0>();
        fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0) {
          tc_fence_after();
          for (int h = 0; h < 2; ++h)
            for (int part = 0; part < 2; ++part)
              for (int kk = 0; kk < a.rk / 16; ++kk)
                mma_bf16<false>(tmem + h * kTile, desc(b_at + h * b_half + kk * 256, pieces),
                                desc(s_at + part * s_half + kk * 256, pieces), idesc_of(n16), part + kk > 0);
          mma_commit<false>(smem_u32(&s_done));
        }
        __syncwarp();
      }
      const int64_t col = col0 + 2 * tid;
      const bool two = col + 1 < a.n, one = col < a.n;
      for (int j0 = 0; j0 < tile.count; j0 += J) {
        V have[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (j0 + j < tile.count) {
            const T* p = y + (int64_t)s_token[j0 + j] * a.ldy + col;
            if (a.pairs && two) {
              have[j] = *reinterpret_cast<const V*>(p);
            } else {
              T lo = T(0.f), hi = T(0.f);
              if (one) lo = p[0];
              if (two) hi = p[1];
              have[j] = join(lo, hi);
            }
          }
        }
        if (adds) {
          if (j0 == 0) {
            if (ok) ok = wait(smem_u32(&s_done), it & 1, a.status);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
          }
          float d0[J], d1[J];
          const uint32_t at = tmem + ((uint32_t)(warp * 32) << 16) + j0;
          tmem_get<J>(at, d0);
          tmem_get<J>(at + kTile, d1);
          if (ok) {
#pragma unroll
            for (int j = 0; j < J; ++j) have[j] = add_to(have[j], d0[j], d1[j]);
          }
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (j0 + j < tile.count) {
            T* p = out + (int64_t)s_token[j0 + j] * a.ldo + col;
            if (a.pairs && two) {
              *reinterpret_cast<V*>(p) = have[j];
            } else {
              T lo, hi;
              split(have[j], lo, hi);
              if (one) p[0] = lo;
              if (two) p[1] = hi;
            }
          }
        }
      }
      tc_fence_before();
      __syncthreads();
      tc_fence_after();
    }
  }
  __syncthreads();
  if (warp == 0) tmem_dealloc<false>(tmem, 2 * kTile);
}

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

struct Layout {
  int64_t max_tiles;
  size_t tiles, order, s, bytes;
};
Layout layout(int64_t tokens, int adapters, int rank) {
  Layout l;
  const int64_t groups = adapters + 1;  // each has at most one tile that is not full
  l.max_tiles = tokens / kTile + (groups < tokens ? groups : tokens);
  l.tiles = 256;  // status, number of tiles
  l.order = align_up(l.tiles + l.max_tiles * sizeof(Tile));
  l.s = align_up(l.order + tokens * sizeof(int));
  l.bytes = l.s + (size_t)l.max_tiles * kTile * ((rank + 15) / 16 * 16) * 4;
  return l;
}

template <typename T>
cudaError_t launch_expand(const Args& a, cudaStream_t st) {
  const int smem = 128 + (2 * kTile + kCols) * a.rk * 2;
  cudaError_t e =
      cudaFuncSetAttribute(k_lr_expand<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (a.n + kCols - 1) / kCols;
  return launch_dependent(k_lr_expand<T>, dim3(a.max_tiles, (unsigned)((blocks + kBlocks - 1) / kBlocks)),
                          kThreads, smem, st, a);
}

}  // namespace
}  // namespace fljsd

using namespace fljsd;

extern "C" size_t fljsd_low_rank_workspace_bytes(int64_t tokens, int32_t adapters, int32_t rank) {
  if (tokens <= 0 || adapters <= 0 || rank <= 0) return 0;
  return layout(tokens, adapters, rank).bytes;
}

extern "C" fljsd_status fljsd_low_rank_add(int64_t tokens, int64_t k, int64_t n, int32_t rank,
                                           int32_t adapters, const void* x, int64_t ldx,
                                           const void* a, const void* b, const int64_t* index,
                                           const float* scales, int32_t dtype, const void* y,
                                           int64_t ldy, void* out, int64_t ldo, void* workspace,
                                           size_t workspace_bytes, fljsd_stream_t stream) {
  if (tokens <= 0 || k <= 0 || n <= 0 || rank <= 0 || adapters <= 0) return FLJSD_ERR_INVALID_ARG;
  if (dtype != FLJSD_F32 && dtype != FLJSD_BF16) return FLJSD_ERR_INVALID_ARG;
  if (!x || !a || !b || !index || !y || !out || !workspace) return FLJSD_ERR_INVALID_ARG;
  if (ldx < k || ldy < n || ldo < n || rank % 8) return FLJSD_ERR_INVALID_ARG;
  const uintptr_t el = dtype == FLJSD_BF16 ? 1 : 3;
  if (((uintptr_t)x & 1u) || ((uintptr_t)a & 1u) || ((uintptr_t)b & 15u) || ((uintptr_t)index & 7u) ||
      ((uintptr_t)scales & 3u) || (((uintptr_t)y | (uintptr_t)out) & el) || ((uintptr_t)workspace & 15u))
    return FLJSD_ERR_INVALID_ARG;
  if (y == out && ldy != ldo) return FLJSD_ERR_INVALID_ARG;
  if (tokens > (1 << 20) || k > (1 << 20) || n > (1 << 26) || rank > kMaxRank || adapters > kMaxAdapters)
    return FLJSD_ERR_UNSUPPORTED;
  const Layout l = layout(tokens, adapters, rank);
  if (workspace_bytes < l.bytes) return FLJSD_ERR_WORKSPACE;
  char* ws = reinterpret_cast<char*>(workspace);
  Args g{};
  g.tokens = tokens; g.k = k; g.n = n; g.ldx = ldx; g.ldy = ldy; g.ldo = ldo;
  g.rank = rank;
  g.rk = (rank + 15) / 16 * 16;
  g.adapters = adapters;
  g.max_tiles = (int)l.max_tiles;
  g.x = reinterpret_cast<const __nv_bfloat16*>(x);
  g.a = reinterpret_cast<const __nv_bfloat16*>(a);
  g.b = reinterpret_cast<const __nv_bfloat16*>(b);
  g.index = index;
  g.scales = scales;
  g.y = y;
  g.out = out;
  const uintptr_t size = dtype == FLJSD_BF16 ? 2 : 4;
  g.vec_k = (((uintptr_t)x | (uintptr_t)a) & 15u) == 0 && k % 8 == 0 && ldx % 8 == 0;
  g.pairs = (((uintptr_t)y | (uintptr_t)out) & (2 * size - 1)) == 0 && ldy % 2 == 0 && ldo % 2 == 0;
  g.copy = y != out;
  g.status = reinterpret_cast<int*>(ws);
  g.num_tiles = g.status + 1;
  g.tiles = reinterpret_cast<Tile*>(ws + l.tiles);
  g.order = reinterpret_cast<int*>(ws + l.order);
  g.s = ws + l.s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int plan_smem = 2 * (adapters + 1) * (int)sizeof(int);
  trace_begin(FLJSD_KERNEL_SMALL, st);
  k_lr_plan<<<1, kPlanThreads, plan_smem, st>>>(g);
  trace_end(FLJSD_KERNEL_SMALL, st);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return FLJSD_ERR_CUDA;
  const int stage = kXStage + rank * 128;
  int smem = 128 + kStages * stage + kSplit * kOwn * rank * (int)sizeof(float);
  const int reach = 128 + (kStages - 1) * stage + kXStage + 128 * 128;  // the last stage's 128 rows
  if (smem < reach) smem = reach;
  e = cudaFuncSetAttribute(k_lr_shrink, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return FLJSD_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {kSplit, 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(l.max_tiles * kSplit));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  trace_begin(FLJSD_KERNEL_SMALL, st);
  e = cudaLaunchKernelEx(&cfg, k_lr_shrink, g);
  trace_end(FLJSD_KERNEL_SMALL, st);
  if (e != cudaSuccess) return FLJSD_ERR_CUDA;
  trace_begin(FLJSD_KERNEL_SMALL, st);
  e = dtype == FLJSD_BF16 ? launch_expand<__nv_bfloat16>(g, st) : launch_expand<float>(g, st);
  trace_end(FLJSD_KERNEL_SMALL, st);
  return e == cudaSuccess ? FLJSD_OK : FLJSD_ERR_CUDA;
}
