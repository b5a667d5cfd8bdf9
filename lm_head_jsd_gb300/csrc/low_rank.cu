// Low-rank adapters of many requests on the output of a projection that they share:
//   out_t = y_t + scale_a B_a (A_a x_t),  a = index[t]  (-1: out_t = y_t)
//
// Bound by reading and writing y (few tokens of many adapters: by reading their B). The
// tokens are first sorted by adapter and cut into tiles of up to 64 that share one
// (k_lr_plan, or by k_lr_shrink itself where there are few); both products of a tile then run on the tensor cores with the adapter's
// rows as the instruction's 128 rows and the tokens as its columns, so that a tile of one
// token costs 16 columns and not 128 rows:
//  - k_lr_shrink: s = scale A x of a tile. A cluster of eight CTAs splits k and adds its
//    parts in shared memory, in one order. s is written as a sum of bf16, the nearest and what
//    is left: two for y in bf16 (2^-16 of s at most is lost; one would be 2^-8 off, as much as
//    y's own rounding), three for y in fp32 (2^-24).
//  - k_lr_expand: y + B s for 256 columns at a time. Accumulator rows i of two products
//    hold columns 2 i and 2 i + 1, so that a thread adds to pairs and a warp to 64
//    neighbouring columns of a token. On an SM (one CTA, or two): warps that copy B's rows
//    and y's ahead, one that issues the products, and two or four groups of four warps, each with a
//    ring of rows of its own (in one ring for all a group could be a round ahead of another),
//    that take a block each in turn and add to y where it lies in shared memory, from which
//    it is copied out. (With y read and written by the adding threads, a pair at a time,
//    addresses and waits took 750 us of 4096 x 128256 bf16 without any product; a copy 306.)
// 4096 tokens of 8 adapters, rank 16, n = 128256 bf16: 370 us = 5.9 TB/s (k_lr_shrink 19, in
// front of it 3 for sorting); 64 tokens of 64 adapters 76 us = 4.0 TB/s, bound by the few
// hundred cycles that issuing a block's products and handing it on take.
#include "dependent.cuh"
#include "elect.cuh"
#include "gemm_tc_kernel.cuh"
#include "tensor_map.cuh"

#include <atomic>

namespace fljsd {
namespace {

using namespace tcgemm;

constexpr int kTile = 64;       // tokens of a tile
constexpr int kCols = 256;      // columns of y that a block of k_lr_expand takes
constexpr int kMaxRank = 128;
// Up to this rank two CTAs share an SM: the warp that issues the products is the bound where
// tiles are small (64 tokens of 64 adapters of rank 16 and 32: 111 and 132 us with one, 77 and
// 118 with two). Above it two rings of B's rows do not fit.
constexpr int kSmallRank = 32;
constexpr int kMaxAdapters = 4096;
constexpr int kSplit = 8;       // CTAs of k_lr_shrink to a tile
constexpr int kOwn = kTile / kSplit;
constexpr int kThreads = 128;
constexpr int kPlanThreads = 1024;
constexpr int kStages = 4;
constexpr int kXStage = kTile * 128;  // 64 tokens x 64 of k
constexpr int kMaxStages = 8;   // of B's rows
constexpr int kMaxSlots = 4;    // places for rows of y in a group's ring
// Threads of k_lr_expand with so many groups.
__host__ __device__ constexpr int expand_threads(int groups) { return groups * 160 + 64; }

struct Tile {
  int adapter, count;  // tokens order[number * kTile ..]
};

struct Args {
  int64_t tokens, k, n, ldx, ldy, ldo;
  int rank, rk, adapters, max_tiles;  // rk: rank up to a multiple of 16
  const __nv_bfloat16 *x, *a, *b;
  const int64_t* index;
  const float* scales;
  const void* y;
  void* out;
  bool vec_k, copy, same;  // same: y's and out's rows lie to 16 bytes alike
  int pitch, boxes, stages, s_bufs, slots, blocks;  // bytes of a row of B's boxes, boxes to it; blocks of a job
  int* status;
  int* num_tiles;
  Tile* tiles;
  int* order;
  int parts;  // of s: two or three bf16
  unsigned long long wait_ns;  // a wait's limit
  // A test's: no product A x; bytes that are waited for and do not come, of B and of y.
  bool no_first;
  uint32_t more_b, more_y;
  char* s;  // a tile's s as it lies in shared memory: parts of kTile rows
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

// Waits with a limit, after which the call's status word says so.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const Args& a) {
  unsigned long long t0 = 0;
  for (uint32_t it = 0;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 255u) == 255u) {  // (reading the timer takes longer than most waits)
      const unsigned long long t = globaltimer();
      if (!t0) t0 = t;
      if (t - t0 > a.wait_ns) {
        atomicExch(a.status, (int)FLJSD_ERR_TIMEOUT);
        return false;
      }
    }
  }
}

// The group of a token: its adapter, or the last one where rows without an adapter are to be
// copied; -1: left as it is. `bad`: an index that names none.
__device__ __forceinline__ int group_of(const Args& a, int64_t t, bool& bad) {
  const int64_t i = a.index[t];
  if (i >= 0 && i < a.adapters) return (int)i;
  bad |= i != -1;
  return a.copy ? a.adapters : -1;
}

// Few tokens are sorted where they are first used: every CTA of k_lr_shrink finds its own
// tile, and its cluster's first one writes it down.
constexpr int kFewTokens = 1024, kFewGroups = 1024, kFewTiles = 16;
struct FewShared {
  int count[kFewGroups];
  int token[kTile];
  int warp[kThreads / 32];
  int group, before, tiles;
};
__device__ __forceinline__ Tile find_tile(const Args& a, int t, FewShared& sh, bool writes) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tokens = (int)a.tokens;
  const int groups = a.adapters + 1;
  bool bad = false;
  for (int i = tid; i < groups; i += kThreads) sh.count[i] = 0;
  __syncthreads();
  for (int i = tid; i < tokens; i += kThreads) {
    const int g = group_of(a, i, bad);
    if (g >= 0) atomicAdd(&sh.count[g], 1);
  }
  bad = __syncthreads_or(bad) != 0;
  if (warp == 0) {  // whose tile this is, and how many there are
    int group = -1, before = 0, tiles = 0;
    for (int g0 = 0; g0 < groups; g0 += 32) {
      const int mine = g0 + lane < groups ? (sh.count[g0 + lane] + kTile - 1) / kTile : 0;
      int sum = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int p = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += p;
      }
      const uint32_t over = __ballot_sync(0xffffffffu, tiles + sum > t);
      if (group < 0 && over) {
        const int l = __ffs(over) - 1;
        group = g0 + l;
        before = tiles + __shfl_sync(0xffffffffu, sum - mine, l);
      }
      tiles += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) {
      sh.group = group;
      sh.before = before;
      sh.tiles = tiles;
    }
  }
  __syncthreads();
  const int group = sh.group, lo = (t - sh.before) * kTile;
  Tile tile{group < a.adapters ? group : -1, 0};
  if (group >= 0) {
    tile.count = min(kTile, sh.count[group] - lo);
    for (int t0 = 0, seen = 0; t0 < tokens && seen < lo + kTile; t0 += kThreads) {
      const bool in = t0 + tid < tokens && group_of(a, t0 + tid, bad) == group;
      const uint32_t them = __ballot_sync(0xffffffffu, in);
      if (lane == 0) sh.warp[warp] = __popc(them);
      __syncthreads();
      int at = seen - lo + __popc(them & ((1u << lane) - 1));
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) at += sh.warp[w];
        seen += sh.warp[w];
      }
      if (in && at >= 0 && at < kTile) sh.token[at] = t0 + tid;
      __syncthreads();
    }
    if (writes && tid < tile.count) a.order[(int64_t)t * kTile + tid] = sh.token[tid];
    if (writes && tid == 0) a.tiles[t] = tile;
  }
  if (blockIdx.x == 0 && tid == 0) {
    *a.num_tiles = sh.tiles;
    *a.status = bad ? (int)FLJSD_ERR_INVALID_ARG : 0;
  }
  return tile;
}

// Sorts the tokens by adapter (those without one last, where they are to be copied) and
// cuts each adapter's into tiles. Which of an adapter's tokens comes first changes
// nothing in their results.
__global__ void __launch_bounds__(kPlanThreads) k_lr_plan(const Args a) {
  extern __shared__ int s_count[];  // [adapters + 1], then the places
  __shared__ int s_warp[kPlanThreads / 32];
  __shared__ int s_carry;
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int groups = a.adapters + 1;
  int* s_place = s_count + groups;
  let_next_launch();
  for (int i = tid; i < groups; i += kPlanThreads) s_count[i] = 0;
  if (tid == 0) s_carry = s_bad = 0;
  __syncthreads();
  bool bad = false;
  for (int64_t t = tid; t < a.tokens; t += kPlanThreads) {
    const int g = group_of(a, t, bad);
    if (g >= 0) atomicAdd(&s_count[g], 1);
  }
  if (bad) s_bad = 1;
  __syncthreads();
  for (int g0 = 0; g0 < groups; g0 += kPlanThreads) {
    const int g = g0 + tid, n = g < groups ? s_count[g] : 0, tiles = (n + kTile - 1) / kTile;
    int sum = tiles;  // running
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int p = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += p;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    int before_t = s_carry;
    for (int w = 0; w < warp; ++w) before_t += s_warp[w];
    before_t += sum - tiles;
    if (g < groups) {
      s_place[g] = before_t * kTile;
      for (int i = 0; i < tiles; ++i)
        a.tiles[before_t + i] = Tile{g < a.adapters ? g : -1, min(kTile, n - i * kTile)};
    }
    __syncthreads();
    if (tid == kPlanThreads - 1) s_carry = before_t + tiles;
    __syncthreads();
  }
  if (tid == 0) {
    *a.num_tiles = s_carry;
    *a.status = s_bad ? (int)FLJSD_ERR_INVALID_ARG : 0;
  }
  for (int64_t t = tid; t < a.tokens; t += kPlanThreads) {
    const int g = group_of(a, t, bad);
    if (g >= 0) a.order[atomicAdd(&s_place[g], 1)] = (int)t;
  }
}

template <bool FEW>
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
  bool live;
  Tile tile;
  int token = 0;
  if constexpr (FEW) {
    __shared__ FewShared few;
    tile = find_tile(a, t, few, rank_in_cluster == 0);
    if (tid < tile.count) token = few.token[tid];
    live = tile.count > 0 && tile.adapter >= 0;
  } else {
    // (three loads at once: a place behind the last tile is there, whatever it holds)
    const int tiles = *a.num_tiles;
    tile = a.tiles[t];
    if (tid < kTile) token = a.order[(int64_t)t * kTile + tid];
    live = t < tiles && tile.adapter >= 0;
  }
  if (!live) tile = Tile{0, 0};
  if (tid < tile.count) s_row[tid] = a.x + (int64_t)token * a.ldx;
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
    if (tid == 0 && !a.no_first) {
      tc_fence_after();
      const uint32_t xs = base + (uint32_t)stage * stage_bytes, as = xs + kXStage;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_bf16<false>(tmem, desc(as + kk * 256, 8), desc(xs + kk * 256, 8), idesc_of(n16), i + kk > 0);
      mma_commit<false>(smem_u32(&s_free[stage]));
    }
    __syncwarp();
    if (c + kStages - 1 < c1) {  // the stage before this one's is free once its products have run
      if (i > 0 && ok) ok = wait(smem_u32(&s_free[(i - 1) % kStages]), ((i - 1) / kStages) & 1, a);
      ask(c + kStages - 1);
    }
    copies_commit();
  }
  copies_wait<0>();
  const int used = (int)(c1 - c0);
  if (used > 0) ok = wait(smem_u32(&s_free[(used - 1) % kStages]), ((used - 1) / kStages) & 1, a) && ok;
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
    char* image = a.s + (int64_t)t * kTile * a.rk * 2 * a.parts;
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
      const uint32_t at = place(tok0 + tok, rr / 8, pieces) + (rr % 8) * 2;
      float left = s;
      for (int p = 0; p < a.parts; ++p) {
        const __nv_bfloat16 h = __float2bfloat16_rn(left);
        *reinterpret_cast<__nv_bfloat16*>(image + (int64_t)p * kTile * a.rk * 2 + at) = h;
        // (an s that bf16 does not hold has nothing left)
        left -= __bfloat162float(h);
        if (!(fabsf(s) < INFINITY && fabsf(left) < INFINITY)) left = 0.f;
      }
    }
  }
}

template <typename T>
struct Pair;
template <>
struct Pair<float> {
  using V = float2;
  static constexpr int kTokens = 8;  // whose rows share a place in shared memory
  static constexpr int kParts = 3;   // of s
};
template <>
struct Pair<__nv_bfloat16> {
  using V = uint32_t;
  static constexpr int kTokens = 16;
  static constexpr int kParts = 2;
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
// Bytes of a row's place: a block's columns from the 16-byte boundary before the first.
template <typename T>
constexpr int row_bytes() {
  return kCols * (int)sizeof(T) + 16;
}

// 32 lanes x 8 or 16 columns of accumulators; tmem_landed before they are used.
__device__ __forceinline__ void tmem_get(uint32_t at, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(at));
}
__device__ __forceinline__ void tmem_get(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}
__device__ __forceinline__ void tmem_landed() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

template <int GROUPS>
struct ExpandShared {
  unsigned long long b_full[kMaxStages], b_empty[kMaxStages];  // a block's rows of B
  unsigned long long s_full[2], s_empty[2];                    // a job's s
  unsigned long long acc_full[GROUPS], acc_empty[GROUPS];
  unsigned long long y_full[GROUPS * kMaxSlots], y_empty[GROUPS * kMaxSlots];    // rows of some tokens
  uint32_t tmem;
  volatile int abort;
};
// Waits with a limit, after which the CTA's all end and the call's status word says so.
// (By whole warps. A barrier has one waiting warp or group, which waits for its every phase.)
template <int GROUPS>
__device__ __forceinline__ bool wait_all(ExpandShared<GROUPS>* sh, const void* bar, uint32_t parity, const Args& a) {
  const uint32_t b = smem_u32(bar);
  bool ok = mbar_try_wait(b, parity);
  unsigned long long t0 = 0;
  for (uint32_t it = 0; !ok; ++it) {
    ok = mbar_try_wait(b, parity);
    if (!ok && (it & 255u) == 255u) {  // (reading the timer takes longer than most waits)
      if (sh->abort) break;
      const unsigned long long t = globaltimer();
      if (!t0) t0 = t;
      if (t - t0 > a.wait_ns) {
        sh->abort = 1;
        atomicExch(a.status, (int)FLJSD_ERR_TIMEOUT);
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok) != 0;
}
// At the end, for copies and products still under way: with the same limit, all of a warp's
// together, and not cut short by a wait that has run out elsewhere.
__device__ __forceinline__ void wait_last(const void* bar, uint32_t parity, unsigned long long& t0, const Args& a) {
  const uint32_t b = smem_u32(bar);
  for (uint32_t it = 0; !mbar_try_wait(b, parity); ++it) {
    if ((it & 255u) != 255u) continue;
    const unsigned long long t = globaltimer();
    if (!t0) t0 = t;
    if (t - t0 > a.wait_ns) {
      atomicExch(a.status, (int)FLJSD_ERR_TIMEOUT);
      break;
    }
  }
  __syncwarp();
}

// A place in a ring and the parity of its round. (A division for each use of one took the
// warp that issues the products half a microsecond a block.)
struct Ring {
  uint32_t at = 0, round = 0;
  __device__ __forceinline__ void next(uint32_t n) {
    if (++at == n) {
      at = 0;
      round ^= 1;
    }
  }
};

// Rows of B that lie in boxes of `pitch` bytes (32, 64 or 128), swizzled so far.
__device__ __forceinline__ uint64_t desc_of(uint32_t addr, int pitch) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)1 << 16 | (uint64_t)((8 * pitch) >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)(pitch == 32 ? 6 : pitch == 64 ? 4 : 2) << 61;
}

// Jobs are a tile with `blocks` blocks of columns, all of one tile before the next one's:
// an adapter's B is still in L2 for its next tile, and the rows of y that are in use at a
// time lie in few pages (all tiles of a stretch of columns first: 4096 tokens 885 us).
// ALIGNED: all rows of y and out lie on 16 bytes, their strides and ends too. Otherwise the
// part of a row between 16-byte boundaries is copied, and up to seven values on either side
// are read and written one by one.
// GROUPS: four on an SM, in one CTA or in two.
template <typename T, bool ALIGNED, int GROUPS>
__global__ void __launch_bounds__(expand_threads(GROUPS), 4 / GROUPS)
    k_lr_expand(const __grid_constant__ CUtensorMap tm_even, const __grid_constant__ CUtensorMap tm_odd, const Args a) {
  using V = typename Pair<T>::V;
  constexpr int kRow = row_bytes<T>(), kSize = (int)sizeof(T), kChunk = Pair<T>::kTokens, kParts = Pair<T>::kParts;
  extern __shared__ uint8_t smem_raw[];
  __shared__ ExpandShared<GROUPS> sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t half = 128u * a.pitch * a.boxes, stage = 2 * half;  // even columns, odd ones
  const uint32_t s_half = (uint32_t)kTile * a.rk * 2, s_at = base + a.stages * stage;
  const uint32_t y_at = s_at + a.s_bufs * kParts * s_half;
  if (tid == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(smem_u32(&sh.b_full[i]), 1);
      mbar_init(smem_u32(&sh.b_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.s_full[i]), 1);
      mbar_init(smem_u32(&sh.s_empty[i]), 1);
    }
    for (int i = 0; i < GROUPS; ++i) {
      mbar_init(smem_u32(&sh.acc_full[i]), 1);
      mbar_init(smem_u32(&sh.acc_empty[i]), 4);
    }
    for (int i = 0; i < GROUPS * a.slots; ++i) {
      mbar_init(smem_u32(&sh.y_full[i]), 1);
      mbar_init(smem_u32(&sh.y_empty[i]), 1);
    }
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_tensormap(&tm_even);
    prefetch_tensormap(&tm_odd);
  }
  wait_for_previous();
  // (only now: what it waits for needs tensor memory too)
  if (warp == 0) tmem_alloc<false>(smem_u32(&sh.tmem), GROUPS * 2 * kTile);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t tiles = (uint32_t)*a.num_tiles;
  const uint32_t num_blocks = (uint32_t)((a.n + kCols - 1) / kCols);
  const uint32_t stretches = (num_blocks + a.blocks - 1) / a.blocks, jobs = tiles * stretches;
  if (warp == GROUPS * 4) {
    // ---------------- copies ----------------
    Ring b_ring, s_ring;
    uint32_t filled = 0, s_filled = 0;
    bool ok = true;
    Tile next = blockIdx.x < jobs ? a.tiles[blockIdx.x / stretches] : Tile{-1, 0};
    for (uint32_t k = blockIdx.x; ok && k < jobs; k += gridDim.x) {
      const Tile tile = next;
      const uint32_t t = k / stretches, b0 = k % stretches * a.blocks;
      if (k + gridDim.x < jobs) next = a.tiles[(k + gridDim.x) / stretches];
      if (tile.adapter < 0) continue;
      const uint32_t si = s_ring.at;
      ok = wait_all(&sh, &sh.s_empty[si], s_ring.round ^ 1, a);
      if (!ok) break;
      if (elect_one()) {
        const uint32_t bar = smem_u32(&sh.s_full[si]), to = s_at + si * kParts * s_half;
        const char* image = a.s + (int64_t)t * kTile * a.rk * 2 * a.parts;
        const uint32_t bytes = (uint32_t)((tile.count + 15) / 16 * 16) * a.rk * 2;
        mbar_arrive_expect_tx(bar, kParts * bytes);
        for (int h = 0; h < kParts; ++h)
          asm volatile(
              "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                  to + h * s_half),
              "l"(image + (int64_t)h * s_half), "r"(bytes), "r"(bar)
              : "memory");
      }
      __syncwarp();
      s_ring.next(a.s_bufs);
      ++s_filled;
      const int64_t row0 = (int64_t)tile.adapter * a.n;
      for (uint32_t b = b0; b < b0 + a.blocks && b < num_blocks; ++b) {
        const uint32_t st = b_ring.at;
        ok = wait_all(&sh, &sh.b_empty[st], b_ring.round ^ 1, a);
        if (!ok) break;
        if (elect_one()) {
          const uint32_t bar = smem_u32(&sh.b_full[st]);
          mbar_arrive_expect_tx(bar, stage + a.more_b);
          const int64_t row = row0 + (int64_t)b * kCols;
          for (int h = 0; h < 2; ++h)
            for (int x = 0; x < a.boxes; ++x)
              tma_load_2d(base + st * stage + h * half + x * 128 * a.pitch, (row + h) & 1 ? &tm_odd : &tm_even, bar,
                          x * 64, (int)((row + h) >> 1));
        }
        __syncwarp();
        b_ring.next(a.stages);
        ++filled;
      }
    }
    // no copy is under way at the end
    unsigned long long t0 = 0;
    for (uint32_t i = 0; i < (uint32_t)a.stages && i < filled; ++i) {
      const uint32_t f = filled - 1 - i;
      wait_last(&sh.b_full[f % a.stages], (f / a.stages) & 1, t0, a);
    }
    for (uint32_t i = 0; i < (uint32_t)a.s_bufs && i < s_filled; ++i) {
      const uint32_t f = s_filled - 1 - i;
      wait_last(&sh.s_full[f % a.s_bufs], (f / a.s_bufs) & 1, t0, a);
    }
  } else if (warp == GROUPS * 4 + 1) {
    // ---------------- products ----------------
    Ring b_ring, s_ring;
    uint32_t used = 0;  // a bit for each accumulator
    // the first descriptors: those of other places, rows and slices are so many 16 bytes on
    const uint64_t b_first = desc_of(base, a.pitch), s_first = desc(s_at, a.rk / 8);
    const uint32_t s_next = s_half >> 4, b_odd = half >> 4;
    bool ok = true;
    Tile next = blockIdx.x < jobs ? a.tiles[blockIdx.x / stretches] : Tile{-1, 0};
    uint32_t last_group = GROUPS;
    for (uint32_t k = blockIdx.x, seq = 0; ok && k < jobs; k += gridDim.x, seq += a.blocks) {
      const Tile tile = next;
      const uint32_t b0 = k % stretches * a.blocks;
      if (k + gridDim.x < jobs) next = a.tiles[(k + gridDim.x) / stretches];
      if (tile.adapter < 0) continue;
      const uint32_t si = s_ring.at;
      ok = wait_all(&sh, &sh.s_full[si], s_ring.round, a);
      const uint64_t s0d = s_first + si * (kParts * s_next);
      const uint32_t id = idesc_of((tile.count + 15) / 16 * 16);
      for (uint32_t c = 0; ok && c < (uint32_t)a.blocks && b0 + c < num_blocks; ++c) {
        const uint32_t g = (seq + c) % GROUPS, st = b_ring.at;
        ok = wait_all(&sh, &sh.acc_empty[g], ((used >> g) & 1) ^ 1, a) &&
             wait_all(&sh, &sh.b_full[st], b_ring.round, a);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t b0d = b_first + st * (stage >> 4);
          const uint32_t d = tmem + g * 2 * kTile;
#pragma unroll 1
          for (int kk = 0; kk < a.rk / 16; ++kk) {
            const uint64_t bd = b0d + (uint32_t)((kk >> 2) * (128 * 128 >> 4) + (kk & 3) * 2), sd = s0d + kk * 16;
#pragma unroll
            for (int p = 0; p < kParts; ++p) {
              mma_bf16<false>(d, bd, sd + p * s_next, id, kk + p > 0);
              mma_bf16<false>(d + kTile, bd + b_odd, sd + p * s_next, id, kk + p > 0);
            }
          }
          mma_commit<false>(smem_u32(&sh.b_empty[st]));
          mma_commit<false>(smem_u32(&sh.acc_full[g]));
          if (c + 1 == (uint32_t)a.blocks || b0 + c + 1 == num_blocks) mma_commit<false>(smem_u32(&sh.s_empty[si]));
        }
        __syncwarp();
        used ^= 1u << g;
        last_group = g;
        b_ring.next(a.stages);
      }
      s_ring.next(a.s_bufs);
    }
    unsigned long long t0 = 0;
    if (last_group < GROUPS)  // no product runs at the end
      wait_last(&sh.acc_full[last_group], ((used >> last_group) & 1) ^ 1, t0, a);
  } else if (warp >= GROUPS * 4 + 2) {
    // ---------------- y's rows for a group, a lane to each ----------------
    const uint32_t g = warp - (GROUPS * 4 + 2);
    const char* y = reinterpret_cast<const char*>(a.y);
    Ring ring;
    uint32_t filled = 0;
    bool ok = true;
    // The ends of rows that a copy leaves out: read now, put in place when the next place is
    // asked for, and their place full only then. (Of a block of few columns all of it.)
    constexpr int kEnds = ALIGNED ? 1 : 32 / kSize;
    T kept_value[kEnds];
    int kept = 0;
    uint32_t kept_at = 0, open_bar = 0, open_bytes = 0;
    auto settle = [&]() {
      if (!open_bar) return;
#pragma unroll
      for (int e = 0; e < kEnds; ++e)
        if (e < kept) *reinterpret_cast<T*>(__cvta_shared_to_generic(kept_at + e * kSize)) = kept_value[e];
      kept = 0;
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(open_bar, open_bytes);
      open_bar = 0;
    };
    auto tile_of = [&](uint32_t k) { return k < jobs ? a.tiles[k / stretches] : Tile{-1, 0}; };
    auto token_of = [&](uint32_t k, int j) { return k < jobs ? a.order[(int64_t)(k / stretches) * kTile + j] : 0; };
    Tile next = tile_of(blockIdx.x);
    int next0 = token_of(blockIdx.x, lane), next1 = token_of(blockIdx.x, lane + 32);
    for (uint32_t k = blockIdx.x, seq = 0; ok && k < jobs; k += gridDim.x, seq += a.blocks) {
      const Tile tile = next;
      const int t0 = next0, t1 = next1;
      next = tile_of(k + gridDim.x);
      next0 = token_of(k + gridDim.x, lane);
      next1 = token_of(k + gridDim.x, lane + 32);
      const uint32_t b0 = k % stretches * a.blocks;
      const uint32_t left = min((uint32_t)a.blocks, num_blocks - b0);
      for (uint32_t c = (g - seq) % GROUPS; ok && c < left; c += GROUPS) {
        const int64_t col0 = (int64_t)(b0 + c) * kCols;
        const int len = (int)min((int64_t)kCols, a.n - col0) * kSize;
        for (int j0 = 0; j0 < tile.count; j0 += kChunk) {
          const uint32_t slot = g * a.slots + ring.at;
          if (a.slots == 1) settle();
          ok = wait_all(&sh, &sh.y_empty[slot], ring.round ^ 1, a);
          if (!ok) break;
          const int r = lane % kChunk, j = j0 + r;
          const int token = __shfl_sync(0xffffffffu, j0 < 32 ? t0 : t1, j & 31);
          const uintptr_t at = (uintptr_t)(y + ((int64_t)token * a.ldy + col0) * kSize);
          const uintptr_t lo = (at + 15) & ~(uintptr_t)15, hi = (at + len) & ~(uintptr_t)15;
          const uint32_t bytes = lane < kChunk && j < tile.count && hi > lo ? (uint32_t)(hi - lo) : 0u;
          const uint32_t place = y_at + (slot * kChunk + r) * kRow;
          if (bytes)
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                    place + (uint32_t)(lo - (at & ~(uintptr_t)15))),
                "l"(lo), "r"(bytes), "r"(smem_u32(&sh.y_full[slot]))
                : "memory");
          const uint32_t all = __reduce_add_sync(0xffffffffu, bytes);
          settle();  // the one before
          if (!ALIGNED && lane < 2 * kChunk && j < tile.count) {
            // this lane's end of the row: what lies before the first boundary, or behind the last one
            const uintptr_t end = at + len;
            const uintptr_t from = lane < kChunk ? at : (hi > lo ? hi : end), to = lane < kChunk ? (hi > lo ? lo : end) : end;
            const T* p = reinterpret_cast<const T*>(from);
            kept = (int)((to - from) / kSize);
            kept_at = place + (uint32_t)(from - (at & ~(uintptr_t)15));
#pragma unroll
            for (int e = 0; e < kEnds; ++e)
              if (e < kept) kept_value[e] = p[e];
          }
          open_bar = smem_u32(&sh.y_full[slot]);
          open_bytes = all + a.more_y;
          if (ALIGNED) settle();
          ring.next(a.slots);
          ++filled;
        }
      }
    }
    settle();
    unsigned long long since = 0;
    for (uint32_t i = 0; i < (uint32_t)a.slots && i < filled; ++i) {  // no copy is under way at the end
      const uint32_t f = filled - 1 - i;
      wait_last(&sh.y_full[g * a.slots + f % a.slots], (f / a.slots) & 1, since, a);
    }
  } else {
    // ---------------- sums ----------------
    const int g = warp >> 2, quarter = warp & 3;
    const char* y = reinterpret_cast<const char*>(a.y);
    char* out = reinterpret_cast<char*>(a.out);
    const uint32_t acc = tmem + ((uint32_t)(quarter * 32) << 16) + g * 2 * kTile;
    const int mine = 2 * (quarter * 32 + lane) * kSize;  // this thread's pair in a block's row
    Ring ring;
    uint32_t used = 0, taken = 0;
    bool ok = true;  // (where a wait ran out, the group still meets, and leaves out as it is)
    auto tile_of = [&](uint32_t k) { return k < jobs ? a.tiles[k / stretches] : Tile{-1, 0}; };
    auto token_of = [&](uint32_t k, int j) { return k < jobs ? a.order[(int64_t)(k / stretches) * kTile + j] : 0; };
    Tile next = tile_of(blockIdx.x);
    int next0 = token_of(blockIdx.x, lane), next1 = token_of(blockIdx.x, lane + 32);
    for (uint32_t k = blockIdx.x, seq = 0; k < jobs; k += gridDim.x, seq += a.blocks) {
      const Tile tile = next;
      const int t0 = next0, t1 = next1;
      next = tile_of(k + gridDim.x);
      next0 = token_of(k + gridDim.x, lane);
      next1 = token_of(k + gridDim.x, lane + 32);
      const bool adds = tile.adapter >= 0;
      const uint32_t b0 = k % stretches * a.blocks;
      const uint32_t left = min((uint32_t)a.blocks, num_blocks - b0);
      const uint32_t chunks = (uint32_t)(tile.count + kChunk - 1) / kChunk;
      // where a row starts in its place (a block is a multiple of 16 bytes)
      const int lead0 = ALIGNED ? 0 : (int)((uintptr_t)(y + (int64_t)t0 * a.ldy * kSize) & 15u);
      const int lead1 = ALIGNED ? 0 : (int)((uintptr_t)(y + (int64_t)t1 * a.ldy * kSize) & 15u);
      for (uint32_t c = (g - seq) % GROUPS; c < left; c += GROUPS) {
        const int64_t col0 = (int64_t)(b0 + c) * kCols;
        const int len = (int)min((int64_t)kCols, a.n - col0) * kSize;
        for (uint32_t ch = 0; ch < chunks; ++ch) {
          const uint32_t slot = g * a.slots + ring.at;
          const uint32_t rows_at = y_at + slot * kChunk * kRow;
          const int j0 = ch * kChunk, count = min(kChunk, tile.count - j0);
          const int held = j0 < 32 ? t0 : t1;  // (by lane j & 31)
          const int held_lead = j0 < 32 ? lead0 : lead1;
          if (adds && ch == 0) {
            ok = ok && wait_all(&sh, &sh.acc_full[g], used & 1, a);
            tc_fence_after();
          }
          uint32_t d0[kChunk], d1[kChunk];
          if (adds) {
            tmem_get(acc + j0, d0);
            tmem_get(acc + kTile + j0, d1);
            tmem_landed();
            if (ch == chunks - 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_u32(&sh.acc_empty[g]));
              ++used;
            }
          }
          ok = ok && wait_all(&sh, &sh.y_full[slot], ring.round, a);
          if (ok && (adds || !ALIGNED)) {
#pragma unroll
            for (int j = 0; j < kChunk; ++j) {
              const int lead = ALIGNED ? 0 : __shfl_sync(0xffffffffu, held_lead, (j0 + j) & 31);
              const int token = ALIGNED || a.same ? 0 : __shfl_sync(0xffffffffu, held, (j0 + j) & 31);
              if (j < count) {
                T* p = reinterpret_cast<T*>(__cvta_shared_to_generic(rows_at + j * kRow + lead + mine));
                V v = ALIGNED ? *reinterpret_cast<const V*>(p) : join(p[0], p[1]);
                if (adds) v = add_to(v, __uint_as_float(d0[j]), __uint_as_float(d1[j]));
                if (ALIGNED) {
                  *reinterpret_cast<V*>(p) = v;
                } else {
                  T lo, hi;
                  split(v, lo, hi);
                  if (a.same) {
                    p[0] = lo;
                    p[1] = hi;
                  } else {  // one by one: out's rows lie otherwise
                    T* o = reinterpret_cast<T*>(out + ((int64_t)token * a.ldo + col0) * kSize + mine);
                    if (mine < len) o[0] = lo;
                    if (mine + kSize < len) o[1] = hi;
                  }
                }
              }
            }
            fence_proxy_async_smem();
          }
          asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory");
          if (quarter == (int)(taken & 3)) {  // out, a lane to each row
            if (a.same && ok) {
              const int r = lane % kChunk;
              const int token = __shfl_sync(0xffffffffu, held, (j0 + r) & 31);
              const uintptr_t at = (uintptr_t)(out + ((int64_t)token * a.ldo + col0) * kSize);
              const uintptr_t lo = (at + 15) & ~(uintptr_t)15, hi = (at + len) & ~(uintptr_t)15;
              const uint32_t place = rows_at + r * kRow - (uint32_t)(at & ~(uintptr_t)15);  // of address 0
              if (lane < count && hi > lo)
                asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(lo),
                             "r"(place + (uint32_t)lo), "r"((uint32_t)(hi - lo))
                             : "memory");
              if (!ALIGNED && r < count && lane < 2 * kChunk) {  // this lane's end of the row
                const uintptr_t end = at + len;
                uintptr_t from = lane < kChunk ? at : hi > lo ? hi : end;
                const uintptr_t to = lane < kChunk && hi > lo ? lo : end;
#pragma unroll 4
                for (; from < to; from += kSize)
                  *reinterpret_cast<T*>(from) =
                      *reinterpret_cast<const T*>(__cvta_shared_to_generic(place + (uint32_t)from));
              }
              bulk_commit();
              asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
              __syncwarp();
            }
            // (after a wait that ran out the place may still be filled: it is not given back)
            if (lane == 0 && ok) mbar_arrive(smem_u32(&sh.y_empty[slot]));
            __syncwarp();
          }
          ring.next(a.slots);
          ++taken;
        }
      }
    }
    bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc<false>(tmem, GROUPS * 2 * kTile);
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
  l.s = align_up(l.order + l.max_tiles * kTile * sizeof(int));
  l.bytes = l.s + (size_t)l.max_tiles * kTile * ((rank + 15) / 16 * 16) * 6;
  return l;
}

// A kernel's dynamic shared memory, allowed once on each device.
template <auto KERNEL>
cudaError_t allow() {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaGetDevice(&dev);
  const bool known = dev >= 0 && dev < 64;
  if (known && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  cudaFuncAttributes at;
  cudaError_t e = cudaFuncGetAttributes(&at, KERNEL);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             SMEM_MAX - (int)at.sharedSizeBytes);
  if (e == cudaSuccess && known) done[dev].store(true, std::memory_order_relaxed);
  return e;
}

template <typename T, bool ALIGNED, int GROUPS>
cudaError_t launch_expand(const CUtensorMap& even, const CUtensorMap& odd, Args a, cudaStream_t st) {
  constexpr int kCtas = 4 / GROUPS, kSlot = Pair<T>::kTokens * row_bytes<T>();
  const int s = Pair<T>::kParts * kTile * a.rk * 2, stage = 2 * 128 * a.pitch * a.boxes;
  a.s_bufs = a.rank > 64 ? 1 : 2;
  // a third of shared memory for B's rows, the rest for y's
  const int room = (SMEM_MAX - (kCtas - 1) * 1024) / kCtas - 1024 - (int)sizeof(ExpandShared<GROUPS>) - a.s_bufs * s;
  a.stages = room / 3 / stage;
  a.stages = a.stages < 2 ? 2 : a.stages > kMaxStages ? kMaxStages : a.stages;
  a.slots = (room - a.stages * stage) / kSlot / GROUPS;
  if (a.slots < 1) return cudaErrorInvalidConfiguration;
  if (a.slots > kMaxSlots) a.slots = kMaxSlots;
  const int smem = 1024 + a.stages * stage + a.s_bufs * s + GROUPS * a.slots * kSlot;
  const cudaError_t e = allow<k_lr_expand<T, ALIGNED, GROUPS>>();
  if (e != cudaSuccess) return e;
  const int64_t blocks = (a.n + kCols - 1) / kCols, most = a.max_tiles * blocks, ctas = num_sms() * kCtas;
  // (jobs long enough to load s once for many blocks, and eight of them to each CTA)
  a.blocks = 1;
  while (a.blocks < 32 && most >= ctas * 8 * 2 * a.blocks) a.blocks *= 2;
  return launch_dependent(k_lr_expand<T, ALIGNED, GROUPS>, dim3((unsigned)(most < ctas ? most : ctas)),
                          expand_threads(GROUPS), smem, st, even, odd, a);
}
template <typename T>
cudaError_t launch_expand(const CUtensorMap& even, const CUtensorMap& odd, const Args& a, bool aligned, cudaStream_t st) {
  if (a.rank <= kSmallRank)
    return aligned ? launch_expand<T, true, 2>(even, odd, a, st) : launch_expand<T, false, 2>(even, odd, a, st);
  return aligned ? launch_expand<T, true, 4>(even, odd, a, st) : launch_expand<T, false, 4>(even, odd, a, st);
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
  if (tokens > (1 << 20) || k > (1 << 20) || n > (1 << 26) || rank > kMaxRank || adapters > kMaxAdapters ||
      adapters * n >= (int64_t)1 << 31)
    return FLJSD_ERR_UNSUPPORTED;
  const Layout l = layout(tokens, adapters, rank);
  if (workspace_bytes < l.bytes) return FLJSD_ERR_WORKSPACE;
  char* ws = reinterpret_cast<char*>(workspace);
  Args g{};
  g.tokens = tokens; g.k = k; g.n = n; g.ldx = ldx; g.ldy = ldy; g.ldo = ldo;
  g.rank = rank;
  g.parts = dtype == FLJSD_BF16 ? Pair<__nv_bfloat16>::kParts : Pair<float>::kParts;
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
  const bool aligned = (((uintptr_t)y | (uintptr_t)out) & 15u) == 0 && ldy * size % 16 == 0 &&
                       ldo * size % 16 == 0 && n * size % 16 == 0;
  g.same = (((uintptr_t)y ^ (uintptr_t)out) & 15u) == 0 && (ldy - ldo) * (int64_t)size % 16 == 0;
  g.copy = y != out;
  g.status = reinterpret_cast<int*>(ws);
  g.num_tiles = g.status + 1;
  g.tiles = reinterpret_cast<Tile*>(ws + l.tiles);
  g.order = reinterpret_cast<int*>(ws + l.order);
  g.s = ws + l.s;
  const int stall = stalled();
  g.no_first = stall & FLJSD_STALL_LOW_RANK_FIRST;
  g.more_b = stall & FLJSD_STALL_LOW_RANK_SECOND ? 16 : 0;
  g.more_y = stall & FLJSD_STALL_LOW_RANK_Y ? 16 : 0;
  g.wait_ns = g.no_first || g.more_b || g.more_y ? kStallNs : kTimeoutNs;
  // B's rows, a column of y each, come as boxes of those of even numbers (among all adapters')
  // and of odd ones, as wide as the rank up to 64
  g.pitch = rank <= 16 ? 32 : rank <= 32 ? 64 : 128;
  g.boxes = rank <= 64 ? 1 : 2;
  CUtensorMap even, odd;
  const int64_t rows = adapters * n;
  const bool made =
      make_tensor_map(&even, MapType::kBf16, g.b, rank, (rows + 1) / 2, 2 * rank, g.pitch / 2, 128) &&
      make_tensor_map(&odd, MapType::kBf16, rows > 1 ? g.b + rank : g.b, rank, rows > 1 ? rows / 2 : 1, 2 * rank,
                      g.pitch / 2, 128);
  if (!made) return FLJSD_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // (one launch fewer, but every tile's CTAs look for it: one token of one adapter 34 us with
  // k_lr_plan and 28 without, 333 of 5 40.7 and 40.3, 64 of 64 78 and 84, 1000 of 1000 157 and 348)
  const bool few = l.max_tiles <= kFewTiles && tokens <= kFewTokens && adapters < kFewGroups;
  cudaError_t e = few ? allow<k_lr_shrink<true>>() : allow<k_lr_shrink<false>>();
  if (e != cudaSuccess) return FLJSD_ERR_CUDA;
  if (!few) {
    trace_begin(FLJSD_KERNEL_SMALL, st);
    k_lr_plan<<<1, kPlanThreads, 2 * (adapters + 1) * (int)sizeof(int), st>>>(g);
    trace_end(FLJSD_KERNEL_SMALL, st);
    if (cudaGetLastError() != cudaSuccess) return FLJSD_ERR_CUDA;
  }
  const int stage = kXStage + rank * 128;
  int smem = 128 + kStages * stage + kSplit * kOwn * rank * (int)sizeof(float);
  const int reach = 128 + (kStages - 1) * stage + kXStage + 128 * 128;  // the last stage's 128 rows
  if (smem < reach) smem = reach;
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
  cfg.numAttrs = few ? 1 : 2;  // (behind k_lr_plan)
  trace_begin(FLJSD_KERNEL_SMALL, st);
  e = few ? cudaLaunchKernelEx(&cfg, k_lr_shrink<true>, g) : cudaLaunchKernelEx(&cfg, k_lr_shrink<false>, g);
  trace_end(FLJSD_KERNEL_SMALL, st);
  if (e != cudaSuccess) return FLJSD_ERR_CUDA;
  trace_begin(FLJSD_KERNEL_SMALL, st);
  e = dtype == FLJSD_BF16 ? launch_expand<__nv_bfloat16>(even, odd, g, aligned, st)
                          : launch_expand<float>(even, odd, g, aligned, st);
  trace_end(FLJSD_KERNEL_SMALL, st);
  return e == cudaSuccess ? FLJSD_OK : FLJSD_ERR_CUDA;
}
