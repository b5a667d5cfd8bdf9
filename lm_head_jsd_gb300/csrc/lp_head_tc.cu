// Token log probabilities fused with the lm_head product (sm_103a): z = X . W^T
// on the tensor cores, reduced in the epilogue; the logits never reach memory.
//
// The product is that of gemm_tc_kernel.cuh (TMA ring, tcgen05.mma, two
// accumulators in tensor memory, CTA pairs on 256 x 256 tiles); what differs is
// the epilogue: eight warps, each thread one row of 128 columns (a part), which
// reads its accumulator twice:
//   1. the part's maximum, the label's logit, the candidates for the k largest;
//   2. d = sum 2^t and s = sum 2^t t relative to that maximum, and for a
//      backward pass 2^t itself in fp16.
// Two readings of tensor memory cost less than rescaling running sums and give
// every stored 2^t the same reference. 2^t is at most 1 and kept in fp16: within
// 2^-11 of its value down to 2^-14 of the part's maximum and within 2^-25 of that
// maximum below, a quarter of what the gradient's own rounding to bf16 costs
// (bf16 here made the gradients' error 1.5 times that of one rounding, fp16 1.4).
// Keeping the logits instead would need fp32 for the same error.
//
// The k largest: what reaches the row's threshold is appended to the row's
// candidates. The threshold: the parts are dealt into k groups (part index mod k),
// gmax[row][g] is the largest logit seen in group g, and at least k logits of the
// row reach the least of the k group maxima. A chunk of 32 columns whose maximum is
// below every lane's threshold costs one vote. Where more than k of a part's logits
// reach it (equal logits, or a threshold that came late), its k largest are found
// with a sorted list in registers (list_part). The order in which parts arrive
// changes how much is skipped, never the result: candidates equal to the threshold
// are kept, and k_lp_join orders them by value and column.
// The first columns, whose tiles run before there is a threshold, are not listed:
// their logits are written out (about one tile for each SM, through shared memory, whose
// copies write whole rows) and k_lp_join reads them against the final threshold. With 333
// rows of H = 2048, V = 40960 and 20 alternatives the listing takes 7 of 64 us; a sorted
// list of every part would take longer than the products it comes from.
//
// Tiles are as narrow as the rounds over the SMs allow (lp_head_tile_cols); a plan with a
// backward pass keeps 256 columns.
//
// Measured, with the join: 4096 rows of H = 4096, V = 128256 and 8 alternatives 2.07 ms
// = 2.08 PFLOP/s, 1.05 of the measured burst rate of a library product, 1.2 of the
// sustained one. Bound by the tensor cores down to H of about 1024; at H = 512 by the
// epilogue (4096 rows, V = 40960: 97 us, 214 with 8 alternatives, for 87 us of products).
#include "dependent.cuh"
#include "elect.cuh"
#include "gemm_tc_kernel.cuh"
#include "lp.cuh"
#include "tensor_map.cuh"

#include <cuda_fp16.h>

namespace fljsd {
namespace {

using namespace tcgemm;

constexpr int kThreads = 320;  // producer, MMA, eight epilogue warps
constexpr int kEpiWarps = 8;
constexpr int kKeepBufs = 2;   // staging buffers of an epilogue warp

struct HeadParams {
  int64_t m, n;
  int num_n_blocks, num_k_blocks, m_units, num_units, group_m, nst;
  int bn;  // columns of a tile, two parts
  float c;
  const int64_t* labels;
  float4* part;
  int64_t parts;
  float* zy;
  int top;
  unsigned* gmax;
  int* count;
  int2* cand;
  int dump_blocks;
  unsigned long long timeout_ns;
  int* status;
};

// Staging buffers of an epilogue warp: of 2^t two, one of which the first columns'
// logits borrow.
__host__ __device__ constexpr int stage_bufs(bool top, bool keep) {
  return keep ? kKeepBufs : top ? 1 : 0;
}
__host__ __device__ constexpr int head_smem(int nst, bool pair, bool top, bool keep) {
  return nst * stage_bytes(pair) + kEpiWarps * stage_bufs(top, keep) * OUT_BUF_BYTES + 1024 +
         CTRL_BYTES;
}
__host__ __device__ constexpr int head_stages(bool pair, bool keep) {
  return pair ? (keep ? 5 : 6) : (keep ? 3 : 4);
}
static_assert(head_smem(head_stages(true, true), true, true, true) <= SMEM_MAX &&
                  head_smem(head_stages(true, false), true, true, false) <= SMEM_MAX &&
                  head_smem(head_stages(false, true), false, true, true) <= SMEM_MAX &&
                  head_smem(head_stages(false, false), false, true, false) <= SMEM_MAX,
              "shared memory");

// A thread's list of its part's largest logits, in descending order; ties keep
// the earlier column in front.
template <int KT>
struct TopList {
  float v[KT];
  int id[KT];
  __device__ __forceinline__ void clear(float below) {
#pragma unroll
    for (int j = 0; j < KT; ++j) {
      v[j] = below;
      id[j] = -1;
    }
  }
  __device__ __forceinline__ void insert(float x, int col) {
#pragma unroll
    for (int j = KT - 1; j > 0; --j) {
      const bool above = x > v[j - 1], here = x > v[j];
      v[j] = above ? v[j - 1] : (here ? x : v[j]);
      id[j] = above ? id[j - 1] : (here ? col : id[j]);
    }
    if (x > v[0]) {
      v[0] = x;
      id[0] = col;
    }
  }
};

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The largest value below x (-inf stays): candidates must exceed it. Below +0.0 that is the
// least negative value (the key between them is no value's: -0.0 has +0.0's).
__device__ __forceinline__ float below(unsigned key) {
  if (key <= 0x00800000u) return -INFINITY;  // no value yet, or -inf
  const unsigned k = key - (key == 0x80000000u ? 2u : 1u);
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

// The `top` largest of a part for the lanes with `mine` (a warp's, all its lanes
// together), appended to their rows' candidates. Out of line: rare, and its list
// would take the registers of the loop around it.
static __device__ __noinline__ void list_part(uint32_t tacc, int ncols, int col0, int top, bool mine,
                                              int* count, int2* cand) {
  TopList<LP_MAX_TOP> list;
  list.clear(-INFINITY);
#pragma unroll 1
  for (int c = 0; c < ncols; c += 32) {
    float v[32];
    tmem_ld32(tacc + c, v);
#pragma unroll 1
    for (int e = 0; e < 32; ++e) {
      float x = v[0];
#pragma unroll
      for (int i = 0; i + 1 < 32; ++i) v[i] = v[i + 1];  // v[e] in front, without an index
      if (mine && c + e < ncols && x > list.v[LP_MAX_TOP - 1]) list.insert(x, col0 + c + e);
    }
  }
  if (mine) {
    int n = 0;
#pragma unroll
    for (int j = 0; j < LP_MAX_TOP; ++j) n += (j < top && list.id[j] >= 0) ? 1 : 0;
    int2* dst = cand + atomicAdd(count, n);
#pragma unroll
    for (int j = 0; j < LP_MAX_TOP; ++j)
      if (j < n) dst[j] = make_int2(__float_as_int(list.v[j]), list.id[j]);
  }
}

template <bool PAIR, bool TOP, bool KEEP>
__global__ void __launch_bounds__(kThreads, 1)
    k_lp_head(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
              const __grid_constant__ CUtensorMap tmE, const __grid_constant__ CUtensorMap tmD,
              const HeadParams p) {
  constexpr int SB = stage_bytes(PAIR);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* stg = smem_raw + (base - raw) + p.nst * SB;
  Ctrl* cb = reinterpret_cast<Ctrl*>(stg + kEpiWarps * stage_bufs(TOP, KEEP) * OUT_BUF_BYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  let_next_launch();

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&cb->full[s]), 1);
      mbar_init(smem_u32(&cb->empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&cb->tmem_full[a]), 1);
      mbar_init(smem_u32(&cb->tmem_empty[a]), PAIR ? 2 * kEpiWarps : kEpiWarps);
    }
    mbar_init(smem_u32(&cb->drain), 1);
    cb->abort = 0;
    cb->timeout_ns = p.timeout_ns;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_tensormap(&tmA);
    prefetch_tensormap(&tmB);
    if (KEEP) prefetch_tensormap(&tmE);
    if (TOP) prefetch_tensormap(&tmD);
  }
  if (PAIR) cluster_sync_all();
  if (warp == 1) tmem_alloc<PAIR>(smem_u32(&cb->tmem_base), TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = cb->tmem_base;
  const int unit0 = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  const int unit_step = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;

  // bands of group_m m-units sweeping all n-blocks (the band of X stays in L2
  // while W streams once per band)
  auto tile_coords = [&](int t, int& mb, int& nb) {
    const int band = t / (p.group_m * p.num_n_blocks);
    const int m0 = band * p.group_m;
    const int gm = min(p.group_m, p.m_units - m0);
    const int r = t - band * p.group_m * p.num_n_blocks;
    const int mu = m0 + r % gm;
    nb = r / gm;
    mb = PAIR ? 2 * mu + (int)rank : mu;
  };

  // (all lanes wait, one issues: elect.cuh)
  auto wait_all = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_bar(cb, bar, parity, p.status)) != 0;
  };
  if (warp == 0) {
    // ---------------- TMA producer (hand-over of a pair's stages: gemm_tc_kernel.cuh) ----------------
    int stage = 0;
    uint32_t phase = 0;
    uint32_t filled = 0;  // stages filled since the start
    bool ok = true;
    const uint32_t flip = (PAIR && !leader) ? 0u : 1u;
    const uint32_t copied = A_BYTES + (PAIR ? p.bn / 2 : p.bn) * (BK * 2);  // of a stage's SB
    for (int t = unit0; ok && t < p.num_units; t += unit_step) {
      int mb, nb;
      tile_coords(t, mb, nb);
      const int nrow = nb * p.bn + (PAIR ? (int)rank * (p.bn / 2) : 0);
      for (int kb = 0; kb < p.num_k_blocks; ++kb) {
        if (!wait_all(smem_u32(&cb->empty[stage]), phase ^ flip)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t sa = base + stage * SB;
          uint32_t fb;
          if (PAIR) {
            fb = map_to_cta(smem_u32(&cb->full[stage]), 0);
            if (leader) {
              mbar_arrive_expect_tx(smem_u32(&cb->full[stage]), 2 * copied);
              mbar_arrive_remote_relaxed(map_to_cta(smem_u32(&cb->empty[stage]), 1));
            }
          } else {
            fb = smem_u32(&cb->full[stage]);
            mbar_arrive_expect_tx(fb, copied);
          }
          tma_operand<PAIR>(sa, &tmA, fb, kb * BK, mb * BM);
          tma_operand<PAIR>(sa + A_BYTES, &tmB, fb, kb * BK, nrow);
        }
        __syncwarp();
        ++filled;
        if (++stage == p.nst) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // every copy has landed before the CTA may exit: the last fill of each stage
    if (!PAIR || leader)
      for (int s = 0; s < p.nst; ++s) {
        const uint32_t fills = filled / p.nst + ((uint32_t)s < filled % p.nst ? 1u : 0u);
        if (fills > 0) wait_bar(cb, smem_u32(&cb->full[s]), (fills - 1) & 1u, p.status);
      }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (leader) {
      // (N, from bit 17 on, is the tile's columns)
      const uint32_t idesc = instr_desc(false, false, PAIR) - ((uint32_t)((BN - p.bn) >> 3) << 17);
      int stage = 0;
      uint32_t phase = 0;
      int local = 0;
      bool ok = true;
      bool any = false;
      for (int t = unit0; ok && t < p.num_units; t += unit_step, ++local) {
        const int acc = local & 1;
        if (!__all_sync(0xffffffffu, wait_bar<PAIR>(cb, smem_u32(&cb->tmem_empty[acc]),
                                                    ((local >> 1) & 1) ^ 1u, p.status)))
          break;
        tc_fence_after();
        const uint32_t tmem_d = tmem_base + acc * ACC_COLS;
        for (int kb = 0; kb < p.num_k_blocks; ++kb) {
          if (!wait_all(smem_u32(&cb->full[stage]), phase)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t sa = base + stage * SB;
#pragma unroll
            for (int kk = 0; kk < BK / UMMA_K; ++kk)
              mma_bf16<PAIR>(tmem_d, smem_desc(sa + kk * (UMMA_K * 2), 16, 1024),
                             smem_desc(sa + A_BYTES + kk * (UMMA_K * 2), 16, 1024), idesc,
                             (kb > 0 || kk > 0) ? 1u : 0u);
            mma_commit<PAIR>(smem_u32(&cb->empty[stage]));
          }
          __syncwarp();
          any = true;
          if (++stage == p.nst) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (elect_one()) mma_commit<PAIR>(smem_u32(&cb->tmem_full[acc]));
        __syncwarp();
      }
      if (any) {
        if (elect_one()) mma_commit<PAIR>(smem_u32(&cb->drain));
        __syncwarp();
        wait_bar(cb, smem_u32(&cb->drain), 0, p.status);
      }
    }
  } else {
    // ---------------- epilogue: one row of 128 columns to a thread ----------------
    const int sub = warp & 3;         // tensor-memory lane quarter of this warp
    const int grp = (warp - 2) >> 2;  // columns 0..127 or 128..255 of the tile
    const int ew = warp - 2;
    int local = 0;
    int sbuf = 0;
    wait_for_previous();  // (the zeroed counts; the products need nothing of it)
    for (int t = unit0; t < p.num_units; t += unit_step, ++local) {
      int mb, nb;
      tile_coords(t, mb, nb);
      const int acc = local & 1;
      const int64_t row0 = (int64_t)mb * BM + sub * 32, row = row0 + lane;
      const bool row_ok = row < p.m;
      const int col0 = nb * p.bn + grp * (p.bn / 2);
      const int ncols = (int)min((int64_t)(p.bn / 2), p.n - col0);
      const bool live = row0 < p.m && ncols > 0;  // of this warp
      int lab = -1;
      if (live && row_ok) {
        if (p.labels) {
          const int64_t y = p.labels[row];
          if (y >= col0 && y < col0 + ncols) lab = (int)(y - col0);
        }
      }
      const bool listed = TOP && live && nb >= p.dump_blocks;
      // the least of the row's group maxima, read from L2 (0: a group has none yet)
      auto least = [&]() {
        unsigned l = 0xffffffffu;
        if (row_ok) {
#pragma unroll 8
          for (int j = 0; j < p.top; ++j) l = min(l, __ldcg(p.gmax + j * p.m + row));
        }
        return l;
      };
      unsigned low = listed ? least() : 0xffffffffu;
      bool ok = true;
      if (lane == 0) {
        ok = wait_bar<PAIR>(cb, smem_u32(&cb->tmem_full[acc]), (local >> 1) & 1, p.status);
        if (PAIR && ok && leader && ew == 0)
          mbar_arrive_remote_relaxed(map_to_cta(smem_u32(&cb->tmem_full[acc]), 1));
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      tc_fence_after();
      if (live) {
        // (the tiles that fill the groups may have ended since)
        if (listed && __any_sync(0xffffffffu, low == 0)) low = least();
        const uint32_t tacc = tmem_base + ((uint32_t)(sub * 32) << 16) + acc * ACC_COLS +
                              grp * (p.bn / 2);
        // ---- the maximum and the label's logit; the columns that reach thr ----
        float mx = -INFINITY;
        unsigned hit[4] = {0u, 0u, 0u, 0u};  // by chunk of 32 columns
        auto scan = [&](float thr, bool again) {
#pragma unroll 1
          for (int c = 0; c < ncols; c += 32) {
            float v[32];
            tmem_ld32(tacc + c, v);
            if (ncols - c < 32) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (c + e >= ncols) v[e] = -INFINITY;
            }
            float cm = v[0];
#pragma unroll
            for (int e = 1; e < 32; ++e) cm = fmaxf(cm, v[e]);
            mx = fmaxf(mx, cm);
            const bool has = lab >= c && lab < c + 32;
            if (!again && __any_sync(0xffffffffu, has)) {
              float z = 0.f;
#pragma unroll
              for (int e = 0; e < 32; ++e) z = c + e == lab ? v[e] : z;
              if (has) p.zy[row] = z;
            }
            if (listed) {
              // rows past the last hold zeros and list nothing
              const bool want = row_ok && cm > thr;
              if (again || __any_sync(0xffffffffu, want)) {
                unsigned w = 0;
#pragma unroll
                for (int e = 0; e < 32; ++e) w |= v[e] > thr ? 1u << e : 0u;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  if (c == q * 32) hit[q] = want ? w : 0u;
              }
            }
          }
        };
        auto hits = [&]() { return __popc(hit[0]) + __popc(hit[1]) + __popc(hit[2]) + __popc(hit[3]); };
        scan(listed ? below(low) : -INFINITY, false);
        const int part = nb * 2 + grp;
        // (at once: the tiles that come next are waiting for a threshold)
        if (TOP && row_ok && mx > -INFINITY)
          atomicMax(p.gmax + (part % p.top) * p.m + row, lp_key(mx));
        int2* dst = nullptr;
        if (listed) {
          int n = hits();
          if (__any_sync(0xffffffffu, n > p.top)) {  // the threshold may have risen since
            scan(below(least()), true);
            n = hits();
          }
          const bool many = n > p.top;
          int2* cand = p.cand + (row_ok ? row : 0) * p.parts * p.top;
          if (__any_sync(0xffffffffu, many)) {
            list_part(tacc, ncols, col0, p.top, many, p.count + (row_ok ? row : 0), cand);
            if (many) hit[0] = hit[1] = hit[2] = hit[3] = 0u;
          }
          if (n > 0 && !many) dst = cand + atomicAdd(p.count + row, n);
        }
        // ---- sums relative to the maximum ----
        const float ref = mx == -INFINITY ? 0.f : mx;
        const float2 c2 = make_float2(p.c, p.c), nref = make_float2(-ref, -ref);
        float2 d = make_float2(0.f, 0.f), s = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int c = 0; c < ncols; c += 32) {
          float v[32];
          tmem_ld32(tacc + c, v);
          if (ncols - c < 32) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c + e >= ncols) v[e] = -INFINITY;
          }
          if (TOP && !listed) {
            // 32 rows of 128 bytes; of 2^t's buffers the one that is not being filled
            uint8_t* buf = stg + (ew * stage_bufs(TOP, KEEP) + (KEEP ? sbuf ^ 1 : 0)) * OUT_BUF_BYTES;
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *reinterpret_cast<float4*>(buf + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                  make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&tmD, smem_u32(buf), (nb * 2 + grp) * LP_PART_COLS + c, (int32_t)row0);
              bulk_commit();
            }
          } else if (TOP) {
            unsigned w = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) w = c == q * 32 ? hit[q] : w;
            if (__any_sync(0xffffffffu, w != 0)) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (w >> e & 1) *dst++ = make_int2(__float_as_int(v[e]), col0 + c + e);
            }
          }
          if (KEEP && (c & 32) == 0) {
            // the store that last used this buffer has read it
            if (lane == 0) bulk_wait_read_1();
            __syncwarp();
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 x = __fmul2_rn(__fadd2_rn(make_float2(v[e], v[e + 1]), nref), c2);
            const float2 y = make_float2(ex2f_approx(x.x), ex2f_approx(x.y));
            d = __fadd2_rn(d, y);
            // 2^t t is 0 for a logit of -inf, and NaN stays NaN
            s = __ffma2_rn(y, make_float2(fmaxf(x.x, -1024.f), fmaxf(x.y, -1024.f)), s);
            v[e] = y.x;
            v[e + 1] = y.y;
          }
          if (KEEP) {
            uint8_t* srow = stg + ((ew * kKeepBufs + sbuf) * 32 + lane) * 128;
            const int h = (c & 32) ? 4 : 0;
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<uint4*>(srow + (((h + q) ^ (lane & 7)) << 4)) =
                  make_uint4(pack_half(v[q * 8], v[q * 8 + 1]), pack_half(v[q * 8 + 2], v[q * 8 + 3]),
                             pack_half(v[q * 8 + 4], v[q * 8 + 5]),
                             pack_half(v[q * 8 + 6], v[q * 8 + 7]));
            if ((c & 32) || c + 32 >= ncols) {
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_2d(&tmE, smem_u32(stg + (ew * kKeepBufs + sbuf) * OUT_BUF_BYTES),
                             col0 + (c & ~63), (int32_t)row0);
                bulk_commit();
              }
              sbuf ^= 1;
            }
          }
        }
        if (row_ok) {
          p.part[row * p.parts + part] =
              make_float4(mx, d.x + d.y, s.x + s.y, 0.f);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR && !leader)
          mbar_arrive_remote_relaxed(map_to_cta(smem_u32(&cb->tmem_empty[acc]), 0));
        else
          mbar_arrive(smem_u32(&cb->tmem_empty[acc]));
      }
    }
    if ((KEEP || TOP) && lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync_all();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc<PAIR>(tmem_base, TMEM_COLS);
  }
}

template <bool PAIR, bool TOP, bool KEEP>
cudaError_t launch_v(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& me,
                     const CUtensorMap& md, const HeadParams& p, bool after, cudaStream_t st) {
  auto kern = k_lp_head<PAIR, TOP, KEEP>;
  const int smem = head_smem(p.nst, PAIR, TOP, KEEP);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX);
  if (e != cudaSuccess) return e;
  if (!PAIR) {
    const int grid = p.num_units < num_sms() ? p.num_units : num_sms();
    if (after) return launch_dependent(kern, grid, kThreads, smem, st, ma, mb, me, md, p);
    kern<<<grid, kThreads, smem, st>>>(ma, mb, me, md, p);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static int resident[64] = {0};  // clusters that run at once, by device
  int dev = 0;
  cudaGetDevice(&dev);
  int most = dev >= 0 && dev < 64 ? resident[dev] : 0;
  if (most == 0) {
    cfg.gridDim = dim3(2 * (num_sms() / 2));
    if (cudaOccupancyMaxActiveClusters(&most, kern, &cfg) != cudaSuccess || most <= 0) most = 1;
    if (dev >= 0 && dev < 64) resident[dev] = most;
  }
  cfg.gridDim = dim3(2 * (p.num_units < most ? p.num_units : most));
  if (after) cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kern, ma, mb, me, md, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool PAIR, bool KEEP>
cudaError_t launch_k(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& me,
                     const CUtensorMap& md, const HeadParams& p, bool after, cudaStream_t st) {
  return p.top ? launch_v<PAIR, true, KEEP>(ma, mb, me, md, p, after, st)
               : launch_v<PAIR, false, KEEP>(ma, mb, me, md, p, after, st);
}

}  // namespace

bool lp_head_supported(const LpHeadArgs& a) {
  auto al = [](const void* q) { return ((uintptr_t)q & 15u) == 0; };
  return a.m > 0 && a.n > 0 && a.k > 0 && a.bn >= BN / 2 && a.bn <= BN && a.bn % 16 == 0 &&
         (a.e == nullptr || a.bn == BN) && al(a.x) && al(a.w) && a.ldx % 8 == 0 && a.ldw % 8 == 0 &&
         (a.e == nullptr || (al(a.e) && a.lde % 8 == 0)) && a.m < (1ll << 31) - 512 &&
         a.n < (1ll << 31) - 512 && a.k < (1ll << 31);
}

namespace {
struct HeadSchedule {
  bool pair;
  int64_t nblocks, m_units, group_m;
};
int64_t up(int64_t x, int64_t q) { return (x + q - 1) / q; }
// rounds of tiles: one CTA each | CTA pairs
int64_t rounds(int64_t mblocks, int64_t nblocks, int64_t sms, bool pair) {
  return pair ? up(up(mblocks, 2) * nblocks, sms >= 2 ? sms / 2 : 1) : up(mblocks * nblocks, sms);
}
// the schedule rule of launch_gemm_tc (gemm_tc.cu)
bool use_pair(int64_t m, int64_t k, int64_t pair_cost, int64_t one_cost) {
  return m > BM && up(k, BK) >= 4 && pair_cost * 100 <= one_cost * 112;
}
HeadSchedule head_schedule(int64_t m, int64_t n, int64_t k, int64_t sms, int bn) {
  HeadSchedule h;
  const int64_t mblocks = up(m, BM);
  h.nblocks = up(n, bn);
  h.pair = use_pair(m, k, rounds(mblocks, h.nblocks, sms, true), rounds(mblocks, h.nblocks, sms, false));
  h.m_units = h.pair ? up(mblocks, 2) : mblocks;
  // bands of about 32 MB of X, as for the logits product
  const int64_t gm = (32ll << 20) / ((int64_t)BM * (h.pair ? 2 : 1) * k * 2);
  h.group_m = gm < 1 ? 1 : gm > h.m_units ? h.m_units : gm;
  return h;
}
}  // namespace

int lp_head_tile_cols(int64_t m, int64_t n, int64_t k) {
  // More tiles read X more often; where it lies in few slices of L2, that costs more than
  // the rounds gain (H = 2048, V = 40960: 24 rows 57 us instead of 45, 32 rows 36 instead
  // of 42; H = 512: 17 rows 19 instead of 15, 96 rows 14 instead of 15).
  if (m * k * 2 < (128 << 10)) return BN;
  const int64_t sms = TC_PLAN_CTAS, mblocks = up(m, BM);
  int64_t cols[2], cost[2];
  for (int pair = 0; pair < 2; ++pair) {
    const int64_t units = pair ? up(mblocks, 2) : mblocks, at_once = pair ? sms / 2 : sms;
    const int64_t r = rounds(mblocks, up(n, BN), sms, pair != 0);
    const int64_t most = r * at_once / units;  // tiles of a row of tiles in r rounds
    cols[pair] = up(up(n, most > 0 ? most : 1), 16) * 16;
    cols[pair] = cols[pair] < BN / 2 ? BN / 2 : cols[pair] > BN ? BN : cols[pair];
    cost[pair] = r * cols[pair];
  }
  return (int)cols[use_pair(m, k, cost[1], cost[0]) ? 1 : 0];
}

int lp_head_dump_blocks(int64_t m, int64_t n, int64_t k, int top, int bn) {
  if (top == 0 || m <= 0) return 0;
  const HeadSchedule h = head_schedule(m, n, k, TC_PLAN_CTAS, bn);
  const int64_t at_once = h.pair ? TC_PLAN_CTAS / 2 : TC_PLAN_CTAS;
  int64_t blocks = (at_once + h.group_m - 1) / h.group_m;
  // the threshold needs a part in each of the k groups
  if (blocks < (top + 1) / 2) blocks = (top + 1) / 2;
  return (int)(blocks < h.nblocks ? blocks : h.nblocks);
}

cudaError_t launch_lp_head(const LpHeadArgs& a, cudaStream_t st) {
  if (!lp_head_supported(a)) return cudaErrorInvalidValue;
  const HeadSchedule h = head_schedule(a.m, a.n, a.k, num_sms(), a.bn);
  const bool pair = h.pair, keep = a.e != nullptr, after = a.own_zeros;
  CUtensorMap ma, mb, me, md;
  if (!make_tensor_map(&ma, MapType::kBf16, a.x, a.k, a.m, a.ldx, BK, BM) ||
      !make_tensor_map(&mb, MapType::kBf16, a.w, a.k, a.n, a.ldw, BK, pair ? a.bn / 2 : a.bn))
    return cudaErrorInvalidValue;
  me = ma;
  if (keep && !make_tensor_map(&me, MapType::kBf16, a.e, a.lde, a.m, a.lde, 64, 32)) return cudaErrorInvalidValue;
  md = ma;
  if (a.top > 0 && !make_tensor_map(&md, MapType::kF32, a.dump, (int64_t)a.dump_blocks * BN, a.m,
                                 (int64_t)a.dump_blocks * BN, 32, 32))
    return cudaErrorInvalidValue;
  HeadParams p{};
  p.m = a.m; p.n = a.n; p.bn = a.bn;
  p.num_n_blocks = (int)h.nblocks;
  p.num_k_blocks = (int)((a.k + BK - 1) / BK);
  p.m_units = (int)h.m_units;
  if (h.m_units * h.nblocks > 0x7fffffff) return cudaErrorInvalidValue;
  p.num_units = (int)(h.m_units * h.nblocks);
  p.group_m = (int)h.group_m;
  p.nst = head_stages(pair, keep);
  p.c = a.c; p.labels = a.labels; p.part = a.part; p.parts = a.parts; p.zy = a.zy;
  p.dump_blocks = a.dump_blocks;
  p.top = a.top; p.gmax = a.gmax; p.count = a.count; p.cand = a.cand;
  p.timeout_ns = kTimeoutNs;
  p.status = a.status;
  if (pair) return keep ? launch_k<true, true>(ma, mb, me, md, p, after, st) : launch_k<true, false>(ma, mb, me, md, p, after, st);
  return keep ? launch_k<false, true>(ma, mb, me, md, p, after, st) : launch_k<false, false>(ma, mb, me, md, p, after, st);
}

}  // namespace fljsd
