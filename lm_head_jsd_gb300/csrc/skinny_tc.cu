// Products of a few rows (up to 16) with a large weight on the tensor cores: the
// lm_head at a decoding step. Bound by reading w once from HBM, so everything else
// is arranged around that stream:
//  - w's rows are the instruction's 128 rows and x's rows its 16 columns: a tile is
//    128 rows of w, half of what the other way round would take, and spreads over
//    the SMs with less left over (128256 rows: 6.6 rounds of 152 instead of 3.3 of
//    twice the length);
//  - x stays in shared memory for the CTA's whole life (2 KB for each 128 bytes of
//    k) where it fits beside five stages of w. One row of x lies in one or two
//    slices of L2; read again for every tile by every SM, it held the stream up
//    (one row took 220 us where sixteen took 175 us; H = 4096, V = 128256);
//  - the rest of shared memory is the ring of w's tiles, 16 KB each.
// For token log probabilities the epilogue reduces what it holds: each warp its 32
// columns of each row, over all of the CTA's tiles, in some 500 instructions of a tile's
// 25 us (one row of H = 4096, V = 128256, with the join: 161 us, 166 with the logits read
// again by the row kernels; H = 512, V = 40960: 14.4 and 16.5).
// H = 4096, V = 128256: bf16 160 us = 6.6 TB/s, e4m3 with the quantisation of x in front
// 84 us = 6.2 TB/s (0.97 and 0.92 of a copy's rate).
// e4m3 (see fp8_gemm.cu): every 128-deep block has an accumulator of its own in a
// ring of eight, and is scaled and added in fp32 registers.
#include "dependent.cuh"
#include "elect.cuh"
#include "gemm_tc_kernel.cuh"
#include "lp_mds.cuh"
#include "skinny_tc.cuh"
#include "tensor_map.cuh"

namespace fljsd {
namespace {

using namespace tcgemm;

constexpr int kThreads = 192;  // producer, MMA, four epilogue warps
constexpr int kStage = BM * 128;        // a tile of w: 128 rows of 128 bytes
constexpr int kXBlock = SK_ROWS * 128;  // x beside it
constexpr int kMaxStages = 13;
constexpr int kMinStages = 5;
constexpr int kAccs = 8, kAccCols = 16;
constexpr int kTmemCols = kAccs * kAccCols;
constexpr int kCtrl = 1024;
constexpr int kScaleBlocks = 256;  // blocks of k whose x scales are held in shared memory

struct SkCtrl {
  unsigned long long full[kMaxStages], empty[kMaxStages];
  unsigned long long tmem_full[kAccs], tmem_empty[kAccs];
  unsigned long long x_full, drain;
  unsigned long long timeout_ns;
  uint32_t tmem_base;
  volatile int abort;
};
static_assert(sizeof(SkCtrl) <= kCtrl, "control block");

struct SkParams {
  int64_t m, n;
  int num_tiles, num_k_blocks, nst, resident;
  bool own_x, zero_status;
  const float *sx, *sw;
  void* out;
  int64_t ldo;
  unsigned long long timeout_ns;
  int* status;
  float4* part;
  float* cmax;
  float c;
  const int64_t* labels;
  float* zy;
};

__device__ __forceinline__ bool sk_wait(SkCtrl* cb, uint32_t bar, uint32_t parity, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = globaltimer();
  for (uint32_t it = 0;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 63u) {
      if (cb->abort) return false;
      if (globaltimer() - t0 > cb->timeout_ns) {
        cb->abort = 1;
        if (status) atomicExch(status, (int)FLJSD_ERR_TIMEOUT);
        return false;
      }
    }
  }
}

// 32 lanes x 16 columns of accumulators.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
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

// M = 128, N = 16, fp32 accumulator, both operands K-major; bf16 (format 1) or
// e4m3 (format 0 of kind::f8f6f4).
template <bool E4M3>
__device__ __forceinline__ void mma16(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                      uint32_t accumulate) {
  constexpr uint32_t idesc = (1u << 4) | (E4M3 ? 0u : (1u << 7) | (1u << 10)) |
                             ((uint32_t)(SK_ROWS >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
  if (E4M3)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}

__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <bool E4M3, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    k_skinny(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
             const SkParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ float s_sx[E4M3 ? kScaleBlocks * SK_ROWS : 1];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const int nkb = p.num_k_blocks;
  const uint32_t xbase = base;  // resident x; otherwise behind each stage
  const int sb = kStage + (p.resident ? 0 : kXBlock);
  const uint32_t wbase = base + (p.resident ? nkb * kXBlock : 0);
  SkCtrl* cb = reinterpret_cast<SkCtrl*>(smem_raw + (wbase - raw) + p.nst * sb);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  let_next_launch();
  constexpr int KE = E4M3 ? 128 : 64;  // elements in 128 bytes

  if (threadIdx.x == 0) {
    if (p.zero_status && blockIdx.x == 0) *p.status = 0;  // (long before a wait runs out)
    for (int s = 0; s < p.nst; ++s) {
      mbar_init(smem_u32(&cb->full[s]), 1);
      mbar_init(smem_u32(&cb->empty[s]), 1);
    }
    for (int a = 0; a < kAccs; ++a) {
      mbar_init(smem_u32(&cb->tmem_full[a]), 1);
      mbar_init(smem_u32(&cb->tmem_empty[a]), 4);
    }
    mbar_init(smem_u32(&cb->x_full), 1);
    mbar_init(smem_u32(&cb->drain), 1);
    cb->abort = 0;
    cb->timeout_ns = p.timeout_ns;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_tensormap(&tmX);
    prefetch_tensormap(&tmW);
  }
  if (warp == 1) tmem_alloc<false>(smem_u32(&cb->tmem_base), kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = cb->tmem_base;

  // (all lanes wait, one issues: elect.cuh)
  auto wait_all = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, sk_wait(cb, bar, parity, p.status)) != 0;
  };
  if (warp == 0) {
    // ---------------- TMA producer ----------------
    int stage = 0;
    uint32_t phase = 0;
    uint32_t filled = 0;  // stages filled since the start
    bool ok = true;
    // x is asked for once the stages are full of w (which x, where it shares them, cannot be)
    bool have_x = false;
    auto ask_x = [&]() {
      wait_for_previous();
      if (p.resident && (int)blockIdx.x < p.num_tiles && elect_one()) {
        const uint32_t xb = smem_u32(&cb->x_full);
        mbar_arrive_expect_tx(xb, nkb * kXBlock);
        for (int kb = 0; kb < nkb; ++kb) tma_load_2d(xbase + kb * kXBlock, &tmX, xb, kb * KE, 0);
      }
      __syncwarp();
      have_x = true;
    };
    if (!p.resident || !p.own_x) ask_x();
    for (int t = blockIdx.x; ok && t < p.num_tiles; t += gridDim.x) {
      for (int kb = 0; kb < nkb; ++kb) {
        if (!have_x && filled == (uint32_t)p.nst) ask_x();
        if (!wait_all(smem_u32(&cb->empty[stage]), phase ^ 1u)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t dst = wbase + stage * sb, fb = smem_u32(&cb->full[stage]);
          mbar_arrive_expect_tx(fb, sb);
          tma_load_2d(dst, &tmW, fb, kb * KE, t * BM);
          if (!p.resident) tma_load_2d(dst + kStage, &tmX, fb, kb * KE, 0);
        }
        __syncwarp();
        ++filled;
        if (++stage == p.nst) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!have_x) ask_x();
    // every copy has landed before the CTA may exit: the last fill of each stage
    if (p.resident && (int)blockIdx.x < p.num_tiles)
      sk_wait(cb, smem_u32(&cb->x_full), 0, p.status);
    for (int s = 0; s < p.nst; ++s) {
      const uint32_t fills = filled / p.nst + ((uint32_t)s < filled % p.nst ? 1u : 0u);
      if (fills > 0) sk_wait(cb, smem_u32(&cb->full[s]), (fills - 1) & 1u, p.status);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    int stage = 0;
    uint32_t phase = 0;
    uint32_t use = 0;  // accumulators handed out
    bool any = false;
    bool ok = true;
    if (p.resident && (int)blockIdx.x < p.num_tiles) ok = wait_all(smem_u32(&cb->x_full), 0);
    for (int t = blockIdx.x; ok && t < p.num_tiles; t += gridDim.x) {
      for (int kb = 0; kb < nkb; ++kb) {
        const int acc = use % kAccs;
        if (((E4M3 || kb == 0) &&
             !wait_all(smem_u32(&cb->tmem_empty[acc]), ((use / kAccs) & 1u) ^ 1u)) ||
            !wait_all(smem_u32(&cb->full[stage]), phase)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const bool last = E4M3 || kb == nkb - 1;  // of this accumulator
        if (elect_one()) {
          const uint32_t sa = wbase + stage * sb;
          const uint32_t sx = p.resident ? xbase + kb * kXBlock : sa + kStage;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // 32 bytes of k each
            mma16<E4M3>(tmem_base + acc * kAccCols, smem_desc(sa + kk * 32, 16, 1024),
                        smem_desc(sx + kk * 32, 16, 1024), (kk > 0 || (!E4M3 && kb > 0)) ? 1u : 0u);
          mma_commit<false>(smem_u32(&cb->empty[stage]));
          if (last) mma_commit<false>(smem_u32(&cb->tmem_full[acc]));
        }
        __syncwarp();
        any = true;
        if (last) ++use;
        if (++stage == p.nst) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (any) {
      if (elect_one()) mma_commit<false>(smem_u32(&cb->drain));
      __syncwarp();
      sk_wait(cb, smem_u32(&cb->drain), 0, p.status);
    }
  } else {
    // ---------------- epilogue: one row of w (a column of out) to a thread ----------------
    const int sub = warp & 3;
    uint32_t use = 0;
    bool ok = true;
    Mds all{-INFINITY, 0.f, 0.f};  // of the tiles so far
    wait_for_previous();
    if (E4M3) {
      for (int i = threadIdx.x - 64; i < nkb * SK_ROWS; i += 128) {
        const int j = i % SK_ROWS;
        s_sx[i] = j < p.m ? p.sx[(int64_t)(i / SK_ROWS) * p.m + j] : 0.f;
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
    }
    for (int t = blockIdx.x; ok && t < p.num_tiles; t += gridDim.x) {
      const int64_t col = (int64_t)t * BM + sub * 32 + lane;
      float sum[SK_ROWS];
#pragma unroll
      for (int j = 0; j < SK_ROWS; ++j) sum[j] = 0.f;
      const int steps = E4M3 ? nkb : 1;
      for (int kb = 0; kb < steps; ++kb, ++use) {
        const int acc = use % kAccs;
        const float sw = E4M3 ? __ldg(p.sw + (int64_t)t * nkb + kb) : 1.f;
        ok = sk_wait(cb, smem_u32(&cb->tmem_full[acc]), (use / kAccs) & 1u, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        float v[SK_ROWS];
        tmem_ld16(tmem_base + ((uint32_t)(sub * 32) << 16) + acc * kAccCols, v);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&cb->tmem_empty[acc]));
#pragma unroll
        for (int j = 0; j < SK_ROWS; ++j)
          sum[j] = E4M3 ? __fmaf_rn(v[j], s_sx[kb * SK_ROWS + j] * sw, sum[j]) : v[j];
      }
      // (m, d, s) of this warp's columns, row by row; lane j keeps row j's
      if (!E4M3 && ok && p.part) {
        Mds mine{-INFINITY, 0.f, 0.f};
#pragma unroll
        for (int j0 = 0; j0 < SK_ROWS; j0 += 4) {  // four rows' reductions side by side
          if (j0 >= p.m) break;
          Mds x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float z = col < p.n ? sum[j0 + i] : -INFINITY;
            // (NaN is no maximum, but stays in the sums)
            x[i] = warp_mds(Mds{fmaxf(z, -INFINITY), z == -INFINITY ? 0.f : z != z ? z : 1.f, 0.f},
                            p.c);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (lane == j0 + i) mine = x[i];
        }
        if (p.labels && col < p.n) {
#pragma unroll
          for (int j = 0; j < SK_ROWS; ++j)
            if (j < p.m && p.labels[j] == col) p.zy[j] = sum[j];
        }
        if (p.cmax && lane < p.m) p.cmax[((int64_t)lane * p.num_tiles + t) * 4 + sub] = mine.m;
        all = merge(all, mine, p.c);
      }
      if (ok && col < p.n && p.out) {
        T* o = reinterpret_cast<T*>(p.out) + col;
#pragma unroll
        for (int j = 0; j < SK_ROWS; ++j)
          if (j < p.m) put(o + j * p.ldo, sum[j]);
      }
    }
    if (!E4M3 && p.part && lane < p.m)
      p.part[((int64_t)lane * gridDim.x + blockIdx.x) * 4 + sub] = make_float4(all.m, all.d, all.s, 0.f);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc<false>(tmem_base, kTmemCols);
  }
}

template <bool E4M3, typename T>
cudaError_t launch(const CUtensorMap& mx, const CUtensorMap& mw, const SkParams& p, int smem,
                   cudaStream_t st) {
  auto kern = k_skinny<E4M3, T>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int grid = p.num_tiles < num_sms() ? p.num_tiles : num_sms();
  if (p.own_x) return launch_dependent(kern, grid, kThreads, smem, st, mx, mw, p);
  kern<<<grid, kThreads, smem, st>>>(mx, mw, p);
  return cudaGetLastError();
}

}  // namespace

bool skinny_supported(const SkinnyArgs& a) {
  auto al = [](const void* q) { return ((uintptr_t)q & 15u) == 0; };
  const int64_t unit = a.e4m3 ? 16 : 8;  // elements of 16 bytes
  return a.m > 0 && a.m <= SK_ROWS && a.n > 0 && a.n < (1ll << 31) - BM && a.k > 0 &&
         a.k < (1ll << 24) && al(a.x) && al(a.w) && a.ldx % unit == 0 && a.ldw % unit == 0 &&
         (!a.e4m3 || a.k <= (int64_t)kScaleBlocks * 128);
}

int64_t skinny_parts(int64_t n) {
  const int64_t tiles = (n + BM - 1) / BM;
  return 4 * (tiles < num_sms() ? tiles : num_sms());
}

cudaError_t launch_skinny(const SkinnyArgs& a, cudaStream_t st) {
  if (!skinny_supported(a)) return cudaErrorInvalidValue;
  SkParams p{};
  const int ke = a.e4m3 ? 128 : 64;
  p.m = a.m; p.n = a.n;
  p.num_tiles = (int)((a.n + BM - 1) / BM);
  p.num_k_blocks = (int)((a.k + ke - 1) / ke);
  const int fixed = kCtrl + 1024 + (a.e4m3 ? kScaleBlocks * SK_ROWS * (int)sizeof(float) : 0) + 1024;
  const int64_t xb = (int64_t)p.num_k_blocks * kXBlock;
  p.resident = xb + kMinStages * kStage + fixed <= SMEM_MAX;
  const int sb = kStage + (p.resident ? 0 : kXBlock);
  const int left = SMEM_MAX - fixed - (p.resident ? (int)xb : 0);
  p.nst = left / sb < kMaxStages ? left / sb : kMaxStages;
  p.sx = a.sx; p.sw = a.sw; p.out = a.out; p.ldo = a.ldo;
  p.timeout_ns = kTimeoutNs;
  p.status = a.status;
  p.own_x = a.own_x;
  p.zero_status = a.zero_status;
  p.part = a.part; p.cmax = a.cmax; p.c = a.c; p.labels = a.labels; p.zy = a.zy;
  CUtensorMap mx, mw;
  const MapType mt = a.e4m3 ? MapType::kU8 : MapType::kBf16;
  const bool ok = make_tensor_map(&mx, mt, a.x, a.k, a.m, a.ldx, ke, SK_ROWS) &&
                  make_tensor_map(&mw, mt, a.w, a.k, a.n, a.ldw, ke, BM);
  if (!ok) return cudaErrorInvalidValue;
  const int smem = (p.resident ? (int)xb : 0) + p.nst * sb + kCtrl + 1024;
  if (a.e4m3)
    return a.out_bf16 ? launch<true, __nv_bfloat16>(mx, mw, p, smem, st)
                      : launch<true, float>(mx, mw, p, smem, st);
  return launch<false, float>(mx, mw, p, smem, st);
}

}  // namespace fljsd
