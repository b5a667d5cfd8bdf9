// Product in 8-bit floating point with a scale for each block of 128 (sm_103a):
//   out[i, j] = sum_b sx[b, i] sw[j / 128, b] sum_{k in block b} qx[i, k] qw[j, k]
// with e4m3 codes qx [m x k], qw [n x k]; the inner sums on the tensor cores
// (tcgen05.mma kind::f8f6f4, products exact, fp32 sums), the outer sum in fp32
// registers.
//
// One CTA computes a 128 x 256 tile. Each 128-deep block of the contraction is one
// stage of the TMA ring (128-byte rows, 128B swizzle) and starts a new accumulator
// in tensor memory; the two accumulators alternate, so that while the tensor cores
// form one block's sums, eight warps add the other's, scaled, to 128 fp32 registers
// a thread (one row, half of the columns). A scale that is no power of two cannot be
// applied by the tensor cores, and folding it into the codes would round them again.
// Two more warps bring the scales: they multiply x's of each row with w's of each
// half of the columns into shared memory as soon as an accumulator is free, long
// before its products are done, and what the epilogue waits for is all three. (Loaded
// by the epilogue itself, however far ahead, they cost it 90 ns a block.)
//
// What bounds it: at full clocks a 128 x 256 x 128 block of a tile takes 990 cycles
// (4096 x 32768 x 4096 of zeros, 412 us = 2.67 PFLOP/s), where the products alone would
// take 512 and shared memory 768 (96 KB written and read again); with random codes the
// card's power limit lowers the clock to 1.75 to 1.85 GHz (460 to 480 us), and what saves
// cycles saves less time than it should. The additions (2.6 cycles for each FFMA2) take
// some 150 ns a block and reading the accumulator about as much; what the two accumulators
// add is the way from commit to hand-back and on to the next products.
//
// Quantisation: one scale for 1 x 128 of x (or 128 x 128 of a weight), amax / 448;
// codes are the nearest to x (448 (1 / amax)).
#include "dependent.cuh"
#include "elect.cuh"
#include "gemm_tc_kernel.cuh"
#include "skinny_tc.cuh"
#include "tensor_map.cuh"

#include <cuda_fp8.h>

namespace fljsd {
namespace {

using namespace tcgemm;

constexpr int FB = 128;         // elements of a scale's block, and of a stage's rows
constexpr int F_UMMA_K = 32;
constexpr int F_ACCS = TMEM_COLS / ACC_COLS;  // accumulators in tensor memory
constexpr int F_EPI = 8;        // epilogue warps
constexpr int F_OUT_BYTES = 32 * 64;  // an epilogue warp's staging: 32 rows of 64 bytes
// Registers: launched with 168 for each of 12 warps; the four that copy and issue
// keep 40, the eight epilogue warps take 232 (128 x 40 + 256 x 232 = 384 x 168).
constexpr int F_REGS_LOW = 40, F_REGS_HIGH = 232;
constexpr int F_THREADS = 128 + 32 * F_EPI;
constexpr int F_STAGES = 4;
constexpr int F_STAGE_BYTES = (BM + BN) * FB;
constexpr int F_SCALES = F_ACCS * 2 * BM;  // of each accumulator: column half x row
constexpr int F_SMEM = F_STAGES * F_STAGE_BYTES + F_EPI * F_OUT_BYTES +
                       F_SCALES * (int)sizeof(float) + 1024 + CTRL_BYTES;
static_assert(F_SMEM <= SMEM_MAX && F_STAGES <= STAGES && F_ACCS == 2, "control block and memory");

// fp32 accumulator, e4m3 operands (format 0), both K-major
constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);

__device__ __forceinline__ void mma_e4m3(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(kIdesc), "r"(accumulate));
}

// 32 lanes x 32 columns of accumulators, in flight until ld_wait names their registers.
__device__ __forceinline__ void ld_start(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr));
}
// Every load started by this thread is done (nothing that uses r moves before it).
__device__ __forceinline__ void ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void add32(float2* sum, const uint32_t (&r)[32], float s) {
  const float2 s2 = make_float2(s, s);
#pragma unroll
  for (int i = 0; i < 16; ++i)
    sum[i] = __ffma2_rn(make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), s2,
                        sum[i]);
}

struct F8Params {
  int64_t m, n;
  int num_n_blocks, num_k_blocks, m_units, num_units, group_m;
  const float* sx;  // [num_k_blocks x m]
  const float* sw;  // [ceil(n / 128) x num_k_blocks]
  void* out;
  int64_t ldo;
  int use_tma;      // rows of out are whole 16-byte units
  unsigned long long timeout_ns;
  int* status;
};

template <typename T>
__global__ void __launch_bounds__(F_THREADS, 1)
    k_fp8_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ CUtensorMap tmO, const F8Params p) {
  constexpr int COLS = 64 / sizeof(T);  // columns of a staged row
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* stg = smem_raw + (base - raw) + F_STAGES * F_STAGE_BYTES;
  float* scales = reinterpret_cast<float*>(stg + F_EPI * F_OUT_BYTES);
  Ctrl* cb = reinterpret_cast<Ctrl*>(scales + F_SCALES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < F_STAGES; ++s) {
      mbar_init(smem_u32(&cb->full[s]), 1);
      mbar_init(smem_u32(&cb->empty[s]), 1);
    }
    for (int a = 0; a < F_ACCS; ++a) {
      mbar_init(smem_u32(&cb->tmem_full[a]), 3);  // the products, and two warps of scales
      mbar_init(smem_u32(&cb->tmem_empty[a]), F_EPI);
    }
    mbar_init(smem_u32(&cb->drain), 1);
    cb->abort = 0;
    cb->timeout_ns = p.timeout_ns;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_tensormap(&tmA);
    prefetch_tensormap(&tmB);
    if (p.use_tma) prefetch_tensormap(&tmO);
  }
  if (warp == 1) tmem_alloc<false>(smem_u32(&cb->tmem_base), TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = cb->tmem_base;

  auto tile_coords = [&](int t, int& mb, int& nb) {
    const int band = t / (p.group_m * p.num_n_blocks);
    const int m0 = band * p.group_m;
    const int gm = min(p.group_m, p.m_units - m0);
    const int r = t - band * p.group_m * p.num_n_blocks;
    mb = m0 + r % gm;
    nb = r / gm;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(F_REGS_LOW));
    // (all lanes wait, one issues: elect.cuh)
    auto wait_all = [&](uint32_t bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wait_bar(cb, bar, parity, p.status)) != 0;
    };
    // ---------------- TMA producer ----------------
    if (warp == 0) {
      int stage = 0;
      uint32_t phase = 0;
      uint32_t filled = 0;  // stages filled since the start
      bool ok = true;
      for (int t = blockIdx.x; ok && t < p.num_units; t += gridDim.x) {
        int mb, nb;
        tile_coords(t, mb, nb);
        for (int kb = 0; kb < p.num_k_blocks; ++kb) {
          if (!wait_all(smem_u32(&cb->empty[stage]), phase ^ 1u)) {
            ok = false;
            break;
          }
          if (elect_one()) {
            const uint32_t sa = base + stage * F_STAGE_BYTES;
            const uint32_t fb = smem_u32(&cb->full[stage]);
            mbar_arrive_expect_tx(fb, F_STAGE_BYTES);
            tma_load_2d(sa, &tmA, fb, kb * FB, mb * BM);
            tma_load_2d(sa + BM * FB, &tmB, fb, kb * FB, nb * BN);
          }
          __syncwarp();
          ++filled;
          if (++stage == F_STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // every copy has landed before the CTA may exit: the last fill of each stage
      for (int s = 0; s < F_STAGES; ++s) {
        const uint32_t fills = filled / F_STAGES + ((uint32_t)s < filled % F_STAGES ? 1u : 0u);
        if (fills > 0) wait_bar(cb, smem_u32(&cb->full[s]), (fills - 1) & 1u, p.status);
      }
    }
    // ---------------- MMA issuer: one accumulator for each 128-deep block ----------------
    if (warp == 1) {
      int stage = 0;
      uint32_t phase = 0;
      uint32_t use = 0;  // accumulators handed out
      bool ok = true;
      for (int t = blockIdx.x; ok && t < p.num_units; t += gridDim.x) {
        for (int kb = 0; kb < p.num_k_blocks; ++kb) {
          const uint32_t acc = use % F_ACCS;
          // (one vote for both: the way from a free accumulator to its products counts)
          const bool have = wait_bar(cb, smem_u32(&cb->full[stage]), phase, p.status);
          const bool room = wait_bar(cb, smem_u32(&cb->tmem_empty[acc]), ((use / F_ACCS) & 1u) ^ 1u,
                                     p.status);
          if (!__all_sync(0xffffffffu, have && room)) {
            ok = false;
            break;
          }
          ++use;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t sa = base + stage * F_STAGE_BYTES, sb = sa + BM * FB;
#pragma unroll
            for (int kk = 0; kk < FB / F_UMMA_K; ++kk)
              mma_e4m3(tmem_base + acc * ACC_COLS, smem_desc(sa + kk * F_UMMA_K, 16, 1024),
                       smem_desc(sb + kk * F_UMMA_K, 16, 1024), kk > 0 ? 1u : 0u);
            mma_commit<false>(smem_u32(&cb->tmem_full[acc]));
            mma_commit<false>(smem_u32(&cb->empty[stage]));
          }
          __syncwarp();
          if (++stage == F_STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (use > 0) {
        if (elect_one()) mma_commit<false>(smem_u32(&cb->drain));
        __syncwarp();
        wait_bar(cb, smem_u32(&cb->drain), 0, p.status);
      }
    }
    // ---------------- scales: rows 32 (warp - 2) + lane and 64 more ----------------
    if (warp >= 2) {
      const int r0 = (warp - 2) * 32 + lane;
      uint32_t use = 0;
      bool ok = true;
      for (int t = blockIdx.x; ok && t < p.num_units; t += gridDim.x) {
        int mb, nb;
        tile_coords(t, mb, nb);
        const int64_t row = (int64_t)mb * BM + r0;
        const float* sx0 = p.sx + (row < p.m ? row : 0);
        const float* sx1 = p.sx + (row + 64 < p.m ? row + 64 : 0);
        const float* sw0 = p.sw + (int64_t)nb * 2 * p.num_k_blocks;
        const float* sw1 = sw0 + ((int64_t)nb * BN + 128 < p.n ? p.num_k_blocks : 0);
        for (int kb = 0; kb < p.num_k_blocks; ++kb, ++use) {
          const float x0 = __ldg(sx0 + (int64_t)kb * p.m), x1 = __ldg(sx1 + (int64_t)kb * p.m);
          const float w0 = __ldg(sw0 + kb), w1 = __ldg(sw1 + kb);
          const int acc = use & 1;
          ok = wait_bar(cb, smem_u32(&cb->tmem_empty[acc]), ((use >> 1) & 1) ^ 1u, p.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          float* to = scales + acc * 2 * BM + r0;
          to[0] = x0 * w0;
          to[64] = x1 * w0;
          to[BM] = x0 * w1;
          to[BM + 64] = x1 * w1;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&cb->tmem_full[acc]));
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(F_REGS_HIGH));
    // ---------------- epilogue: one row of 128 columns to a thread ----------------
    const int sub = warp & 3, ew = warp - 4;
    const int grp = ew >> 2;
    uint32_t use = 0;
    bool ok = true;
    uint8_t* srow0 = stg + ew * F_OUT_BYTES;
    const uint32_t tsub = tmem_base + ((uint32_t)(sub * 32) << 16) + grp * 128;
    uint32_t ra[32], rb[32];  // two loads take turns: one in flight while the other is added
    auto full = [&]() {
      ok = wait_bar(cb, smem_u32(&cb->tmem_full[use % F_ACCS]), (use / F_ACCS) & 1u, p.status);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
    };
    auto hand_back = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&cb->tmem_empty[use % F_ACCS]));
      ++use;
    };
    for (int t = blockIdx.x; ok && t < p.num_units; t += gridDim.x) {
      int mb, nb;
      tile_coords(t, mb, nb);
      const int64_t row0 = (int64_t)mb * BM + sub * 32;
      const int64_t col0 = (int64_t)nb * BN + grp * 128;
      const bool live = row0 < p.m && col0 < p.n;  // of this warp
      if (!live) {
        for (int kb = 0; ok && kb < p.num_k_blocks; ++kb) {
          full();
          if (ok) hand_back();
        }
        continue;
      }
      float2 sum[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) sum[i] = make_float2(0.f, 0.f);
      const int last = p.num_k_blocks - 1;
      full();
      if (!ok) break;
      ld_start(tsub + (use % F_ACCS) * ACC_COLS, ra);
      for (int kb = 0; kb <= last; ++kb) {
        const uint32_t ta = tsub + (use % F_ACCS) * ACC_COLS;
        const float s = scales[((use % F_ACCS) * 2 + grp) * BM + sub * 32 + lane];
        ld_wait(ra);
        ld_start(ta + 32, rb);
        add32(sum, ra, s);
        ld_wait(rb);
        ld_start(ta + 64, ra);
        add32(sum + 16, rb, s);
        ld_wait(ra);
        ld_start(ta + 96, rb);
        add32(sum + 32, ra, s);
        ld_wait(rb);
        hand_back();
        if (kb < last) {
          full();
          if (!ok) break;
          ld_start(tsub + (use % F_ACCS) * ACC_COLS, ra);
        }
        add32(sum + 48, rb, s);
      }
      if (!ok) break;
      // ---- out: 64 bytes of a row at a time through shared memory ----
#pragma unroll
      for (int c = 0; c < 128 / COLS; ++c) {
        const int64_t cc = col0 + c * COLS;
        if (cc >= p.n) break;
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
        uint4* srow = reinterpret_cast<uint4*>(srow0 + lane * 64);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2* q = sum + (c * COLS + u * (COLS / 4)) / 2;
          if (sizeof(T) == 2)
            srow[u] = make_uint4(pack_bf16(q[0].x, q[0].y), pack_bf16(q[1].x, q[1].y),
                                 pack_bf16(q[2].x, q[2].y), pack_bf16(q[3].x, q[3].y));
          else
            srow[u] = make_uint4(__float_as_uint(q[0].x), __float_as_uint(q[0].y),
                                 __float_as_uint(q[1].x), __float_as_uint(q[1].y));
        }
        if (p.use_tma) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tmO, smem_u32(srow0), (int32_t)cc, (int32_t)row0);
            bulk_commit();
          }
        } else {
          // rows of any alignment: one element a lane, 32 / COLS rows at a time
          __syncwarp();
          const int rows = (int)min((int64_t)32, p.m - row0);
          const int e = lane % COLS;
          if (cc + e < p.n)
            for (int r = lane / COLS; r < rows; r += 32 / COLS)
              reinterpret_cast<T*>(p.out)[(row0 + r) * p.ldo + cc + e] =
                  reinterpret_cast<const T*>(srow0 + r * 64)[e];
          __syncwarp();
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc<false>(tmem_base, TMEM_COLS);
  }
}

__device__ __forceinline__ float val(const float* p) { return *p; }
__device__ __forceinline__ float val(const __nv_bfloat16* p) { return __bfloat162float(*p); }

constexpr float kAmaxFloor = 0x1p-100f;

__device__ __forceinline__ uint32_t code4(const float (&x)[4], float inv) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(x[0], inv), __fmul_rn(x[1], inv)),
                                               __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(x[2], inv), __fmul_rn(x[3], inv)),
                                               __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Zeros from the end of a row's last block on (ldq may be any length).
__device__ __forceinline__ void zero_tail(uint8_t* row, int64_t from, int64_t ldq) {
  for (int64_t j = from; j < ldq; j += FB) *reinterpret_cast<uint32_t*>(row + j) = 0u;
}

// One warp to a 1 x 128 block, four consecutive elements a lane. `scales` is
// [blocks x rows], so that the product's threads (one row each) read it whole.
template <typename T>
__global__ void __launch_bounds__(256) k_quantise_rows(const T* x, int64_t ldx, int64_t rows,
                                                       int64_t cols, int64_t blocks, uint8_t* q,
                                                       int64_t ldq, float* scales, int* status) {
  const int lane = threadIdx.x & 31;
  let_next_launch();
  if (status && blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
  const int64_t units = rows * blocks;
  for (int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); u < units; u += (int64_t)gridDim.x * 8) {
    const int64_t r = u / blocks, b = u - r * blocks;
    const int64_t j = b * FB + lane * 4;
    const T* px = x + r * ldx + j;
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = j + e < cols ? val(px + e) : 0.f;
    float a = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    a = fmaxf(a, kAmaxFloor);
    const uint32_t c = code4(v, __fmul_rn(__frcp_rn(a), 448.f));
    if (j < ldq) *reinterpret_cast<uint32_t*>(q + r * ldq + j) = c;  // (ldq: whole 16-byte units)
    if (b == blocks - 1) zero_tail(q + r * ldq, j + FB, ldq);
    if (lane == 0) scales[b * rows + r] = __fmul_rn(a, 1.f / 448.f);
  }
}

// One CTA to a 128 x 128 block, 64 elements a thread. scales: [row blocks x blocks].
template <typename T>
__global__ void __launch_bounds__(256) k_quantise_blocks(const T* x, int64_t ldx, int64_t rows,
                                                         int64_t cols, int64_t blocks, uint8_t* q,
                                                         int64_t ldq, float* scales) {
  __shared__ float sh[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t rb = blockIdx.x / blocks, b = blockIdx.x - rb * blocks;
  const int64_t j = b * FB + lane * 4;
  float v[16][4];
  float a = kAmaxFloor;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t r = rb * FB + i * 8 + warp;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[i][e] = r < rows && j + e < cols ? val(x + r * ldx + j + e) : 0.f;
      a = fmaxf(a, fabsf(v[i][e]));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  if (lane == 0) sh[warp] = a;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) a = fmaxf(a, sh[w]);
  const float inv = __fmul_rn(__frcp_rn(a), 448.f);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t r = rb * FB + i * 8 + warp;
    if (r < rows && j < ldq) *reinterpret_cast<uint32_t*>(q + r * ldq + j) = code4(v[i], inv);
    if (r < rows && b == blocks - 1) zero_tail(q + r * ldq, j + FB, ldq);
  }
  if (threadIdx.x == 0) scales[blockIdx.x] = __fmul_rn(a, 1.f / 448.f);
}

inline bool aligned(const void* q, uintptr_t a) { return ((uintptr_t)q & (a - 1)) == 0; }
inline size_t dsize(int dt) { return dt == FLJSD_BF16 ? 2 : 4; }
inline size_t align_up(size_t x) { return (x + 255) / 256 * 256; }
inline int64_t up(int64_t x, int64_t q) { return (x + q - 1) / q * q; }

bool known(int dt) { return dt == FLJSD_F32 || dt == FLJSD_BF16; }

cudaError_t quantise(int64_t rows, int64_t cols, int dtype, int block_rows, const void* x,
                     int64_t ldx, void* codes, int64_t ldq, float* scales, int* status,
                     cudaStream_t st) {
  const int64_t blocks = (cols + FB - 1) / FB;
  auto* q = static_cast<uint8_t*>(codes);
  trace_begin(FLJSD_KERNEL_SMALL, st);
  if (block_rows == 1) {
    const int64_t need = (rows * blocks + 7) / 8, most = (int64_t)num_sms() * 32;
    const unsigned grid = (unsigned)(need < most ? need : most);
    if (dtype == FLJSD_BF16)
      k_quantise_rows<<<grid, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(x), ldx, rows, cols,
                                            blocks, q, ldq, scales, status);
    else
      k_quantise_rows<<<grid, 256, 0, st>>>(static_cast<const float*>(x), ldx, rows, cols, blocks,
                                            q, ldq, scales, status);
  } else {
    const unsigned grid = (unsigned)((rows + FB - 1) / FB * blocks);
    if (dtype == FLJSD_BF16)
      k_quantise_blocks<<<grid, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(x), ldx, rows,
                                              cols, blocks, q, ldq, scales);
    else
      k_quantise_blocks<<<grid, 256, 0, st>>>(static_cast<const float*>(x), ldx, rows, cols,
                                              blocks, q, ldq, scales);
  }
  trace_end(FLJSD_KERNEL_SMALL, st);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_product(const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mo,
                           const F8Params& p, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(k_fp8_gemm<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       F_SMEM);
  if (e != cudaSuccess) return e;
  const int grid = p.num_units < num_sms() ? p.num_units : num_sms();
  k_fp8_gemm<T><<<grid, F_THREADS, F_SMEM, st>>>(ma, mb, mo, p);
  return cudaGetLastError();
}

struct F8Layout {
  int64_t ldq, blocks;
  size_t codes, scales, total;  // the status word comes first
};
F8Layout f8_layout(int64_t m, int64_t k) {
  F8Layout L;
  L.ldq = up(k, 16);
  L.blocks = (k + FB - 1) / FB;
  L.codes = 256;
  L.scales = L.codes + align_up((size_t)m * L.ldq);
  L.total = L.scales + align_up((size_t)m * L.blocks * sizeof(float));
  return L;
}

}  // namespace
}  // namespace fljsd

using namespace fljsd;

extern "C" {

fljsd_status fljsd_fp8_quantize(int64_t rows, int64_t cols, int32_t dtype, int32_t block_rows,
                                const void* x, int64_t ldx, void* codes, int64_t ldq, float* scales,
                                fljsd_stream_t stream) {
  if (rows <= 0 || cols <= 0 || ldx < cols || ldq < cols || ldq % 16 != 0 || !known(dtype) ||
      (block_rows != 1 && block_rows != FB))
    return FLJSD_ERR_INVALID_ARG;
  if (!x || !codes || !scales || !aligned(x, dsize(dtype)) || !aligned(codes, 16) ||
      !aligned(scales, 4))
    return FLJSD_ERR_INVALID_ARG;
  if (rows > (int64_t)1 << 30 || cols > (int64_t)1 << 20) return FLJSD_ERR_UNSUPPORTED;
  if (block_rows == FB && (rows + FB - 1) / FB * ((cols + FB - 1) / FB) > 0x7fffffff)
    return FLJSD_ERR_UNSUPPORTED;
  return quantise(rows, cols, dtype, block_rows, x, ldx, codes, ldq, scales, nullptr,
                  reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FLJSD_OK
             : FLJSD_ERR_CUDA;
}

size_t fljsd_fp8_linear_workspace_bytes(int64_t m, int64_t k) {
  return m <= 0 || k <= 0 ? 0 : f8_layout(m, k).total;
}

fljsd_status fljsd_fp8_linear(int64_t m, int64_t n, int64_t k, int32_t x_dtype, const void* x,
                              int64_t ldx, const void* w_codes, int64_t ldw, const float* w_scales,
                              int32_t out_dtype, void* out, int64_t ldo, void* workspace,
                              size_t workspace_bytes, fljsd_stream_t stream) {
  if (m <= 0 || n <= 0 || k <= 0 || ldx < k || ldw < k || ldw % 16 != 0 || ldo < n ||
      !known(x_dtype) || !known(out_dtype))
    return FLJSD_ERR_INVALID_ARG;
  if (!x || !w_codes || !w_scales || !out || !workspace || !aligned(x, dsize(x_dtype)) ||
      !aligned(w_codes, 16) || !aligned(w_scales, 4) || !aligned(out, dsize(out_dtype)) ||
      !aligned(workspace, 16))
    return FLJSD_ERR_INVALID_ARG;
  if (m > (int64_t)1 << 30 || n > (int64_t)1 << 30 || k > (int64_t)1 << 20)
    return FLJSD_ERR_UNSUPPORTED;
  const F8Layout L = f8_layout(m, k);
  if (workspace_bytes < L.total) return FLJSD_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  int* status = reinterpret_cast<int*>(ws);
  float* sx = reinterpret_cast<float*>(ws + L.scales);
  F8Params p{};
  const int64_t mblocks = (m + BM - 1) / BM, nblocks = (n + BN - 1) / BN;
  if (mblocks * nblocks > 0x7fffffff) return FLJSD_ERR_UNSUPPORTED;
  p.m = m; p.n = n;
  p.num_n_blocks = (int)nblocks;
  p.num_k_blocks = (int)L.blocks;
  p.m_units = (int)mblocks;
  p.num_units = (int)(mblocks * nblocks);
  // bands of about 32 MB of x, as for bf16
  const int64_t gm = (32ll << 20) / ((int64_t)BM * k);
  p.group_m = (int)(gm < 1 ? 1 : gm > mblocks ? mblocks : gm);
  p.sx = sx; p.sw = w_scales; p.out = out; p.ldo = ldo;
  p.use_tma = aligned(out, 16) && (ldo * dsize(out_dtype)) % 16 == 0 && (n * dsize(out_dtype)) % 16 == 0;
  p.timeout_ns = kTimeoutNs;
  p.status = status;
  CUtensorMap ma, mb, mo;
  if (!make_tensor_map(&ma, MapType::kU8, ws + L.codes, k, m, L.ldq, FB, BM) ||
      !make_tensor_map(&mb, MapType::kU8, w_codes, k, n, ldw, FB, BN))
    return FLJSD_ERR_CUDA;
  mo = ma;
  const bool b16 = out_dtype == FLJSD_BF16;
  if (p.use_tma && !make_tensor_map(&mo, b16 ? MapType::kBf16 : MapType::kF32, out, n, m, ldo,
                                    b16 ? 32 : 16, 32, false))
    return FLJSD_ERR_CUDA;
  if (quantise(m, k, x_dtype, 1, x, ldx, ws + L.codes, L.ldq, sx, status, st) != cudaSuccess)
    return FLJSD_ERR_CUDA;
  // a few rows are bound by reading w: the product arranged around that
  SkinnyArgs few{1, ws + L.codes, L.ldq, w_codes, ldw, m, n, k, sx, w_scales, out, ldo,
                 out_dtype == FLJSD_BF16, status, true};
  cudaError_t e;
  trace_begin(FLJSD_KERNEL_GEMM_LOGITS, st);
  if (skinny_supported(few))
    e = launch_skinny(few, st);
  else
    e = b16 ? launch_product<__nv_bfloat16>(ma, mb, mo, p, st)
            : launch_product<float>(ma, mb, mo, p, st);
  trace_end(FLJSD_KERNEL_GEMM_LOGITS, st);
  return e == cudaSuccess ? FLJSD_OK : FLJSD_ERR_CUDA;
}

}  // extern "C"
