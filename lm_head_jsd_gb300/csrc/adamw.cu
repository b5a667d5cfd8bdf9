// One AdamW step over many tensors in one launch, with fp32 states or 8-bit ones.
//
// Per element, each operation rounded once to fp32 (no fused multiply-add, so that
// the step is the same sequence of operations wherever it is computed):
//   g = grad * scale                    (scale: optional device scalar)
//   m = m beta1 + g (1 - beta1)
//   v = v beta2 + (g (1 - beta2)) g
//   p = p (1 - lr decay) - (m / (sqrt(v) rsqrt(1 - beta2^t) + eps)) lr / (1 - beta1^t)
// 8-bit states are e4m3 codes with one fp32 scale for 128 consecutive elements of
// a tensor: m, and the root of v (e4m3 spans 2^18 between its least and its
// greatest value; held as the root, v spans 2^36). amax = max |x| of the block,
// not below 2^-100; scale = amax (1 / 448); code = rn(x (448 (1 / amax))), each
// product and reciprocal rounded once. The step itself uses the unrounded m and v; what
// the rounding (at most 2^-4 of a value) changes is what the next step starts from.
//
// 22 bytes an element for bf16 with fp32 states, bound by HBM (525M elements 1.68 ms =
// 6.9 TB/s, what a copy reaches); 16 bytes with 8-bit states and fp32 master weights,
// 66 instructions, bound by issue (131M elements 406 us = 5.2 TB/s; the exact root and
// quotient are half of it, and have to be: a code changes where a root is off by one
// step). Every thread takes eight consecutive elements, so all its loads are in flight
// before the first is used; 16 threads share an 8-bit block. Tried and slower with
// 8-bit states: four elements a thread (402 us against 376, one tensor), the next
// chunk's loads under way while one is stepped (391), five CTAs an SM (427). The
// tensors' table is a kernel parameter: no copy to the device, nothing that must
// outlive the call. Many small tensors are bound by the host (64 tensors 39 us a step,
// 7 of them the kernel's).
#include "internal.cuh"

#include <cuda_fp8.h>

#include <cmath>

namespace fljsd {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                     // elements a thread takes
constexpr int kChunk = kThreads * kPer;     // elements a block takes at a time
constexpr int kBlock8 = 128;                // elements of an 8-bit block
constexpr float kAmaxFloor = 0x1p-100f;
constexpr float kE4m3Max = 448.f;

struct Entry {
  const void* grad;
  void* param;
  float* master;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t n;
};

// Tensors [0, count): tensor i's chunks are numbered first[i] .. first[i + 1).
template <int CAP>
struct Table {
  Entry e[CAP];
  float2 bias[CAP];  // by the tensor's own step t: {1 / sqrt(1 - beta2^t), lr / (1 - beta1^t)}
  int64_t first[CAP + 1];
  unsigned char vec[CAP];  // every pointer allows vector accesses
  int count;
};
struct Hyper {
  float b1, omb1, b2, omb2, eps, keep;
  const float* scale;
};

__device__ __forceinline__ float to_f(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float to_f(const __nv_bfloat16* p, int64_t i) {
  return __bfloat162float(p[i]);
}
__device__ __forceinline__ void put(float* p, int64_t i, float x) { p[i] = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, int64_t i, float x) {
  p[i] = __float2bfloat16_rn(x);
}
__device__ __forceinline__ void load8(const float* p, float (&o)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
  o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&o)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = __uint_as_float(w[i] << 16);
    o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&o)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(o[0], o[1], o[2], o[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(o[4], o[5], o[6], o[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&o)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Products two to an instruction, sums one by one: a packed product and a packed sum
// are contracted to one rounding, whatever their rounding mode says.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}

__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
  const __half2 h(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3));
  return __half22float2(h);
}
__device__ __forceinline__ uint32_t to_e4m3x2(float2 x) {
  return __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
}

// The block scale of 16 threads' values (eight each): {448 (1 / amax), amax (1 / 448)}.
__device__ __forceinline__ float2 block_scale(const float (&x)[8]) {
  float a = kAmaxFloor;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(x[i]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return make_float2(__fmul_rn(__frcp_rn(a), kE4m3Max), __fmul_rn(a, 1.f / kE4m3Max));
}

// Eight 8-bit states: codes in, values out, and back.
__device__ __forceinline__ void decode8(uint2 c, float s, float (&o)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = from_e4m3x2(((i < 2 ? c.x : c.y) >> (16 * (i & 1))) & 0xffffu);
    const float2 x = mul2(f, make_float2(s, s));
    o[2 * i] = x.x;
    o[2 * i + 1] = x.y;
  }
}
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = to_e4m3x2(mul2(make_float2(x[2 * i], x[2 * i + 1]), make_float2(inv, inv)));
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

template <typename P, typename G, int BITS, bool MASTER, int CAP>
__global__ void __launch_bounds__(kThreads) k_adamw(const __grid_constant__ Table<CAP> t,
                                                    const Hyper h) {
  const float scale = h.scale ? *h.scale : 1.f;
  int at = 0;  // the last tensor that starts at or before chunk c (it only rises)
  for (int64_t c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
    if (c >= t.first[at + 1])
      for (int end = t.count; end - at > 1;) {
        const int mid = (at + end) / 2;
        if (c >= t.first[mid])
          at = mid;
        else
          end = mid;
      }
    const Entry& e = t.e[at];
    const float2 bias = t.bias[at];
    const int64_t i0 = (c - t.first[at]) * kChunk + threadIdx.x * kPer;
    const int n = (int)max((int64_t)0, min((int64_t)kPer, e.n - i0));  // this thread's elements
    const bool vec = t.vec[at] && n == kPer;
    const G* gp = reinterpret_cast<const G*>(e.grad) + i0;
    P* pp = reinterpret_cast<P*>(e.param) + i0;
    float* mp32 = reinterpret_cast<float*>(e.m) + i0;
    float* vp32 = reinterpret_cast<float*>(e.v) + i0;
    uint8_t* mp8 = reinterpret_cast<uint8_t*>(e.m) + i0;
    uint8_t* vp8 = reinterpret_cast<uint8_t*>(e.v) + i0;
    float* ma = MASTER ? e.master + i0 : nullptr;
    float g[8] = {}, p[8] = {}, m[8] = {}, v[8] = {};
    if (vec) {
      load8(gp, g);
      if (MASTER) load8(ma, p); else load8(pp, p);
      if (BITS == 32) {
        load8(mp32, m);
        load8(vp32, v);
      }
    } else {
      for (int i = 0; i < n; ++i) {
        g[i] = to_f(gp, i);
        p[i] = MASTER ? ma[i] : to_f(pp, i);
        if (BITS == 32) {
          m[i] = mp32[i];
          v[i] = vp32[i];
        }
      }
    }
    if (BITS == 8) {
      uint2 cm = make_uint2(0, 0), cv = make_uint2(0, 0);
      float sm = 0.f, sv = 0.f;
      if (n > 0) {
        sm = e.m_scale[i0 / kBlock8];
        sv = e.v_scale[i0 / kBlock8];
        if (vec) {
          cm = *reinterpret_cast<const uint2*>(mp8);
          cv = *reinterpret_cast<const uint2*>(vp8);
        } else {
          for (int i = 0; i < n; ++i) {
            const uint32_t a = mp8[i], b = vp8[i];
            (i < 4 ? cm.x : cm.y) |= a << (8 * (i & 3));
            (i < 4 ? cv.x : cv.y) |= b << (8 * (i & 3));
          }
        }
      }
      decode8(cm, sm, m);
      decode8(cv, sv, v);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 r = make_float2(v[i], v[i + 1]), q = mul2(r, r);
        v[i] = q.x;
        v[i + 1] = q.y;
      }
    }
    float r[8];
    auto both = [](float x) { return make_float2(x, x); };
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 gi = mul2(make_float2(g[i], g[i + 1]), both(scale));
      const float2 mi = add2(mul2(make_float2(m[i], m[i + 1]), both(h.b1)),
                                   mul2(gi, both(h.omb1)));
      const float2 vi = add2(mul2(make_float2(v[i], v[i + 1]), both(h.b2)),
                                   mul2(mul2(gi, both(h.omb2)), gi));
      const float2 ri = make_float2(__fsqrt_rn(vi.x), __fsqrt_rn(vi.y));
      const float2 den = add2(mul2(ri, both(bias.x)), both(h.eps));
      const float2 u = make_float2(__fdiv_rn(mi.x, den.x), __fdiv_rn(mi.y, den.y));
      // (p keep) - (u step): a sum with the negated product, which rounds the same
      const float2 pi = add2(mul2(make_float2(p[i], p[i + 1]), both(h.keep)),
                                   mul2(u, both(-bias.y)));
      m[i] = mi.x; m[i + 1] = mi.y;
      v[i] = vi.x; v[i + 1] = vi.y;
      r[i] = ri.x; r[i + 1] = ri.y;
      p[i] = pi.x; p[i + 1] = pi.y;
    }
    if (vec) {
      store8(pp, p);
      if (MASTER) store8(ma, p);
      if (BITS == 32) {
        store8(mp32, m);
        store8(vp32, v);
      }
    } else {
      for (int i = 0; i < n; ++i) {
        put(pp, i, p[i]);
        if (MASTER) ma[i] = p[i];
        if (BITS == 32) {
          mp32[i] = m[i];
          vp32[i] = v[i];
        }
      }
    }
    if (BITS == 8) {
      // elements past the tensor's end were zeros and stay out of the maximum
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i >= n) m[i] = r[i] = 0.f;
      const float2 bm = block_scale(m), bv = block_scale(r);
      const uint2 cm = encode8(m, bm.x), cv = encode8(r, bv.x);
      if (vec) {
        *reinterpret_cast<uint2*>(mp8) = cm;
        *reinterpret_cast<uint2*>(vp8) = cv;
      } else {
        for (int i = 0; i < n; ++i) {
          mp8[i] = (uint8_t)((i < 4 ? cm.x : cm.y) >> (8 * (i & 3)));
          vp8[i] = (uint8_t)((i < 4 ? cv.x : cv.y) >> (8 * (i & 3)));
        }
      }
      if (n > 0 && threadIdx.x % (kBlock8 / kPer) == 0) {
        e.m_scale[i0 / kBlock8] = bm.y;
        e.v_scale[i0 / kBlock8] = bv.y;
      }
    }
  }
}

template <typename P, typename G, int BITS, bool MASTER, int CAP>
cudaError_t launch(const Table<CAP>& t, const Hyper& h, cudaStream_t st) {
  // (CTAs of one or few chunks: as they come and go, their loads and stores spread out
  // evenly; CTAs that stay walk in step. 131M bf16 elements, fp32 states: 8 CTAs an SM
  // 484 us, 64 CTAs 419 us)
  const int64_t most = (int64_t)num_sms() * 64, chunks = t.first[t.count];
  if (chunks == 0) return cudaSuccess;
  trace_begin(FLJSD_KERNEL_SMALL, st);
  k_adamw<P, G, BITS, MASTER, CAP>
      <<<(unsigned)(chunks < most ? chunks : most), kThreads, 0, st>>>(t, h);
  trace_end(FLJSD_KERNEL_SMALL, st);
  return cudaGetLastError();
}

template <typename P, typename G, int CAP>
cudaError_t launch_pg(int bits, bool master, const Table<CAP>& t, const Hyper& h, cudaStream_t st) {
  if constexpr (sizeof(P) == 2) {
    if (master)
      return bits == 8 ? launch<P, G, 8, true>(t, h, st) : launch<P, G, 32, true>(t, h, st);
  }
  return bits == 8 ? launch<P, G, 8, false>(t, h, st) : launch<P, G, 32, false>(t, h, st);
}

using bf = __nv_bfloat16;

float2 bias_of(const fljsd_adamw_options& o, int64_t step) {
  const double t = (double)step;
  return make_float2((float)(1.0 / std::sqrt(1.0 - std::pow(o.beta2, t))),
                     (float)(o.lr / (1.0 - std::pow(o.beta1, t))));
}

// Launches of up to CAP tensors each.
template <int CAP>
cudaError_t run(const fljsd_adamw_tensor* ts, const int64_t* steps, int count,
                const fljsd_adamw_options& o, const Hyper& h, cudaStream_t st) {
  Table<CAP> t;
  int64_t last = 0;  // the step of `bias` (most tensors share it)
  float2 bias{};
  for (int at = 0; at < count;) {
    t.count = 0;
    t.first[0] = 0;
    for (; at < count && t.count < CAP; ++at) {
      const fljsd_adamw_tensor& x = ts[at];
      if (x.n == 0) continue;
      const int i = t.count++;
      t.e[i] = Entry{x.grad, x.param, x.master, x.exp_avg, x.exp_avg_sq, x.exp_avg_scale,
                     x.exp_avg_sq_scale, x.n};
      const int64_t step = steps ? steps[at] : o.step;
      if (step != last) bias = bias_of(o, last = step);
      t.bias[i] = bias;
      t.first[i + 1] = t.first[i] + (x.n + kChunk - 1) / kChunk;
      uintptr_t bits = (uintptr_t)x.grad | (uintptr_t)x.param | (uintptr_t)x.master;
      const uintptr_t state = (uintptr_t)x.exp_avg | (uintptr_t)x.exp_avg_sq;
      if (o.state_bits == 32) bits |= state;
      t.vec[i] = (bits & 15u) == 0 && (state & 7u) == 0;
    }
    cudaError_t e;
    const bool p16 = o.param_dtype == FLJSD_BF16, g16 = o.grad_dtype == FLJSD_BF16;
    if (p16)
      e = g16 ? launch_pg<bf, bf, CAP>(o.state_bits, o.master, t, h, st)
              : launch_pg<bf, float, CAP>(o.state_bits, o.master, t, h, st);
    else
      e = g16 ? launch_pg<float, bf, CAP>(o.state_bits, false, t, h, st)
              : launch_pg<float, float, CAP>(o.state_bits, false, t, h, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

constexpr int kFew = 64, kMany = 400;
static_assert(sizeof(Table<kMany>) + sizeof(Hyper) <= 32764, "kernel parameters");

}  // namespace
}  // namespace fljsd

using namespace fljsd;

extern "C" fljsd_status fljsd_adamw_step(const fljsd_adamw_options* o,
                                         const fljsd_adamw_tensor* tensors, int32_t count,
                                         const float* grad_scale, fljsd_stream_t stream) {
  return fljsd_adamw_step_each(o, tensors, nullptr, count, grad_scale, stream);
}

extern "C" fljsd_status fljsd_adamw_step_each(const fljsd_adamw_options* o,
                                              const fljsd_adamw_tensor* tensors,
                                              const int64_t* steps, int32_t count,
                                              const float* grad_scale, fljsd_stream_t stream) {
  if (!o || count < 0 || (count > 0 && !tensors)) return FLJSD_ERR_INVALID_ARG;
  if ((o->param_dtype != FLJSD_F32 && o->param_dtype != FLJSD_BF16) ||
      (o->grad_dtype != FLJSD_F32 && o->grad_dtype != FLJSD_BF16))
    return FLJSD_ERR_INVALID_ARG;
  if (o->state_bits != 32 && o->state_bits != 8) return FLJSD_ERR_INVALID_ARG;
  if ((o->master != 0 && o->master != 1) || (o->master && o->param_dtype != FLJSD_BF16))
    return FLJSD_ERR_INVALID_ARG;
  if (!(o->beta1 >= 0 && o->beta1 < 1) || !(o->beta2 >= 0 && o->beta2 < 1) || !(o->eps >= 0) ||
      !std::isfinite(o->eps) || !std::isfinite(o->lr) || !std::isfinite(o->weight_decay) ||
      (!steps && o->step < 1))
    return FLJSD_ERR_INVALID_ARG;
  if ((uintptr_t)grad_scale & 3u) return FLJSD_ERR_INVALID_ARG;
  const uintptr_t pa = o->param_dtype == FLJSD_BF16 ? 1 : 3, ga = o->grad_dtype == FLJSD_BF16 ? 1 : 3;
  const uintptr_t sa = o->state_bits == 32 ? 3 : 0;
  for (int i = 0; i < count; ++i) {
    const fljsd_adamw_tensor& t = tensors[i];
    if (t.n < 0 || (steps && steps[i] < 1)) return FLJSD_ERR_INVALID_ARG;
    if (t.n == 0) continue;
    if (!t.grad || !t.param || !t.exp_avg || !t.exp_avg_sq || (o->master && !t.master) ||
        (!o->master && t.master))
      return FLJSD_ERR_INVALID_ARG;
    if (o->state_bits == 8 && (!t.exp_avg_scale || !t.exp_avg_sq_scale))
      return FLJSD_ERR_INVALID_ARG;
    if (((uintptr_t)t.param & pa) || ((uintptr_t)t.grad & ga) || ((uintptr_t)t.master & 3u) ||
        (((uintptr_t)t.exp_avg | (uintptr_t)t.exp_avg_sq) & sa) ||
        (((uintptr_t)t.exp_avg_scale | (uintptr_t)t.exp_avg_sq_scale) & 3u))
      return FLJSD_ERR_INVALID_ARG;
    if (t.n > (int64_t)1 << 40) return FLJSD_ERR_UNSUPPORTED;
  }
  Hyper h;
  h.b1 = (float)o->beta1;
  h.omb1 = (float)(1.0 - o->beta1);
  h.b2 = (float)o->beta2;
  h.omb2 = (float)(1.0 - o->beta2);
  h.eps = (float)o->eps;
  h.keep = (float)(1.0 - o->lr * o->weight_decay);
  h.scale = grad_scale;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // a smaller table is a smaller parameter block to hand over at launch
  const cudaError_t e = count <= kFew ? run<kFew>(tensors, steps, count, *o, h, st)
                                      : run<kMany>(tensors, steps, count, *o, h, st);
  return e == cudaSuccess ? FLJSD_OK : FLJSD_ERR_CUDA;
}
