// Joining the (m, d, s) of lp.cuh, which the row kernels and the product of a few rows share.
#pragma once

#include "jsd_math.cuh"

namespace fljsd {

// (m, d, s) of two sets, each relative to its own maximum (lp.cuh); a set without a
// finite value has m = -inf and d = s = 0, or NaN where it holds one.
struct Mds {
  float m, d, s;
};
__device__ __forceinline__ Mds merge(const Mds& a, const Mds& b, float c) {
  const float m = fmaxf(a.m, b.m);
  const float ta = a.m == -INFINITY ? 0.f : __fmul_rn(a.m - m, c);
  const float tb = b.m == -INFINITY ? 0.f : __fmul_rn(b.m - m, c);
  const float fa = rowmath::ex2(ta), fb = rowmath::ex2(tb);
  // 2^t (s + d t): both vanish where 2^t does
  return Mds{m, __fmaf_rn(a.d, fa, b.d * fb),
             __fmaf_rn(fa, __fmaf_rn(a.d, fmaxf(ta, -1024.f), a.s),
                       fb * __fmaf_rn(b.d, fmaxf(tb, -1024.f), b.s))};
}
// The warp's: its maximum in one instruction (exact, so order-free), every lane's sums
// rescaled to it once and added in a fixed order.
__device__ __forceinline__ Mds warp_mds(Mds x, float c) {
  float m;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x.m));
  const float t = x.m == -INFINITY ? 0.f : __fmul_rn(x.m - m, c);
  const float f = rowmath::ex2(t);
  float2 ds = make_float2(x.d * f, f * __fmaf_rn(x.d, fmaxf(t, -1024.f), x.s));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    ds = __fadd2_rn(ds, make_float2(__shfl_xor_sync(0xffffffffu, ds.x, o),
                                    __shfl_xor_sync(0xffffffffu, ds.y, o)));
  return Mds{m, ds.x, ds.y};
}

}  // namespace fljsd
