// rounded.cuh -- fp32 operations that are rounded each by itself, two at a time.
#pragma once

#include "lm_common.cuh"

namespace rcc {
namespace lm {

// Sums of products, each rounded, as a product with a 1 that the compiler does not
// see: ptxas (13.0) makes one fused operation of a packed product and a packed sum,
// although each has its rounding written to it.
__device__ __forceinline__ float2 sum2(float2 a, float2 b, float one) {
  return fma2(a, both(one), b);
}

__device__ __forceinline__ float inverse_root_of(float v) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float inverse_of(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Roots and quotients, correctly rounded, two at a time: a first value by an
// approximate inverse is put right by its remainder, which a fused operation gives
// exactly (P. Markstein, IBM J. Res. Dev. 34, 1990).  The scaling keeps the remainders
// of the smallest values out of the underflow.
//   root2, 0 <= v <= kMostSquare: the bits of __fsqrt_rn for every one of them, tried
//   one by one.
//   quotient2, 2^64 m / b for |m| <= kMost and kLeastBelow <= b <= 2^24: r = 1 / b to
//   the nearest (tried for every b), a quotient within one last place after the first
//   remainder; Markstein's theorem has it that the second one makes it the nearest.
// An AdamW step of 544 M elements in 8-bit states: 1,754 us; 2,092 with __fsqrt_rn and
// __fdiv_rn.
constexpr float kMostSquare = 0x1p30f, kMost = 0x1p10f, kLeastBelow = 0x1p-50f;
__device__ __forceinline__ float2 root2(float2 v) {
  const float2 x = mul2(v, both(0x1p64f)), neg_x = mul2(v, both(-0x1p64f));
  const float2 y = make_float2(inverse_root_of(fmaxf(x.x, 0x1p-96f)),
                               inverse_root_of(fmaxf(x.y, 0x1p-96f)));
  float2 s = mul2(x, y);
  s = fma2(fma2(s, s, neg_x), mul2(y, both(-0.5f)), s);
  return mul2(s, both(0x1p-32f));
}
__device__ __forceinline__ float2 quotient2(float2 m, float2 b) {
  float2 r = make_float2(inverse_of(-b.x), inverse_of(-b.y));  // -1 / b
  r = fma2(r, fma2(b, r, both(1.f)), r);
  const float2 neg_m = mul2(m, both(-0x1p64f));
  float2 q = mul2(neg_m, r);
  q = fma2(fma2(b, q, neg_m), r, q);
  return fma2(fma2(b, q, neg_m), r, q);
}

}  // namespace lm
}  // namespace rcc
