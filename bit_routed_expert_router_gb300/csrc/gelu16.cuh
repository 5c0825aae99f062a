// GELU and its derivative for the 16-bit operators, in fp32.
//
// With P the normal distribution function and p its density: g P(g) and
// P(g) + g p(g).  The tanh form replaces P by (1 + tanh(s)) / 2 =
// 1 / (1 + exp(-2 s)), s = c (g + 0.044715 g^3), c = sqrt(2 / pi): one
// exponential and one division (the fast ones: a few ulp of a value up to 1,
// far below a 16-bit output's step) where tanhf took the gradient of 32,768
// rows from memory-bound to 75% of the issue slots.  Past |g| = 30 the
// derivative is 0 or 1 to the last bit.
#pragma once

#include "common.cuh"

namespace moe {

// 1 / (1 + exp(-2 s)) and what it leaves to 1, each with its own relative precision.
__device__ __forceinline__ float2 gelu_tanh_shares(float g) {
  const float e = __expf(-2.f * 0.7978845608028654f * fabsf(g) * (1.f + 0.044715f * g * g));
  const float big = __fdividef(1.f, 1.f + e), small = e * big;
  return g < 0.f ? make_float2(small, big) : make_float2(big, small);
}

__device__ __forceinline__ float gelu16(float g, int variant) {
  if (variant == 1) return g * gelu_tanh_shares(g).x;
  return 0.5f * g * (1.f + erff(g * 0.7071067811865476f));
}

template <int kVariant>
__device__ __forceinline__ float2 gelu16_and_slope(float g) {
  if (kVariant == 1) {
    const float gc = fabsf(g) > 30.f ? copysignf(30.f, g) : g;   // a NaN stays
    const float2 q = gelu_tanh_shares(gc);
    const float slope2 = 2.f * 0.7978845608028654f * (1.f + 0.134145f * gc * gc);   // 2 s'
    return make_float2(g * q.x, q.x * (1.f + gc * q.y * slope2));
  }
  const float half = 0.5f + 0.5f * erff(g * 0.7071067811865476f);
  return make_float2(g * half, half + g * 0.3989422804014327f * __expf(-0.5f * g * g));
}

}  // namespace moe
