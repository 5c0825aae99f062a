// GELU and its derivative for the 16-bit operators, in fp32.
//
// With P the normal distribution function and p its density: g P(g) and
// P(g) + g p(g).  The tanh form replaces P by (1 + tanh(s)) / 2 =
// 1 / (1 + exp(-2 s)), s = c (g + 0.044715 g^3), c = sqrt(2 / pi): one
// exponential and one division (the fast ones: a few ulp of a value up to 1,
// far below a 16-bit output's step) where tanhf took the gradient of 32,768
// rows from memory-bound to 75% of the issue slots.  Past |g| = 30 the
// derivative is 0 or 1 to the last bit.
//
// The erf form takes the smaller of P(g) and P(-g) as exp(-g^2 / 2) M(|g|), so
// that it keeps its relative precision far below zero, where 1 + erf cancels (4%
// of the value at g = -5, five steps of bf16).  M, the normal tail over its
// density without the constant, is smooth and falls like 1 / |g|: a polynomial in
// t = 1 / (1 + 0.3 |g|) (the form of Hastings, Approximations for Digital
// Computers, 1955), its coefficients fitted in 64 bits by iteratively reweighted
// least squares to 1.3e-7 of M on 0 .. 13.5, where exp(-g^2 / 2) leaves fp32's
// normal range.  The exponential is the density that the slope needs.  Gradient
// of 32,768 rows 38 us (with erff 47, with erfcf 60), forward 239 (238, 253).
#pragma once

#include "common.cuh"

namespace moe {

// 1 / (1 + exp(-2 s)) and what it leaves to 1, each with its own relative precision.
__device__ __forceinline__ float2 gelu_tanh_shares(float g) {
  const float e = __expf(-2.f * 0.7978845608028654f * fabsf(g) * (1.f + 0.044715f * g * g));
  const float big = __fdividef(1.f, 1.f + e), small = e * big;
  return g < 0.f ? make_float2(small, big) : make_float2(big, small);
}

// exp(-g^2 / 2), and P(-|g|).
__device__ __forceinline__ float2 normal_tail(float g) {
  const float a = fabsf(g), e = __expf(-0.5f * a * a), t = __fdividef(1.f, fmaf(0.3f, a, 1.f));
  float m = 0.03593174f;
  m = fmaf(m, t, -0.158276007f);
  m = fmaf(m, t, 0.208206564f);
  m = fmaf(m, t, -0.055393815f);
  m = fmaf(m, t, 0.129469186f);
  m = fmaf(m, t, 0.0996375009f);
  m = fmaf(m, t, 0.120798364f);
  m = fmaf(m, t, 0.119626395f);
  return make_float2(e, e * (m * t));
}

__device__ __forceinline__ float gelu16(float g, int variant) {
  if (variant == 1) return g * gelu_tanh_shares(g).x;
  const float small = normal_tail(g).y;
  return g * (g < 0.f ? small : 1.f - small);
}

template <int kVariant>
__device__ __forceinline__ float2 gelu16_and_slope(float g) {
  if (kVariant == 1) {
    const float gc = fabsf(g) > 30.f ? copysignf(30.f, g) : g;   // a NaN stays
    const float2 q = gelu_tanh_shares(gc);
    const float slope2 = 2.f * 0.7978845608028654f * (1.f + 0.134145f * gc * gc);   // 2 s'
    return make_float2(g * q.x, q.x * (1.f + gc * q.y * slope2));
  }
  const float2 tail = normal_tail(g);
  const float share = g < 0.f ? tail.y : 1.f - tail.y;
  return make_float2(g * share, share + g * 0.3989422804014327f * tail.x);
}

}  // namespace moe
