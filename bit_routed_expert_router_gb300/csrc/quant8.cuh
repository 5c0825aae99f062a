// e4m3 values with an fp32 scale for each 128 of a row.
//
// The scale is max|v| / 448, so that the largest value lands on e4m3's largest;
// the maximum is taken as at least 2^-100, so that a group of zeros has a scale
// too.  v is multiplied by 448 / max|v| (fp32, rounded) before its one rounding
// to e4m3, to the nearest, ties to even.  Maxima are compared as bit patterns, in
// which an infinity and then a NaN lie above every number: a group with a NaN
// has the scale NaN and only NaN, one with an infinity the scale infinity, its
// finite values 0 and its infinities NaN.
#pragma once

#include "common.cuh"

namespace moe {

constexpr float kMaxE4m3 = 448.f;
constexpr uint32_t kTinyBits = 0x0D800000u;   // 2^-100

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

struct Scale8 {
  float scale, inverse;
};

__device__ __forceinline__ Scale8 scale8(uint32_t max_bits) {
  const float top = __uint_as_float(max(max_bits, kTinyBits));
  return {top / kMaxE4m3, kMaxE4m3 / top};
}

// Two values as e4m3, a in the low byte; what is past 448 is 448, NaN stays.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  return to_e4m3x2(a, b) | to_e4m3x2(c, d) << 16;
}

// Two e4m3 values (exact in fp16) as floats.
__device__ __forceinline__ float2 from_e4m3x2(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
  return make_float2(half_lo(h), half_hi(h));
}

}  // namespace moe
