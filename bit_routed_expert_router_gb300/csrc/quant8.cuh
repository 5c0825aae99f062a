// e4m3 values with an fp32 scale for each 128 of a row.
//
// The scale is max|v| / 448, so that the largest value lands on e4m3's largest;
// the maximum is taken as at least 2^-100, so that a group of zeros has a scale
// too.  v is multiplied by 448 / max|v| before its one rounding to e4m3, to the
// nearest, ties to even.  Both factors are products with fast reciprocals, within
// 2^-22 of the quotients (as quotients they were a third of the norm's
// instructions).  A NaN is the maximum of whatever it is with: a group with a NaN
// has the scale NaN and only NaN, one with an infinity the scale infinity, its
// finite values 0 and its infinities NaN.
#pragma once

#include "common.cuh"

namespace moe {

constexpr float kMaxE4m3 = 448.f;
constexpr float kTiny = 7.888609052210118e-31f;   // 2^-100

// The larger magnitude (top has none yet: 0); NaN if either is.
__device__ __forceinline__ float max_abs(float top, float v) {
  float r;
  asm("{\n\t.reg .f32 a;\n\tabs.f32 a, %2;\n\tmax.NaN.f32 %0, %1, a;\n\t}" : "=f"(r) : "f"(top), "f"(v));
  return r;
}

struct Scale8 {
  float scale, inverse;
};

__device__ __forceinline__ Scale8 scale8(float top) {
  top = max_abs(kTiny, top);
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(top));   // subnormal results too
  return {top * (1.f / kMaxE4m3), kMaxE4m3 * r};
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

}  // namespace moe
