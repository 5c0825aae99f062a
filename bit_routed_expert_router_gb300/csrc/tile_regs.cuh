// What the 16-bit and the 8-bit grouped products share beside their primitives:
// pairs of fp32 values, 16-bit outputs, and the experts' row ranges.
#pragma once

#include "f32x2.cuh"
#include "tc16.cuh"

namespace moe {

using namespace tc16;

__device__ __forceinline__ uint32_t pack16(float lo, float hi, int bf16) {
  if (bf16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Row range of expert e: inside [0, m] whatever the offsets hold.
__device__ __forceinline__ int clamp_off(int v, int m) { return min(max(v, 0), m); }

}  // namespace moe
