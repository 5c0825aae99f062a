// What the grouped products' storing warps share: pairs of fp32 values, and
// stores of accumulator fragments.
#pragma once

#include "tc16.cuh"

namespace moe {

using namespace tc16;

// Bytes between staged rows of 64 bytes: a multiple of 16, and the 16-byte words of eight rows hit all 32 banks.
constexpr int kEpiPitch = 80;

// Two fp32 values in one register pair, and d = a b + d on both at once.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  return static_cast<uint64_t>(__float_as_uint(hi)) << 32 | __float_as_uint(lo);
}
__device__ __forceinline__ void fma_f32x2(uint64_t& d, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}

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
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 w;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at) : "memory");
  return w;
}

// The stores of one warp: 32 columns of its accumulator lanes as fragments,
// turned through the warp's own shared memory so that every lane stores 16
// bytes.  All of a tensor's fragments are staged before the first is read
// back: one warp barrier each way, and four independent loads and stores.

// 32 features x 32 columns of 16-bit values: 64 contiguous bytes of a column.
__device__ __forceinline__ void store_32x32(uint32_t buf, const float (&v)[2][16], int bf16, uint16_t* out, long long ld,
                                            int cols, int feats, int lane) {
  __syncwarp();   // earlier reads of this buffer are done
#pragma unroll
  for (int j = 0; j < 4; ++j)
    stmatrix4_trans(buf + j * 8 * kEpiPitch + (lane & 7) * kEpiPitch + (lane >> 3) * 16,
                    pack16(v[0][4 * j], v[0][4 * j + 1], bf16), pack16(v[0][4 * j + 2], v[0][4 * j + 3], bf16),
                    pack16(v[1][4 * j], v[1][4 * j + 1], bf16), pack16(v[1][4 * j + 2], v[1][4 * j + 3], bf16));
  __syncwarp();
  const int f = 8 * (lane & 3);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = 8 * j + (lane >> 2);
    const uint4 w = lds128(buf + c * kEpiPitch + (lane & 3) * 16);
    if (c < cols && f < feats) *reinterpret_cast<uint4*>(out + c * ld + f) = w;
  }
}

}  // namespace moe
