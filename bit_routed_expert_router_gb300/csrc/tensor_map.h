// Tensor maps for the TMA loads.
#pragma once

#include <atomic>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

namespace moe {

// cuTensorMapEncodeTiled, looked up through the runtime so that the library
// does not link libcuda itself (it loads on machines without a driver).
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> encode{nullptr};
  if (!encode.load(std::memory_order_acquire)) {
    cudaDriverEntryPointQueryResult q{};
    void* fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fn)
      return nullptr;
    encode.store(reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn), std::memory_order_release);
  }
  return encode.load(std::memory_order_acquire);
}

// A map over bf16 or fp16 values for tiles with 128-byte-swizzled rows of 64
// values; what a box reaches past the tensor reads as zero.
inline bool encode_tiles(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dim, const cuuint64_t* stride,
                         const cuuint32_t* box, bool bf16) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  return encode && encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                          static_cast<cuuint32_t>(rank), const_cast<void*>(base), dim, stride, box, ones,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same over bytes, in rows of 128.
inline bool encode_byte_tiles(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dim, const cuuint64_t* stride,
                              const cuuint32_t* box) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  return encode && encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dim, stride,
                          box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A map over bf16 or fp16 values for stores of 32 x 32: rows of 64 bytes in
// shared memory, swizzled over their own width.
inline bool encode_store(CUtensorMap* m, void* base, const cuuint64_t (&dim)[3], const cuuint64_t (&stride)[2], bool bf16) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  const cuuint32_t box[3] = {32, 32, 1}, ones[3] = {1, 1, 1};
  return encode && encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, base, dim,
                          stride, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                          CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace moe
