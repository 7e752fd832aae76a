// Tensor maps of paged caches for the TMA engine (host side).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace tki {

// The driver's encoder, looked up once; null where the driver has none.
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();  // nobody's launch error
      return nullptr;
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// A map of a tensor of `rank` dimensions (innermost first, contiguous; strides
// of the others in elements of `size` bytes) in boxes of 128 bytes by `rows`
// by the further extents, written with the 128-byte swizzle; what lies outside
// the tensor reads as zeros. False where the engine cannot do it.
inline bool box_map(CUtensorMap* map, CUtensorMapDataType type, int size, const void* base, int rank, const int64_t* extents,
                    const int64_t* strides, const int* box_rows) {
  const auto encode = tensor_map_encoder();
  if (encode == nullptr || (reinterpret_cast<uintptr_t>(base) & 15) != 0) return false;
  cuuint64_t dims[4], bytes[3];
  cuuint32_t box[4], steps[4];
  for (int i = 0; i < rank; ++i) {
    if (extents[i] < 1 || extents[i] > INT32_MAX) return false;
    dims[i] = static_cast<cuuint64_t>(extents[i]);
    box[i] = i == 0 ? static_cast<cuuint32_t>(128 / size) : static_cast<cuuint32_t>(box_rows[i - 1]);
    steps[i] = 1;
    if (i == 0) continue;
    const int64_t stride = extents[i] == 1 ? 16 / size : strides[i - 1];  // of one: never used
    if (stride <= 0 || stride * size % 16 != 0 || stride >= (int64_t{1} << 40) / size) return false;
    bytes[i - 1] = static_cast<cuuint64_t>(stride) * size;
  }
  return encode(map, type, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, bytes, box, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tki
