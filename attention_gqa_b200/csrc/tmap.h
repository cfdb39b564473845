// Host-side construction of TMA tensor maps (CUtensorMap) for bf16 tensors.
//
// The driver entry point is looked up through the runtime, so the library
// links only against cudart.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace gqa {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_tiled_fn() {
  static EncodeTiledFn fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  }
  return fn;
}

// 4-D tensor map, dims innermost first, strides in bytes for dims 1..3, zero
// fill out of bounds. Returns false when the driver rejects the description.
inline bool make_tmap_4d(CUtensorMap* map, CUtensorMapDataType type, CUtensorMapSwizzle swizzle,
                         const void* base, const uint64_t dims[4],
                         const uint64_t strides_bytes[3], const uint32_t box[4]) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  cuuint64_t gdim[4] = {dims[0], dims[1], dims[2], dims[3]};
  cuuint64_t gstr[3] = {strides_bytes[0], strides_bytes[1], strides_bytes[2]};
  cuuint32_t bdim[4] = {box[0], box[1], box[2], box[3]};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(map, type, 4, const_cast<void*>(base), gdim, gstr, bdim, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// bf16 with the 128-byte swizzle (the innermost box extent must be 64 elements).
inline bool make_tmap_bf16_4d(CUtensorMap* map, const void* base, const uint64_t dims[4],
                              const uint64_t strides_bytes[3], const uint32_t box[4]) {
  return make_tmap_4d(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, base,
                      dims, strides_bytes, box);
}

// Bytes with the 64-byte swizzle (the innermost box extent must be 64 elements).
inline bool make_tmap_u8_4d(CUtensorMap* map, const void* base, const uint64_t dims[4],
                            const uint64_t strides_bytes[3], const uint32_t box[4]) {
  return make_tmap_4d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_64B, base, dims,
                      strides_bytes, box);
}

}  // namespace gqa
