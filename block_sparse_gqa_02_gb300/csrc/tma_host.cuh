// Host-side creation of TMA tensor maps (128-byte swizzle) for the tensor-core
// kernels.  The driver's encoder is fetched through the runtime, so the library does not
// link libcuda directly.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace msa {

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// A rank-`rank` tensor map of `type` (8-bit records start at odd multiples of 128 bytes, so their
// L2 fetches are of 128).  dims[0] is the innermost (contiguous) dimension;
// strides_bytes[i] is the byte stride of dimension i+1; box[] is the tile each copy moves
// (its first side must be at most 128 bytes for the 128-byte swizzle).  Out-of-range elements of a
// box read as zero.
inline cudaError_t make_tensor_map(CUtensorMapDataType type, CUtensorMap* map, const void* base,
                                   int rank, const uint64_t* dims, const uint64_t* strides_bytes,
                                   const uint32_t* box) {
  auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  cuuint64_t gd[5], gs[4];
  cuuint32_t bx[5], es[5];
  for (int i = 0; i < rank; ++i) {
    gd[i] = dims[i];
    bx[i] = box[i];
    es[i] = 1;
    if (i + 1 < rank) gs[i] = strides_bytes[i];
  }
  CUresult r = enc(map, type, (cuuint32_t)rank,
                   const_cast<void*>(base), gd, gs, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B,
                   type == CU_TENSOR_MAP_DATA_TYPE_UINT8 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                         : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

inline cudaError_t make_tensor_map_bf16(CUtensorMap* map, const void* base, int rank,
                                        const uint64_t* dims, const uint64_t* strides_bytes,
                                        const uint32_t* box) {
  return make_tensor_map(CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, map, base, rank, dims, strides_bytes, box);
}

}  // namespace msa
