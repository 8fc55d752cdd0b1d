// The 8-bit index-key cache's record of one block (include/msa.h): 128 rows of codes, then the
// rows' exponent bytes.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace msa {

constexpr int kIndexBlock = 128;       // keys of a block

__host__ __device__ constexpr size_t index_record(int dI) { return (size_t)kIndexBlock * (dI + 1); }

// Physical block of logical block blk of sequence b, or -1 when the table's entry is no block.
__device__ __forceinline__ int physical_index_block(const Dims& p, int b, int blk) {
  const int phys = p.block_table ? p.block_table[(size_t)b * p.nB + blk] : b * p.nB + blk;
  return phys >= 0 && phys < p.n_phys ? phys : -1;
}

// Exponent byte of a row from its largest magnitude (finite): the least e, at least -126, with
// magnitude <= 1.75 * 2^kTop * 2^e, plus 127: the magnitude's exponent less kTop, or less kTop - 1
// where its fraction is above 1.75.  kTop 8: 448, the largest e4m3 value; 15: 57344, the largest of e5m2.
template <int kTop = 8>
__host__ __device__ __forceinline__ uint32_t index_exponent(uint32_t amax_bits) {
  const uint32_t e = (amax_bits >> 23) + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e > kTop ? e - kTop : 1;
}

__device__ __forceinline__ float pow2_byte(uint32_t byte) { return __uint_as_float(byte << 23); }

// Two values as codes, nearest even (below 448 in magnitude here, or NaN), and back.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 from_e4m3_pair(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
  return __half22float2(__half2(h));
}

// The same with three significant bits and a wider range, 2^-16 to 57344, from and to fp16 values.
__device__ __forceinline__ uint32_t e5m2_pair(__half2 x) {
  return __nv_cvt_halfraw2_to_fp8x2(x, __NV_SATFINITE, __NV_E5M2);
}
__device__ __forceinline__ __half2 from_e5m2_pair(uint32_t codes) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E5M2));
}

}  // namespace msa
