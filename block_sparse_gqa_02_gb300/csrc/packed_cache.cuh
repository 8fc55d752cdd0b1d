// The 4-bit KV cache's record of one block and KV head (include/msa.h): where the codes, steps
// and mids of a token lie, and the quantiser.
#pragma once

#include "common.cuh"

namespace msa {

constexpr int kPackedBlock = 128;      // keys of a block
constexpr int kPackedGroup = 32;       // dims that share a step and a mid

template <int D>
struct PackedRecord {
  static constexpr int kGroups = D / kPackedGroup;
  static constexpr int kStepOffset = 64 * D;
  static constexpr int kMidOffset = 72 * D;
  static constexpr int kBytes = 80 * D;                    // K's or V's record
  static constexpr int kPairBytes = 160 * D;               // both
  // first byte of K's codes of dims 32 g + 8 c .. + 7 of key j (four bytes)
  __host__ __device__ static constexpr int k_word(int j, int g, int c) {
    return j * (D / 2) + c * 4 * kGroups + g * 4;
  }
  // first byte of V's codes of dims 32 g + 4 r .. + 3 of key j (two bytes); the exchanged key
  // pairs put the eight lanes of a shared-memory phase on different banks
  __host__ __device__ static constexpr int v_half(int j, int g, int r) {
    return (r * kPackedBlock + 2 * ((j / 2) ^ (4 * (r & (kGroups == 4 ? 1 : 3)))) + (j & 1)) * 2 *
               kGroups + g * 2;
  }
  // byte of step (kStepOffset) or mid (kMidOffset) of key j, group g
  __host__ __device__ static constexpr int plane(int base, int j, int g) {
    return base + (g * kPackedBlock + j) * 2;
  }
};

// Physical block of logical block blk of sequence b, or -1 when the table's entry is no block.
__device__ __forceinline__ int physical_block(const Dims& p, int b, int blk) {
  const int phys = p.block_table ? p.block_table[(size_t)b * p.nB + blk] : b * p.nB + blk;
  return phys >= 0 && phys < p.n_phys ? phys : -1;
}

// Step, mid and reciprocal step of a group from its largest and smallest value.  Single
// operations, each rounded to nearest, so that the result is the definition's bit for bit.
__device__ __forceinline__ void packed_scales(float hi, float lo, bool bad, float& step,
                                              float& mid, float& inv) {
  constexpr float kFifteenth = (float)(1.0 / 15.0);
  step = __fsub_rn(__fmul_rn(hi, kFifteenth), __fmul_rn(lo, kFifteenth));
  step = __bfloat162float(__float2bfloat16_rn(step));
  if (!(step >= 0x1p-100f)) step = 0.f;
  mid = __bfloat162float(__float2bfloat16_rn(__fadd_rn(lo, 8.f * step)));
  inv = step > 0.f ? __frcp_rn(step) : 0.f;
  if (bad) {
    step = inv = 0.f;
    mid = __int_as_float(0x7fc00000);
  }
}

__device__ __forceinline__ float packed_value(uint32_t code, float step, float mid) {
  return fmaf((float)((int)code - 8), step, mid);
}

__device__ __forceinline__ float load_bf16(const uint8_t* p) {
  return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16);
}

}  // namespace msa
