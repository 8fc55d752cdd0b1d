// Tokens into the 4-bit KV cache and back (format: include/msa.h, packed_cache.cuh).
// Four lanes hold a group of 32 dims, eight dims each: the group's range is two shuffles, and a
// lane's eight codes are one 32-bit word of K's record or two 16-bit halves of V's.
#include "packed_cache.cuh"

namespace msa {

namespace {

constexpr int kThreads = 256;

// Position and cache byte address of token i of sequence b, head g; null when not stored.
template <int D>
__device__ __forceinline__ long long token_offset(const Dims& p, const int32_t* starts, int n,
                                                  int b, int g, int i, int& row) {
  const int L = seq_len_of(p, b);
  const long long pos = (starts ? (long long)starts[b] : (long long)L - n) + i;
  if (pos < 0 || pos >= L) return -1;
  const int phys = physical_block(p, b, (int)(pos / kPackedBlock));
  if (phys < 0) return -1;
  row = (int)(pos % kPackedBlock);
  return ((long long)phys * p.Hkv + g) * PackedRecord<D>::kPairBytes;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) pack_kernel(const T* __restrict__ k,
                                                        const T* __restrict__ v,
                                                        uint8_t* __restrict__ cache,
                                                        const int32_t* __restrict__ starts, int n,
                                                        Dims p) {
  using R = PackedRecord<D>;
  constexpr int kLanes = D / 8;                            // lanes of one row
  const long long rows = 2ll * p.B * p.Hkv * n;            // K's rows, then V's
  const long long e = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long row_id = e / kLanes;
  const bool there = row_id < rows;
  const bool is_v = row_id >= rows / 2;
  const long long r = is_v ? row_id - rows / 2 : row_id;
  const int i = (int)(r % n), bg = there ? (int)(r / n) : 0, b = bg / p.Hkv, g = bg % p.Hkv;
  const int lane = (int)(e % kLanes), grp = lane / 4, c = lane % 4;
  int row = 0;
  const long long at = there ? token_offset<D>(p, starts, n, b, g, i, row) : -1;
  float x[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) x[u] = 0.f;
  if (at >= 0) {
    const T* src = (is_v ? v : k) + (size_t)r * D + lane * 8;
#pragma unroll
    for (int u = 0; u < 8; u += Vec16<T>::N) Vec16<T>::load(src + u, x + u);
  }
  float hi = x[0], lo = x[0];
  int bad = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    hi = fmaxf(hi, x[u]);
    lo = fminf(lo, x[u]);
    bad |= !(fabsf(x[u]) <= 3.402823466e38f);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    bad |= __shfl_xor_sync(0xffffffffu, bad, o);
  }
  if (at < 0) return;
  float step, mid, inv;
  packed_scales(hi, lo, bad != 0, step, mid, inv);
  uint32_t w = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) w |= packed_code(x[u], mid, inv) << (4 * u);
  uint8_t* rec = cache + at + (is_v ? R::kBytes : 0);
  if (is_v) {
    *reinterpret_cast<uint16_t*>(rec + R::v_half(row, grp, 2 * c)) = (uint16_t)w;
    *reinterpret_cast<uint16_t*>(rec + R::v_half(row, grp, 2 * c + 1)) = (uint16_t)(w >> 16);
  } else {
    *reinterpret_cast<uint32_t*>(rec + R::k_word(row, grp, c)) = w;
  }
  if (c == 0) {
    *reinterpret_cast<__nv_bfloat16*>(rec + R::plane(R::kStepOffset, row, grp)) =
        __float2bfloat16_rn(step);
    *reinterpret_cast<__nv_bfloat16*>(rec + R::plane(R::kMidOffset, row, grp)) =
        __float2bfloat16_rn(mid);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) unpack_kernel(T* __restrict__ k, T* __restrict__ v,
                                                          const uint8_t* __restrict__ cache,
                                                          const int32_t* __restrict__ starts,
                                                          int n, Dims p) {
  using R = PackedRecord<D>;
  constexpr int kLanes = D / 8;
  const long long rows = 2ll * p.B * p.Hkv * n;
  const long long e = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long row_id = e / kLanes;
  if (row_id >= rows) return;
  const bool is_v = row_id >= rows / 2;
  const long long r = is_v ? row_id - rows / 2 : row_id;
  const int i = (int)(r % n), bg = (int)(r / n), b = bg / p.Hkv, g = bg % p.Hkv;
  const int lane = (int)(e % kLanes), grp = lane / 4, c = lane % 4;
  int row = 0;
  const long long at = token_offset<D>(p, starts, n, b, g, i, row);
  if (at < 0) return;
  const uint8_t* rec = cache + at + (is_v ? R::kBytes : 0);
  uint32_t w;
  if (is_v)
    w = *reinterpret_cast<const uint16_t*>(rec + R::v_half(row, grp, 2 * c)) |
        (uint32_t)*reinterpret_cast<const uint16_t*>(rec + R::v_half(row, grp, 2 * c + 1)) << 16;
  else
    w = *reinterpret_cast<const uint32_t*>(rec + R::k_word(row, grp, c));
  const float step = load_bf16(rec + R::plane(R::kStepOffset, row, grp));
  const float mid = load_bf16(rec + R::plane(R::kMidOffset, row, grp));
  T* dst = (is_v ? v : k) + (size_t)r * D + lane * 8;
#pragma unroll
  for (int u = 0; u < 8; ++u) dst[u] = from_f32<T>(packed_value((w >> (4 * u)) & 15u, step, mid));
}

template <typename T, int D>
cudaError_t pack(const Dims& p, int n, const int32_t* starts, const void* k, const void* v,
                 void* cache, cudaStream_t st) {
  const long long lanes = 2ll * p.B * p.Hkv * n * (D / 8);
  const long long grid = (lanes + kThreads - 1) / kThreads;
  if (grid > 2147483647ll) return cudaErrorInvalidConfiguration;
  pack_kernel<T, D><<<(unsigned)grid, kThreads, 0, st>>>((const T*)k, (const T*)v,
                                                         (uint8_t*)cache, starts, n, p);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t unpack(const Dims& p, int n, const int32_t* starts, const void* cache, void* k,
                   void* v, cudaStream_t st) {
  const long long lanes = 2ll * p.B * p.Hkv * n * (D / 8);
  const long long grid = (lanes + kThreads - 1) / kThreads;
  if (grid > 2147483647ll) return cudaErrorInvalidConfiguration;
  unpack_kernel<T, D><<<(unsigned)grid, kThreads, 0, st>>>((T*)k, (T*)v, (const uint8_t*)cache,
                                                           starts, n, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_pack(const Dims& p, int n, const int32_t* starts, const void* k,
                              const void* v, void* cache, cudaStream_t st) {
  if (p.dtype == 1)
    return p.d == 128 ? pack<__nv_bfloat16, 128>(p, n, starts, k, v, cache, st)
                      : pack<__nv_bfloat16, 64>(p, n, starts, k, v, cache, st);
  return p.d == 128 ? pack<float, 128>(p, n, starts, k, v, cache, st)
                    : pack<float, 64>(p, n, starts, k, v, cache, st);
}

cudaError_t launch_cache_unpack(const Dims& p, int n, const int32_t* starts, const void* cache,
                                void* k, void* v, cudaStream_t st) {
  if (p.dtype == 1)
    return p.d == 128 ? unpack<__nv_bfloat16, 128>(p, n, starts, cache, k, v, st)
                      : unpack<__nv_bfloat16, 64>(p, n, starts, cache, k, v, st);
  return p.d == 128 ? unpack<float, 128>(p, n, starts, cache, k, v, st)
                    : unpack<float, 64>(p, n, starts, cache, k, v, st);
}

}  // namespace msa
