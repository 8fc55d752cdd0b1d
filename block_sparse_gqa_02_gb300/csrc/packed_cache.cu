// Tokens into the 4-bit KV cache and back (format: include/msa.h, packed_cache.cuh).
//
// CTA = the tokens of one call that fall into K's or V's record of one block and head.  Four
// lanes hold a group of 32 dims, eight dims each: the group's range is two shuffles, and a
// lane's eight codes are one 32-bit word of K's record or two 16-bit halves of V's.  Both
// kernels stream, so HBM bounds them; V's halves lie 8 D bytes apart, so the record goes
// through shared memory: a block that is filled whole leaves it in 16-byte stores, of any other
// only the stored tokens' bytes are written.  Unpacking stages the record when it needs a
// quarter of it or more, and reads a few tokens' bytes where they are.
#include "packed_cache.cuh"

namespace msa {

namespace {

constexpr int kThreads = 256;
constexpr int kStageRows = 32;         // rows of a block from which unpacking stages it

// What a CTA works on: rows [lo, hi) of a block are the call's tokens first .. first + hi - lo - 1
// of (b, g); record is null when there are none.
struct Part {
  uint8_t* record;
  int lo, hi;
  long long token;                     // row of k, v [B, Hkv, n] of the block's row lo
};

template <int D>
__device__ __forceinline__ Part part_of(const Dims& p, const int32_t* starts, int n, int per_seq,
                                        uint8_t* cache, bool& is_v) {
  Part r = {nullptr, 0, 0, 0};
  int e = blockIdx.x;
  const int x = e % per_seq;
  e /= per_seq;
  is_v = e & 1;
  const int bg = e >> 1, b = bg / p.Hkv, g = bg % p.Hkv;
  const int L = seq_len_of(p, b);
  const long long start = starts ? (long long)starts[b] : (long long)L - n;
  const long long from = start > 0 ? start : 0;
  const long long to = start + n < L ? start + n : L;
  const long long blk = from / kPackedBlock + x;
  const long long p0 = blk * kPackedBlock;
  const long long lo = from > p0 ? from : p0, hi = to < p0 + kPackedBlock ? to : p0 + kPackedBlock;
  if (lo >= hi) return r;                                  // blk is a block of the sequence here
  const int phys = physical_block(p, b, (int)blk);
  if (phys < 0) return r;
  r.record = cache + ((size_t)phys * p.Hkv + g) * PackedRecord<D>::kPairBytes +
             (is_v ? PackedRecord<D>::kBytes : 0);
  r.lo = (int)(lo - p0);
  r.hi = (int)(hi - p0);
  r.token = (long long)bg * n + (lo - start);
  return r;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) pack_kernel(const T* __restrict__ k,
                                                        const T* __restrict__ v,
                                                        uint8_t* __restrict__ cache,
                                                        const int32_t* __restrict__ starts, int n,
                                                        int per_seq, Dims p) {
  using R = PackedRecord<D>;
  constexpr int kLanes = D / 8;                            // lanes of one row
  constexpr int kRowsAtOnce = kThreads / kLanes;
  __shared__ __align__(16) uint8_t image[R::kBytes];
  bool is_v;
  const Part part = part_of<D>(p, starts, n, per_seq, cache, is_v);
  if (!part.record) return;
  const int lane = threadIdx.x % kLanes, grp = lane / 4, c = lane % 4;
  const T* src = is_v ? v : k;
  // whole warps go round together: the shuffles need all lanes
  for (int r0 = part.lo; r0 < part.hi; r0 += kRowsAtOnce) {
    const int row = r0 + (int)threadIdx.x / kLanes;
    const bool there = row < part.hi;
    float x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = 0.f;
    if (there) {
      const T* s = src + (size_t)(part.token + row - part.lo) * D + lane * 8;
#pragma unroll
      for (int u = 0; u < 8; u += Vec16<T>::N) Vec16<T>::load(s + u, x + u);
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
    if (!there) continue;
    float step, mid, inv;
    packed_scales(hi, lo, bad != 0, step, mid, inv);
    uint32_t w = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) w |= packed_code(x[u], mid, inv) << (4 * u);
    if (is_v) {
      *reinterpret_cast<uint16_t*>(image + R::v_half(row, grp, 2 * c)) = (uint16_t)w;
      *reinterpret_cast<uint16_t*>(image + R::v_half(row, grp, 2 * c + 1)) = (uint16_t)(w >> 16);
    } else {
      *reinterpret_cast<uint32_t*>(image + R::k_word(row, grp, c)) = w;
    }
    if (c < 2)
      *reinterpret_cast<__nv_bfloat16*>(
          image + R::plane(c ? R::kMidOffset : R::kStepOffset, row, grp)) =
          __float2bfloat16_rn(c ? mid : step);
  }
  __syncthreads();
  if (part.hi - part.lo == kPackedBlock) {
    for (int e = threadIdx.x; e < R::kBytes / 16; e += kThreads)
      reinterpret_cast<uint4*>(part.record)[e] = reinterpret_cast<const uint4*>(image)[e];
    return;
  }
  // only the bytes of rows [lo, hi)
  const int rows = part.hi - part.lo;
  if (is_v) {
    constexpr int kUnit = 2 * R::kGroups;                  // codes of one key and r
    for (int e = threadIdx.x; e < rows * 8; e += kThreads) {
      const int at = R::v_half(part.lo + e / 8, 0, e % 8);
#pragma unroll
      for (int u = 0; u < kUnit; u += 4)
        *reinterpret_cast<uint32_t*>(part.record + at + u) =
            *reinterpret_cast<const uint32_t*>(image + at + u);
    }
  } else {
    for (int e = threadIdx.x; e < rows * (D / 32); e += kThreads) {
      const int at = part.lo * (D / 2) + e * 16;
      *reinterpret_cast<uint4*>(part.record + at) = *reinterpret_cast<const uint4*>(image + at);
    }
  }
  for (int e = threadIdx.x; e < rows * 2 * R::kGroups; e += kThreads) {
    const int at = R::plane(R::kStepOffset, part.lo + e % rows, e / rows);   // mids follow steps
    *reinterpret_cast<uint16_t*>(part.record + at) =
        *reinterpret_cast<const uint16_t*>(image + at);
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* dst, const float* x);
template <>
__device__ __forceinline__ void store8<float>(float* dst, const float* x) {
  reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* dst, const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) unpack_kernel(T* __restrict__ k, T* __restrict__ v,
                                                          const uint8_t* __restrict__ cache,
                                                          const int32_t* __restrict__ starts,
                                                          int n, int per_seq, Dims p) {
  using R = PackedRecord<D>;
  constexpr int kLanes = D / 8;
  constexpr int kRowsAtOnce = kThreads / kLanes;
  __shared__ __align__(16) uint8_t image[R::kBytes];
  bool is_v;
  const Part part = part_of<D>(p, starts, n, per_seq, const_cast<uint8_t*>(cache), is_v);
  if (!part.record) return;
  const uint8_t* rec = part.record;
  if (part.hi - part.lo >= kStageRows) {
    for (int e = threadIdx.x; e < R::kBytes / 16; e += kThreads)
      reinterpret_cast<uint4*>(image)[e] = reinterpret_cast<const uint4*>(rec)[e];
    __syncthreads();
    rec = image;
  }
  const int lane = threadIdx.x % kLanes, grp = lane / 4, c = lane % 4;
  for (int row = part.lo + (int)threadIdx.x / kLanes; row < part.hi; row += kRowsAtOnce) {
    uint32_t w;
    if (is_v)
      w = *reinterpret_cast<const uint16_t*>(rec + R::v_half(row, grp, 2 * c)) |
          (uint32_t)*reinterpret_cast<const uint16_t*>(rec + R::v_half(row, grp, 2 * c + 1)) << 16;
    else
      w = *reinterpret_cast<const uint32_t*>(rec + R::k_word(row, grp, c));
    const float step = load_bf16(rec + R::plane(R::kStepOffset, row, grp));
    const float mid = load_bf16(rec + R::plane(R::kMidOffset, row, grp));
    float x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = packed_value((w >> (4 * u)) & 15u, step, mid);
    store8<T>((is_v ? v : k) + (size_t)(part.token + row - part.lo) * D + lane * 8, x);
  }
}

// CTAs of a call: n tokens touch at most that many blocks of a sequence.
long long grid_of(const Dims& p, int n, int& per_seq) {
  per_seq = (int)(((long long)n + 126) / kPackedBlock + 1);
  if (per_seq > p.nB) per_seq = p.nB;
  return 2ll * p.B * p.Hkv * per_seq;
}

template <typename T, int D>
cudaError_t pack(const Dims& p, int n, const int32_t* starts, const void* k, const void* v,
                 void* cache, cudaStream_t st) {
  int per_seq;
  const long long grid = grid_of(p, n, per_seq);
  if (grid > 2147483647ll) return cudaErrorInvalidConfiguration;
  pack_kernel<T, D><<<(unsigned)grid, kThreads, 0, st>>>((const T*)k, (const T*)v,
                                                         (uint8_t*)cache, starts, n, per_seq, p);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t unpack(const Dims& p, int n, const int32_t* starts, const void* cache, void* k,
                   void* v, cudaStream_t st) {
  int per_seq;
  const long long grid = grid_of(p, n, per_seq);
  if (grid > 2147483647ll) return cudaErrorInvalidConfiguration;
  unpack_kernel<T, D><<<(unsigned)grid, kThreads, 0, st>>>((T*)k, (T*)v, (const uint8_t*)cache,
                                                           starts, n, per_seq, p);
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
