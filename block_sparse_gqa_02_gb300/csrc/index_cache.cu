// Index keys into the 8-bit cache and back (format: include/msa.h, index_cache.cuh).
//
// A row is quantised by dI / 8 lanes, eight values each: 16-byte loads of bf16, 8-byte stores of
// codes, the largest magnitude by shuffles.  The scale is a power of two, so scaling is exact, a
// code is the nearest of 8 bits to the value itself, and what the cache holds has four
// significant bits: a bf16 value again without a further rounding.  Both kernels stream: four prompts
// of 128K tokens and fewer (425,984 rows of 128) are packed in 36 us (4.5 TB/s) and read back in 25
// (6.4 TB/s).  Twice the rows a thread, half of them, and resident CTAs that load the next rows while
// they quantise were all slower (86, 72 and 70 us for the pair, against 64 cold).
#include "index_cache.cuh"
#include "launch.cuh"
#include "ptx.cuh"

namespace msa {

namespace {

constexpr int kThreads = 256;
constexpr int kFlight = 4;             // rows of a thread, their loads in flight together

template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* x) {
    w = __ldcs(reinterpret_cast<const uint4*>(x));
  }
  __device__ __forceinline__ void get(float* o) const {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = __uint_as_float(v[i] << 16);
      o[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float* o) {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
      v[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    w = make_uint4(v[0], v[1], v[2], v[3]);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* x) const {
    __stcs(reinterpret_cast<uint4*>(x), w);
  }
};
template <> struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* x) {
    a = __ldcs(reinterpret_cast<const float4*>(x));
    b = __ldcs(reinterpret_cast<const float4*>(x) + 1);
  }
  __device__ __forceinline__ void get(float* o) const {
    o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
    o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
  }
  __device__ __forceinline__ void set(const float* o) {
    a = make_float4(o[0], o[1], o[2], o[3]);
    b = make_float4(o[4], o[5], o[6], o[7]);
  }
  __device__ __forceinline__ void store(float* x) const {
    __stcs(reinterpret_cast<float4*>(x), a);
    __stcs(reinterpret_cast<float4*>(x) + 1, b);
  }
};

// Position of token i of a call, or -1 when it is not one of the sequence's.
__device__ __forceinline__ long long token_pos(long long start, int i, int L) {
  const long long pos = start + i;
  return pos >= 0 && pos < L ? pos : -1;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
index_pack_kernel(const T* __restrict__ x, const int32_t* __restrict__ starts,
                  uint8_t* __restrict__ cache, Dims p, int n, int per_seq) {
  constexpr int kLanes = D / 8, kRows = kThreads / kLanes;
  ptx::grid_wait();
  ptx::launch_dependents();
  const int b = blockIdx.x / per_seq, part = blockIdx.x % per_seq;
  const int L = seq_len_of(p, b), sub = threadIdx.x % kLanes;
  const long long start = starts ? (long long)starts[b] : (long long)L - n;
  const int i0 = part * kRows * kFlight + threadIdx.x / kLanes;
  Eight<T> v[kFlight] = {};
  long long pos[kFlight];
#pragma unroll
  for (int f = 0; f < kFlight; ++f) {
    const int i = i0 + f * kRows;
    pos[f] = i < n ? token_pos(start, i, L) : -1;
    if (pos[f] >= 0) v[f].load(x + ((size_t)b * n + i) * D + sub * 8);
  }
#pragma unroll
  for (int f = 0; f < kFlight; ++f) {
    float o[8];
    v[f].get(o);
    uint32_t amax = 0;                                     // of the bits: NaN and infinity on top
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = max(amax, __float_as_uint(o[e]) & 0x7fffffffu);
#pragma unroll
    for (int s = 1; s < kLanes; s <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, s));
    if (pos[f] < 0) continue;
    const int r = (int)(pos[f] % kIndexBlock);
    const int phys = physical_index_block(p, b, (int)(pos[f] / kIndexBlock));
    if (phys < 0) continue;
    uint8_t* rec = cache + (size_t)phys * index_record(D);
    uint2 c = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);        // NaN codes of a row that is not finite
    uint32_t byte = 255;
    if (amax < 0x7f800000u) {
      byte = index_exponent(amax);
      const float inv = pow2_byte(254 - byte);
      c.x = e4m3_pair(o[0] * inv, o[1] * inv) | e4m3_pair(o[2] * inv, o[3] * inv) << 16;
      c.y = e4m3_pair(o[4] * inv, o[5] * inv) | e4m3_pair(o[6] * inv, o[7] * inv) << 16;
    }
    *reinterpret_cast<uint2*>(rec + (size_t)r * D + sub * 8) = c;
    if (sub == 0) rec[kIndexBlock * D + r] = (uint8_t)byte;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
index_unpack_kernel(const uint8_t* __restrict__ cache, const int32_t* __restrict__ starts,
                    T* __restrict__ x, Dims p, int n, int per_seq) {
  constexpr int kLanes = D / 8, kRows = kThreads / kLanes;
  ptx::grid_wait();
  ptx::launch_dependents();
  const int b = blockIdx.x / per_seq, part = blockIdx.x % per_seq;
  const int L = seq_len_of(p, b), sub = threadIdx.x % kLanes;
  const long long start = starts ? (long long)starts[b] : (long long)L - n;
  const int i0 = part * kRows * kFlight + threadIdx.x / kLanes;
  uint2 c[kFlight];
  uint32_t byte[kFlight];
  bool there[kFlight];
#pragma unroll
  for (int f = 0; f < kFlight; ++f) {
    const int i = i0 + f * kRows;
    const long long pos = i < n ? token_pos(start, i, L) : -1;
    int phys = -1;
    if (pos >= 0) phys = physical_index_block(p, b, (int)(pos / kIndexBlock));
    there[f] = phys >= 0;
    if (there[f]) {
      const uint8_t* rec = cache + (size_t)phys * index_record(D);
      const int r = (int)(pos % kIndexBlock);
      c[f] = *reinterpret_cast<const uint2*>(rec + (size_t)r * D + sub * 8);
      byte[f] = rec[kIndexBlock * D + r];
    }
  }
#pragma unroll
  for (int f = 0; f < kFlight; ++f) {
    if (!there[f]) continue;
    const float s = pow2_byte(byte[f]);
    float o[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 y = from_e4m3_pair(((e < 2 ? c[f].x : c[f].y) >> (e & 1) * 16) & 0xffffu);
      o[2 * e] = y.x * s;
      o[2 * e + 1] = y.y * s;
    }
    Eight<T> v;
    v.set(o);
    v.store(x + ((size_t)b * n + i0 + f * kRows) * D + sub * 8);
  }
}

template <typename T, int D>
cudaError_t launch_rows(const Dims& p, int n, const int32_t* starts, const void* src, void* dst,
                        bool pack, cudaStream_t st) {
  constexpr int kRows = kThreads / (D / 8) * kFlight;
  const long long per = ((long long)n + kRows - 1) / kRows;
  if (per * p.B > 2147483647ll) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)(per * p.B));
  if (pack)
    return launch_after(index_pack_kernel<T, D>, grid, kThreads, 0, 0, st, (const T*)src, starts,
                        (uint8_t*)dst, p, n, (int)per);
  return launch_after(index_unpack_kernel<T, D>, grid, kThreads, 0, 0, st, (const uint8_t*)src,
                      starts, (T*)dst, p, n, (int)per);
}

cudaError_t dispatch(const Dims& p, int n, const int32_t* starts, const void* src, void* dst,
                     bool pack, cudaStream_t st) {
  if (p.dtype == 1)
    return p.dI == 128 ? launch_rows<__nv_bfloat16, 128>(p, n, starts, src, dst, pack, st)
                       : launch_rows<__nv_bfloat16, 64>(p, n, starts, src, dst, pack, st);
  return p.dI == 128 ? launch_rows<float, 128>(p, n, starts, src, dst, pack, st)
                     : launch_rows<float, 64>(p, n, starts, src, dst, pack, st);
}

}  // namespace

cudaError_t launch_index_pack(const Dims& p, int n, const int32_t* starts, const void* x,
                              void* cache, cudaStream_t st) {
  return dispatch(p, n, starts, x, cache, true, st);
}

cudaError_t launch_index_unpack(const Dims& p, int n, const int32_t* starts, const void* cache,
                                void* x, cudaStream_t st) {
  return dispatch(p, n, starts, cache, x, false, st);
}

}  // namespace msa
