// Tokens into the 4-bit KV cache and back (format: include/msa.h, packed_cache.cuh).
//
// CTA = the tokens of one call that fall into K's or V's record of one block and head.  Both
// kernels stream, so HBM should bound them; what they cost is instructions, so packing gives a
// thread a whole group of 32 dims (its range needs no shuffles, its scales are formed once) and
// unpacking works on pairs of bf16.  V's 16-bit halves lie 16 D bytes apart, so the record goes
// through shared memory: a block that is filled whole leaves it in 16-byte stores, of any other
// only the stored tokens' bytes are written.  Unpacking stages the record when it needs a
// quarter of it or more, and reads a few tokens' bytes where they are.  Measured: two prompts of
// 32768 and 24576 tokens, 4 heads of 128 dims, are packed and unpacked in 56 us (308 MB, 5.5
// TB/s); both are bound by their instructions (issue slots 78 % and 61 % used).
#include "launch.cuh"
#include "packed_cache.cuh"
#include "ptx.cuh"

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
  ptx::grid_wait();
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

// The 32 values of a group, and its largest and smallest (NaN if there is one).
template <typename T> struct GroupLoad;
template <> struct GroupLoad<__nv_bfloat16> {
  uint4 w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ static __nv_bfloat162 pair(uint32_t x) {
    return *reinterpret_cast<const __nv_bfloat162*>(&x);
  }
  __device__ __forceinline__ void range(float& hi, float& lo) const {
    __nv_bfloat162 h = pair(w[0].x), l = h;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h = __hmax2_nan(__hmax2_nan(h, pair(w[i].x)), __hmax2_nan(pair(w[i].y), pair(w[i].z)));
      l = __hmin2_nan(__hmin2_nan(l, pair(w[i].x)), __hmin2_nan(pair(w[i].y), pair(w[i].z)));
      h = __hmax2_nan(h, pair(w[i].w));
      l = __hmin2_nan(l, pair(w[i].w));
    }
    hi = __bfloat162float(__hmax_nan(h.x, h.y));
    lo = __bfloat162float(__hmin_nan(l.x, l.y));
  }
  // values 8 c .. 8 c + 7
  __device__ __forceinline__ void eight(int c, float* x) const {
    const uint32_t v[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(v[i] << 16);
      x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  }
};
template <> struct GroupLoad<float> {
  float4 w[8];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = reinterpret_cast<const float4*>(p)[i];
  }
  __device__ __forceinline__ static float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
  }
  __device__ __forceinline__ static float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
  }
  __device__ __forceinline__ void range(float& hi, float& lo) const {
    hi = lo = w[0].x;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      hi = max_nan(max_nan(hi, w[i].x), max_nan(max_nan(w[i].y, w[i].z), w[i].w));
      lo = min_nan(min_nan(lo, w[i].x), min_nan(min_nan(w[i].y, w[i].z), w[i].w));
    }
  }
  __device__ __forceinline__ void eight(int c, float* x) const {
    reinterpret_cast<float4*>(x)[0] = w[2 * c];
    reinterpret_cast<float4*>(x)[1] = w[2 * c + 1];
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) pack_kernel(const T* __restrict__ k,
                                                        const T* __restrict__ v,
                                                        uint8_t* __restrict__ cache,
                                                        const int32_t* __restrict__ starts, int n,
                                                        int per_seq, Dims p) {
  using R = PackedRecord<D>;
  constexpr int NG = R::kGroups;
  __shared__ __align__(16) uint8_t image[R::kBytes];
  bool is_v;
  const Part part = part_of<D>(p, starts, n, per_seq, cache, is_v);
  if (!part.record) return;
  const T* src = (is_v ? v : k) + (size_t)part.token * D;
  const int items = (part.hi - part.lo) * NG;              // a thread a group of 32 dims
  for (int e = threadIdx.x; e < items; e += kThreads) {
    const int row = part.lo + e / NG, g = e % NG;
    GroupLoad<T> x;
    x.load(src + (size_t)e * kPackedGroup);
    float hi, lo;
    x.range(hi, lo);
    const bool bad = !(fabsf(hi) <= 3.402823466e38f && fabsf(lo) <= 3.402823466e38f);
    float step, mid, inv;
    packed_scales(hi, lo, bad, step, mid, inv);
    // codes are monotone in x: unless the ends of the range need it, nothing is clamped
    const float top = __fmul_rn(__fsub_rn(hi, mid), inv), end = __fmul_rn(__fsub_rn(lo, mid), inv);
    const bool clamp = !(top <= 7.25f && end >= -8.25f);
    uint32_t word[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float y[8];
      x.eight(c, y);
      // rint(t) + 8 in the low bits of t + (3 * 2^22 + 8); the constant's own bits, shifted like
      // the codes, are taken off beforehand
      constexpr uint32_t kMagic = 0x4B400000u;
      uint32_t w = 0;
#pragma unroll
      for (int u = 0; u < 8; ++u) w -= kMagic << (4 * u);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        float t = __fmul_rn(__fsub_rn(y[u], mid), inv);
        if (clamp) t = fminf(fmaxf(t, -8.f), 7.f);
        w += __float_as_uint(__fadd_rn(t, 12582920.f)) << (4 * u);
      }
      word[c] = inv > 0.f ? w : 0x88888888u;
    }
    if (is_v) {
#pragma unroll
      for (int r = 0; r < 8; ++r)
        *reinterpret_cast<uint16_t*>(image + R::v_half(row, g, r)) =
            (uint16_t)(word[r / 2] >> (16 * (r & 1)));
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint32_t*>(image + R::k_word(row, g, c)) = word[c];
    }
    *reinterpret_cast<__nv_bfloat16*>(image + R::plane(R::kStepOffset, row, g)) =
        __float2bfloat16_rn(step);
    *reinterpret_cast<__nv_bfloat16*>(image + R::plane(R::kMidOffset, row, g)) =
        __float2bfloat16_rn(mid);
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

// The eight values of a word of codes, lowest nibble first.
__device__ __forceinline__ void store_values(float* dst, uint32_t w, uint32_t step, uint32_t mid,
                                             uint32_t) {
  const float s = __uint_as_float(step << 16), m = __uint_as_float(mid << 16);
  float x[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) x[u] = packed_value((w >> (4 * u)) & 15u, s, m);
  reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
// In bf16: codes as exact integers (or-ed into the mantissa of 128, 136 subtracted), pairs of
// nibbles i and i + 4, one fused multiply-add (one rounding, the product is exact), and the
// pairs put in order.
__device__ __forceinline__ void store_values(__nv_bfloat16* dst, uint32_t w, uint32_t step,
                                             uint32_t mid, uint32_t magic) {
  const uint32_t s2 = step * 0x10001u, m2 = mid * 0x10001u;
  uint32_t x[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    uint32_t c;
    // (x & mask) | magic is one instruction when the magic is in a register
    asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xEA;" : "=r"(c) : "r"(w >> (4 * u)), "r"(magic));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(c), "r"(0x43084308u));
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(x[u]) : "r"(c), "r"(s2), "r"(m2));
  }
  *reinterpret_cast<uint4*>(dst) =
      make_uint4(__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410),
                 __byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632));
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
  const int row0 = part.lo + (int)threadIdx.x / kLanes;
  uint32_t magic;                                          // the bf16 pair 128
  asm volatile("mov.b32 %0, 0x43004300;" : "=r"(magic));
  T* dst = (is_v ? v : k) + (size_t)(part.token + row0 - part.lo) * D + lane * 8;
  // rows go in steps that leave the exchange of V's key pairs alone, so offsets grow evenly
  static_assert(kRowsAtOnce % 16 == 0 && (D == 128 || kRowsAtOnce % 32 == 0), "exchanged pairs");
  int at = is_v ? R::v_half(row0, grp, 2 * c) : R::k_word(row0, grp, c);
  const int more = R::v_half(row0, grp, 2 * c + 1) - R::v_half(row0, grp, 2 * c);
  int plane = R::plane(R::kStepOffset, row0, grp);
#pragma unroll 2
  for (int row = row0; row < part.hi; row += kRowsAtOnce) {
    uint32_t w;
    if (is_v)
      w = *reinterpret_cast<const uint16_t*>(rec + at) |
          (uint32_t)*reinterpret_cast<const uint16_t*>(rec + at + more) << 16;
    else
      w = *reinterpret_cast<const uint32_t*>(rec + at);
    const uint32_t step = *reinterpret_cast<const uint16_t*>(rec + plane);
    const uint32_t mid = *reinterpret_cast<const uint16_t*>(rec + plane + R::kMidOffset -
                                                            R::kStepOffset);
    store_values(dst, w, step, mid, magic);
    at += is_v ? kRowsAtOnce * 2 * R::kGroups : kRowsAtOnce * (D / 2);
    plane += kRowsAtOnce * 2;
    dst += (size_t)kRowsAtOnce * D;
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
  return launch_after(pack_kernel<T, D>, dim3((unsigned)grid), kThreads, 0, 0, st, (const T*)k,
                      (const T*)v, (uint8_t*)cache, starts, n, per_seq, p);
}

template <typename T, int D>
cudaError_t unpack(const Dims& p, int n, const int32_t* starts, const void* cache, void* k,
                   void* v, cudaStream_t st) {
  int per_seq;
  const long long grid = grid_of(p, n, per_seq);
  if (grid > 2147483647ll) return cudaErrorInvalidConfiguration;
  return launch_after(unpack_kernel<T, D>, dim3((unsigned)grid), kThreads, 0, 0, st, (T*)k, (T*)v,
                      (const uint8_t*)cache, starts, n, per_seq, p);
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
