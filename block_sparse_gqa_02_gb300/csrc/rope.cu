// Rotary positions: pairs of dims of every head turn by an angle proportional to the token's
// position, y = scale * R(2 pi p f_i) x, and back for the gradient.  Elementwise, so bound by
// HBM: every element is read once and written once.
//
// The angle is kept as a fraction of a turn in 64-bit fixed point: p * freqs[i] wraps modulo
// one turn in integer arithmetic, exactly, so a position of a million loses nothing and no
// slow range reduction is needed.  The fraction is reduced to an eighth of a turn around the
// nearest quarter, cut to units of 2^-34 turns and becomes an fp32 number (|x| <= 1/4 half turn, so
// its rounding is at most 2^-28 turns), and sine and cosine come from sincospif.
//
// A CTA takes a tile of tokens and heads of one tensor: it forms the tile's sines and cosines
// once in shared memory (each is shared by the heads), then streams the tile with two 16-byte
// loads and stores a unit (the table lies so that neighbouring units read neighbouring banks: in
// the order of the dims its reads took 78 % of shared memory's cycles).  All tensors of a call
// share one launch: their tiles are numbered one after the other.  Measured: 743 us for the
// tensors of a 128K prefill (4.9 GB, 6.6 TB/s), 64.5 us for 420 MB of fp32 gradients (6.5 TB/s);
// 3.7 us on the device for a decode step's four.
#include "common.cuh"
#include "launch.cuh"
#include "ptx.cuh"

namespace msa {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 2;              // units in flight per thread (two 16-byte loads each)
constexpr int kMaxTable = 4096;        // (cos, sin) pairs a tile may hold: 32 KiB

// n / d for 0 <= n < 2^16, 1 <= d < 2^16
struct SmallDiv {
  uint32_t mul;
  int d;
  __device__ __forceinline__ int div(int n) const {
    return d == 1 ? n : (int)__umulhi((uint32_t)n, mul);
  }
};

inline SmallDiv small_div(int d) {
  return {(uint32_t)(d == 1 ? 0 : (1ull << 32) / (uint64_t)d + 1), d};
}

struct Tensor {
  const void* x;
  void* y;
  const uint64_t* freqs;
  int H, d, half, head_major;
  int tk, ht;                          // tokens and heads of a tile
  int tiles_t, tiles_h;                // tiles along a sequence, along the heads
  long long first;                     // number of the tensor's first tile
  SmallDiv by_units, by_ht, by_tk, by_half;
};

struct Args {
  Tensor t[MSA_ROPE_MAX_TENSORS];
  int n, seq, pos_offset, inverse;
  float scale;
  const int32_t* positions;
};

// cos and sin of phase / 2^64 turns
__device__ __forceinline__ float2 turn(uint64_t phase) {
  const uint32_t quarter = (uint32_t)((phase + (1ull << 61)) >> 62);
  const int64_t rest = (int64_t)(phase - ((uint64_t)quarter << 62));   // [-2^61, 2^61)
  const float x = (float)(int32_t)(rest >> 30) * 0x1p-33f;             // half turns
  float s, c;
  sincospif(x, &s, &c);
  const float a = (quarter & 1) ? s : c, b = (quarter & 1) ? c : s;
  return make_float2((quarter == 1 || quarter == 2) ? -a : a, quarter >= 2 ? -b : b);
}

template <typename T> __device__ __forceinline__ uint4 pack16(const float* v);
template <> __device__ __forceinline__ uint4 pack16<float>(const float* v) {
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                    __float_as_uint(v[3]));
}
template <> __device__ __forceinline__ uint4 pack16<__nv_bfloat16>(const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T> __device__ __forceinline__ void unpack16(uint4 u, float* v);
template <> __device__ __forceinline__ void unpack16<float>(uint4 u, float* v) {
  v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
  v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
}
template <> __device__ __forceinline__ void unpack16<__nv_bfloat16>(uint4 u, float* v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// A unit is VP pairs of one row: two 16-byte vectors, at dims VP u and half + VP u (halves)
// or 2 VP u and 2 VP u + VP (interleaved); units past the rotated dims are copied.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ Args a) {
  constexpr int VP = 16 / (int)sizeof(T);
  // cos, sin [tk][VP / 2][unit][2]: the units' loads of one pair of pairs are neighbours
  extern __shared__ __align__(16) float2 table[];
  int ti = 0;
  while (ti + 1 < a.n && (long long)blockIdx.x >= a.t[ti + 1].first) ++ti;
  const Tensor& tn = a.t[ti];
  long long tile = (long long)blockIdx.x - tn.first;
  const int h0 = (int)(tile % tn.tiles_h) * tn.ht;
  tile /= tn.tiles_h;
  const int t0 = (int)(tile % tn.tiles_t) * tn.tk;
  const long long b = tile / tn.tiles_t;
  const int nt = min(tn.tk, a.seq - t0), nh = min(tn.ht, tn.H - h0);
  const int units = tn.by_units.d, rot_units = tn.half / VP;
  const int total = nt * nh * units;
  const bool in_place = tn.x == tn.y;
  const T* x = static_cast<const T*>(tn.x);                // may be y itself
  T* y = static_cast<T*>(tn.y);
  ptx::grid_wait();

  for (int e0 = 0; e0 < total; e0 += kThreads * kBatch) {
    uint4 lo[kBatch], hi[kBatch];
    size_t at[kBatch];
    int tok[kBatch], unit[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int e = e0 + k * kThreads + (int)threadIdx.x;
      unit[k] = -1;
      if (e >= total) continue;
      int r = tn.by_units.div(e);
      const int u = e - r * units;
      int h;
      if (tn.head_major) {                                 // tokens follow each other in memory
        h = nt == tn.tk ? tn.by_tk.div(r) : r / nt;
        tok[k] = r - h * nt;
      } else {                                             // heads do
        tok[k] = nh == tn.ht ? tn.by_ht.div(r) : r / nh;
        h = r - tok[k] * nh;
      }
      if (u >= rot_units && in_place) continue;
      unit[k] = u;
      const size_t row = tn.head_major
          ? ((size_t)b * tn.H + h0 + h) * a.seq + t0 + tok[k]
          : ((size_t)b * a.seq + t0 + tok[k]) * tn.H + h0 + h;
      const int dim = (kInterleaved || u >= rot_units) ? 2 * VP * u : VP * u;
      at[k] = row * tn.d + dim;
      const int gap = (kInterleaved || u >= rot_units) ? VP : tn.half;
      lo[k] = *reinterpret_cast<const uint4*>(x + at[k]);
      hi[k] = *reinterpret_cast<const uint4*>(x + at[k] + gap);
    }
    if (e0 == 0) {                                         // the loads above are in flight
      for (int i = threadIdx.x; i < nt * tn.half; i += kThreads) {
        const int t = tn.by_half.div(i);
        const int f = i - t * tn.half;
        const uint32_t base = a.positions ? (uint32_t)a.positions[b * a.seq + t0 + t]
                                          : (uint32_t)(t0 + t);
        const int32_t p = (int32_t)(base + (uint32_t)a.pos_offset);
        const uint64_t phase = (uint64_t)(int64_t)p * tn.freqs[f];
        const float2 cs = turn(a.inverse ? 0 - phase : phase);
        const int u = f / VP, r = f % VP;
        table[t * tn.half + (r / 2 * rot_units + u) * 2 + (r & 1)] =
            make_float2(cs.x * a.scale, cs.y * a.scale);
      }
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (unit[k] < 0) continue;
      const bool rotate = unit[k] < rot_units;
      const int gap = (kInterleaved || !rotate) ? VP : tn.half;
      if (rotate) {
        float p[VP], q[VP];
        unpack16<T>(lo[k], p);
        unpack16<T>(hi[k], q);
        const float4* cs = reinterpret_cast<const float4*>(table + tok[k] * tn.half) + unit[k];
#pragma unroll
        for (int i = 0; i < VP; ++i) {
          const float4 both = cs[i / 2 * rot_units];
          const float2 w = i & 1 ? make_float2(both.z, both.w) : make_float2(both.x, both.y);
          if (kInterleaved) {                              // pairs (2 i, 2 i + 1) of p then q
            float* v = i < VP / 2 ? p : q;
            const int j = 2 * (i % (VP / 2));
            const float v0 = v[j], v1 = v[j + 1];
            v[j] = v0 * w.x - v1 * w.y;
            v[j + 1] = v0 * w.y + v1 * w.x;
          } else {
            const float v0 = p[i], v1 = q[i];
            p[i] = v0 * w.x - v1 * w.y;
            q[i] = v0 * w.y + v1 * w.x;
          }
        }
        lo[k] = pack16<T>(p);
        hi[k] = pack16<T>(q);
      }
      *reinterpret_cast<uint4*>(y + at[k]) = lo[k];
      *reinterpret_cast<uint4*>(y + at[k] + gap) = hi[k];
    }
  }
}

}  // namespace

cudaError_t launch_rope(const msa_rope_desc& desc, const msa_rope_tensor* tensors, int n,
                        const int32_t* positions, cudaStream_t st) {
  Args a;
  a.n = n;
  a.seq = desc.seq;
  a.pos_offset = desc.pos_offset;
  a.inverse = desc.inverse;
  a.scale = desc.scale == 0.f ? 1.f : desc.scale;
  a.positions = positions;
  const int vp = desc.dtype == MSA_BF16 ? 8 : 4;
  long long all = 0;                                       // units of the whole call
  for (int i = 0; i < n; ++i)
    all += (long long)desc.batch * desc.seq * tensors[i].n_heads * (tensors[i].head_dim / (2 * vp));
  // A tile is up to four units a thread (a CTA's start costs the more the smaller the tile: 2, 4,
  // 8 and 16 units take 765, 743, 741 and 745 us on 4.9 GB), halved until there are five waves of
  // tiles (on 420 MB 2, 4, 8 and 16 units take 65, 65, 69 and 72 us).
  int target = 4 * kThreads;
  while (target > kThreads && all < 5ll * 152 * 8 * target) target /= 2;
  long long tiles = 0;
  int table = 0;
  for (int i = 0; i < n; ++i) {
    const msa_rope_tensor& s = tensors[i];
    Tensor& t = a.t[i];
    t.x = s.x;
    t.y = s.y;
    t.freqs = s.freqs;
    t.H = s.n_heads;
    t.d = s.head_dim;
    t.half = s.rotary_dim / 2;
    t.head_major = s.head_major;
    const int units = s.head_dim / (2 * vp);
    t.ht = target / units;
    if (t.ht < 1) t.ht = 1;
    if (t.ht > s.n_heads) t.ht = s.n_heads;
    t.tk = target / (units * t.ht);
    if (t.tk > kMaxTable / t.half) t.tk = kMaxTable / t.half;
    if (t.tk > desc.seq) t.tk = desc.seq;
    if (t.tk < 1) t.tk = 1;
    t.tiles_t = (desc.seq + t.tk - 1) / t.tk;
    t.tiles_h = (s.n_heads + t.ht - 1) / t.ht;
    t.first = tiles;
    t.by_units = small_div(units);
    t.by_ht = small_div(t.ht);
    t.by_tk = small_div(t.tk);
    t.by_half = small_div(t.half);
    tiles += (long long)desc.batch * t.tiles_t * t.tiles_h;
    if (t.tk * t.half > table) table = t.tk * t.half;
  }
  if (tiles > 2147483647ll) return cudaErrorInvalidConfiguration;
  const size_t smem = (size_t)table * sizeof(float2);
  auto kern = desc.dtype == MSA_BF16
      ? (desc.interleaved ? rope_kernel<__nv_bfloat16, true> : rope_kernel<__nv_bfloat16, false>)
      : (desc.interleaved ? rope_kernel<float, true> : rope_kernel<float, false>);
  return launch_after(kern, dim3((unsigned)tiles), kThreads, smem, 0, st, a);
}

}  // namespace msa
