// The attention weight that every selected block of a decode step receives, added up per KV
// head: mass[b, g, blk] += sum over the group's heads h and the block's keys j of
// exp(z_hj - lse_h).
//
// Where decode runs on the tensor cores, its kernel writes each row's log-sum per block (k
// floats a warp, nothing beside the keys it reads) and the merge forms the weights in CTAs of its
// own: 30.7 us for 134 MB (8 ragged sequences, 64 blocks a head) against 32.7 for the same step
// without them, whose two launches do not overlap.  A block's weight is one atomic addition, the
// only one to its address in a call, so results repeat bit for bit.
//
// Other shapes (fp32, head_dim 64, other blocks, wide groups) are computed here, on the CUDA
// cores, in fp32 whatever the caches' type: one kernel for every shape that the call takes.  On the
// tensor cores fp32 products would need operands split in three bf16 parts and six products for
// their 24 bits; bf16 ones the decode kernel with head_dim 64, passes of heads and other tiles.
// Neither is built, and the shapes with many heads a KV head are that far from memory's time.
// 4 x 50000 keys, 48 blocks a head: 41 us for 200 MB (fp32, head_dim 128, 8 KV heads of 2), 17 for
// 100 MB (fp32, head_dim 64, 8 of 1: memory), 46 for 100 MB (fp32, head_dim 128, 4 of 16: the
// latency of a tile's 4096 products a lane at two warps a scheduler), 25 for 25 MB (bf16, head_dim
// 64, 4 of 16).
#include <type_traits>

#include "common.cuh"
#include "launch.cuh"
#include "ptx.cuh"
#include "sparse_decode_mma.cuh"

namespace msa {

namespace {

constexpr int kWarps = kDecodeWarps;   // of a CTA; a tile of 32 keys each
constexpr int kThreads = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int kH> __device__ __forceinline__ void load_row(const float* s, float (&o)[kH]) {
  if constexpr (kH == 2) {
    const float2 x = *reinterpret_cast<const float2*>(s);
    o[0] = x.x; o[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < kH; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(s + i);
      o[i] = x.x; o[i + 1] = x.y; o[i + 2] = x.z; o[i + 3] = x.w;
    }
  }
}

// kH values a lane -> the warp's maximum or sum of value `lane / (32 / kH)`: halves of the values
// change lanes until each lane holds one, kH + log2(32 / kH) - 1 shuffles where a reduction per
// value takes 5 kH.
template <int kH, bool kMax>
__device__ __forceinline__ float reduce_heads(const float (&in)[kH], int lane) {
  float v[kH];
#pragma unroll
  for (int i = 0; i < kH; ++i) v[i] = in[i];
  int o = 16;
#pragma unroll
  for (int n = kH / 2; n >= 1; n /= 2, o /= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float mine = up ? v[i + n] : v[i], other = up ? v[i] : v[i + n];
      const float got = __shfl_xor_sync(0xffffffffu, other, o);
      v[i] = kMax ? fmaxf(mine, got) : mine + got;
    }
  }
#pragma unroll
  for (; o > 0; o /= 2) {
    const float got = __shfl_xor_sync(0xffffffffu, v[0], o);
    v[0] = kMax ? fmaxf(v[0], got) : v[0] + got;
  }
  return v[0];
}

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src)
               : "memory");
}

// Elements of V that a lane holds, converted: 4 or 2.
template <typename T, int N> __device__ __forceinline__ void unpack_v(const void* raw, float* o);
template <> __device__ __forceinline__ void unpack_v<float, 4>(const void* raw, float* o) {
  const float4 x = *static_cast<const float4*>(raw);
  o[0] = x.x; o[1] = x.y; o[2] = x.z; o[3] = x.w;
}
template <> __device__ __forceinline__ void unpack_v<float, 2>(const void* raw, float* o) {
  const float2 x = *static_cast<const float2*>(raw);
  o[0] = x.x; o[1] = x.y;
}
template <> __device__ __forceinline__ void unpack_v<__nv_bfloat16, 4>(const void* raw, float* o) {
  const uint2 x = *static_cast<const uint2*>(raw);
  o[0] = __uint_as_float(x.x << 16); o[1] = __uint_as_float(x.x & 0xffff0000u);
  o[2] = __uint_as_float(x.y << 16); o[3] = __uint_as_float(x.y & 0xffff0000u);
}
template <> __device__ __forceinline__ void unpack_v<__nv_bfloat16, 2>(const void* raw, float* o) {
  const uint32_t x = *static_cast<const uint32_t*>(raw);
  o[0] = __uint_as_float(x << 16); o[1] = __uint_as_float(x & 0xffff0000u);
}
template <int kBytes> struct Raw;
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<16> { using type = uint4; };

template <typename T, int D, int kH> struct Layout {
  static constexpr int kKRow = D * (int)sizeof(T) + 16;    // bytes of a staged key: 16 mod 128
  static constexpr int kPRow = kH == 2 ? 2 : kH + 4;       // floats of a key's weights
  static constexpr int kTileBytes = 32 * kKRow;            // K of a warp; its output at the end
  static constexpr int kQ = kWarps * kTileBytes;
  static constexpr int kP = kQ + kH * D * 4;
  static constexpr int kStat = kP + kWarps * 32 * kPRow * 4;
  static constexpr int kBytes = kStat + kWarps * 2 * kH * 4;
  static constexpr int kResident = 232448 / (kBytes + 1024) < 3 ? 232448 / (kBytes + 1024) : 3;
  static_assert(kH * D * 4 <= kTileBytes, "a warp's output fits its K tile");
};

// Grid (splits, B * Hkv, chunks of kH heads).  A warp takes 32 keys of every block of its split
// (again 128 further on, in longer blocks) for kH heads and keeps their running maximum, sum and
// output by itself; the CTA's four are joined at its end.
//   scores: a lane per key, K from shared memory (one read serves kH heads), Q broadcast;
//   output: a lane per D / 32 dims, V from memory to registers, the weights broadcast.
// The copy of the next tile of K runs under the second part.
template <typename T, int D, int kH>
__global__ void __launch_bounds__(kThreads, Layout<T, D, kH>::kResident)
decode_mass_partial(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                    const int32_t* __restrict__ sel, float* __restrict__ ws_o,
                    float* __restrict__ ws_l, float* __restrict__ ws_b, Dims p, int n_split,
                    int per) {
  using L = Layout<T, D, kH>;
  constexpr int kVec = D / 32;                             // dims of a lane
  constexpr int kChunk = 16 / (int)sizeof(T);              // dims of a 16-byte load
  constexpr int kOwn = 32 / kH;                            // lanes that share a head's statistics
  constexpr int kAhead = kH == 2 ? 16 : 8;                 // loads of V in flight
  using RawV = typename Raw<kVec * (int)sizeof(T)>::type;
  extern __shared__ __align__(16) unsigned char smem[];
  ptx::grid_wait();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int bg = blockIdx.y, b = bg / p.Hkv, g = bg % p.Hkv, h0 = blockIdx.z * kH;
  const size_t head0 = (size_t)b * p.Hq + (size_t)g * p.G + h0;
  const int heads = min(kH, p.G - h0);
  unsigned char* ks = smem + warp * L::kTileBytes;
  float* qs = reinterpret_cast<float*>(smem + L::kQ);
  float* ps = reinterpret_cast<float*>(smem + L::kP) + warp * 32 * L::kPRow;
  float* stat = reinterpret_cast<float*>(smem + L::kStat) + warp * 2 * kH;
  const int32_t* srow = sel + (size_t)bg * p.k;
  const T* kb = k + (size_t)bg * p.Sk * D;
  const T* vb = v + (size_t)bg * p.Sk * D;
  const int e0 = blockIdx.x * per, e1 = min(p.k, e0 + per);

  // the warp's tiles in order: entry e, its block's keys [j, j + n) of the cache
  struct Tile { int e, off, j, n; };
  auto settle = [&](Tile& t) {                             // the first tile from (e, off) on
    for (; t.e < e1; ++t.e, t.off = 32 * warp) {
      const int blk = srow[t.e];
      if (blk < 0 || blk >= p.nB) continue;
      const int seen = min(p.Bk, p.Sk - blk * p.Bk);
      if (t.off >= seen) continue;
      t.j = blk * p.Bk + t.off;
      t.n = min(32, seen - t.off);
      return;
    }
    t.n = 0;
  };
  auto copy_k = [&](const Tile& t) {
    const T* src = kb + (size_t)t.j * D;
    for (int c = lane; c < t.n * (D / kChunk); c += 32)
      copy16(ks + c / (D / kChunk) * L::kKRow + c % (D / kChunk) * 16, src + c * kChunk);
  };
  Tile t{e0, 32 * warp, 0, 0};
  settle(t);
  copy_k(t);
  for (int x = threadIdx.x; x < kH * D; x += kThreads)     // rows past the last head are zero
    qs[x] = x / D < heads ? to_f32(q[head0 * D + x]) * (p.sm_scale * kLog2e) : 0.f;
  const int own = lane / kOwn;                             // the head of this lane's statistics
  const bool writer = lane % kOwn == 0 && own < heads;
  float* wb = ws_b + (head0 + own) * p.k * kWarps + warp;
  if (writer)
    for (int e = e0; e < e1; ++e) wb[(size_t)e * kWarps] = -INFINITY;
  __syncthreads();

  float acc[kH][kVec];
#pragma unroll
  for (int h = 0; h < kH; ++h)
#pragma unroll
    for (int i = 0; i < kVec; ++i) acc[h][i] = 0.f;
  float m = -INFINITY, l = 0.f, le = 0.f;                  // maximum, sum, sum of this entry
  while (t.n > 0) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    float2 s2[kH];
#pragma unroll
    for (int h = 0; h < kH; ++h) s2[h] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int c = 0; c < D / kChunk; ++c) {
      float kx[kChunk];
      Vec16<T>::load(reinterpret_cast<const T*>(ks + lane * L::kKRow + c * 16), kx);
#pragma unroll
      for (int h = 0; h < kH; ++h)
#pragma unroll
        for (int i = 0; i < kChunk; i += 4) {
          const float4 qx = *reinterpret_cast<const float4*>(qs + h * D + c * kChunk + i);
          s2[h] = __ffma2_rn(make_float2(qx.x, qx.y), make_float2(kx[i], kx[i + 1]), s2[h]);
          s2[h] = __ffma2_rn(make_float2(qx.z, qx.w), make_float2(kx[i + 2], kx[i + 3]), s2[h]);
        }
    }
    float s[kH];
#pragma unroll
    for (int h = 0; h < kH; ++h) s[h] = s2[h].x + s2[h].y;
    if (lane >= t.n) {
#pragma unroll
      for (int h = 0; h < kH; ++h) s[h] = -INFINITY;
    }
    __syncwarp();                                          // K is read
    const Tile now = t;
    t.off += 32 * kWarps;
    settle(t);
    copy_k(t);

    // a maximum of -inf (nothing but -inf so far) is subtracted as 0; NaN passes the maximum and
    // stays in the sums
    const float mx = fmaxf(m, reduce_heads<kH, true>(s, lane));
    const float ref = mx == -INFINITY ? 0.f : mx;
    const float scale = exp2f(m - ref);
    m = mx;
    if (lane % kOwn == 0) {
      stat[own] = ref;
      stat[kH + own] = scale;
    }
    __syncwarp();
    float r[kH];
    load_row<kH>(stat, r);
#pragma unroll
    for (int h = 0; h < kH; ++h) s[h] = exp2f(s[h] - r[h]);
    load_row<kH>(stat + kH, r);
#pragma unroll
    for (int h = 0; h < kH; ++h)
#pragma unroll
      for (int i = 0; i < kVec; ++i) acc[h][i] *= r[h];
    float* pw = ps + lane * L::kPRow;
    if constexpr (kH == 2) {
      *reinterpret_cast<float2*>(pw) = make_float2(s[0], s[1]);
    } else {
#pragma unroll
      for (int h = 0; h < kH; h += 4)
        *reinterpret_cast<float4*>(pw + h) = make_float4(s[h], s[h + 1], s[h + 2], s[h + 3]);
    }
    const float sum = reduce_heads<kH, false>(s, lane);
    l = l * scale + sum;
    le = le * scale + sum;
    if (t.e != now.e) {                                    // the entry's last tile of this warp
      if (writer) wb[(size_t)now.e * kWarps] = ref + log2f(le);
      le = 0.f;
    }
    __syncwarp();                                          // the weights are there
    const RawV* vr = reinterpret_cast<const RawV*>(vb + (size_t)now.j * D) + lane;
    auto add_v = [&](auto whole) {
      constexpr bool kWhole = decltype(whole)::value;      // 32 keys: nothing to check
#pragma unroll 2
      for (int j0 = 0; j0 < (kWhole ? 32 : now.n); j0 += kAhead) {
        RawV raw[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          if (kWhole || j0 + j < now.n) raw[j] = vr[(j0 + j) * 32];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (!kWhole && j0 + j >= now.n) break;
          float vx[kVec];
          unpack_v<T, kVec>(&raw[j], vx);
          load_row<kH>(ps + (j0 + j) * L::kPRow, r);
#pragma unroll
          for (int h = 0; h < kH; ++h)
#pragma unroll
            for (int i = 0; i < kVec; ++i) acc[h][i] = fmaf(r[h], vx[i], acc[h][i]);
        }
      }
    };
    if (now.n == 32) add_v(std::true_type{});
    else add_v(std::false_type{});
  }

  // the four warps' maxima, sums and outputs
  __syncwarp();                                            // stat of the last tile is read
  if (lane % kOwn == 0) {
    stat[own] = m;
    stat[kH + own] = l;
  }
  float* os = reinterpret_cast<float*>(ks);                // no copy is in flight
#pragma unroll
  for (int h = 0; h < kH; ++h)
#pragma unroll
    for (int i = 0; i < kVec; ++i) os[h * D + lane * kVec + i] = acc[h][i];
  __syncthreads();
  const float* st = reinterpret_cast<const float*>(smem + L::kStat);
  for (int x = threadIdx.x; x < heads * D; x += kThreads) {
    const int h = x / D;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, st[w * 2 * kH + h]);
    const float ref = mx == -INFINITY ? 0.f : mx;
    float o = 0.f, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = exp2f(st[w * 2 * kH + h] - ref);
      sum = fmaf(f, st[w * 2 * kH + kH + h], sum);
      o = fmaf(f, reinterpret_cast<const float*>(smem + w * L::kTileBytes)[x], o);
    }
    const size_t slot = (head0 + h) * n_split + blockIdx.x;
    ws_o[slot * D + x % D] = sum == 0.f ? 0.f : o / sum;
    if (x % D == 0) ws_l[slot] = ref + log2f(sum);
  }
}

// log2 of the sum of 2^l over a head's splits, by a warp; -inf for none.
__device__ __forceinline__ float log_sum(const float* l, int n, int lane) {
  float mx = -INFINITY, sum = 0.f;
  for (int s = lane; s < n; s += 32) mx = fmaxf(mx, l[s]);
#pragma unroll
  for (int o = 16; o > 0; o /= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float ref = mx == -INFINITY ? 0.f : mx;
  for (int s = lane; s < n; s += 32) sum += exp2f(l[s] - ref);
#pragma unroll
  for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return ref + log2f(sum);
}

constexpr int kMergeEntries = 32;      // selection entries of a CTA that adds weights

// CTA = one (b, head): the output and its log-sum-exp, a warp taking every fourth split.  After
// those, CTA = 32 selection entries of one (b, KV head): their weights, the sum over heads and
// warps of 2^(ws_b - log_sum), a warp taking every fourth head.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
decode_mass_merge(const float* __restrict__ ws_o, const float* __restrict__ ws_l,
                  const float* __restrict__ ws_b, const int32_t* __restrict__ sel,
                  T* __restrict__ out, float* __restrict__ lse, float* __restrict__ mass, Dims p,
                  int n_split) {
  constexpr int kMaxG = 64, kVec = D / 32, kAhead = 8;
  __shared__ float norm[kMaxG], part[kWarps][D];
  ptx::grid_wait();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if ((int)blockIdx.x < p.B * p.Hq) {
    const size_t bh = blockIdx.x;
    const float* l = ws_l + bh * n_split;
    const float* o = ws_o + bh * n_split * D + lane * kVec;
    const float all = log_sum(l, n_split, lane);
    float acc[kVec] = {};
    if (all != -INFINITY)
      for (int s0 = warp; s0 < n_split; s0 += kWarps * kAhead) {
        float x[kAhead][kVec], f[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int s = s0 + u * kWarps;
          if (s >= n_split) break;
          unpack_v<float, kVec>(o + (size_t)s * D, x[u]);
          f[u] = l[s];
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if (s0 + u * kWarps >= n_split) break;
          f[u] = exp2f(f[u] - all);
#pragma unroll
          for (int i = 0; i < kVec; ++i) acc[i] = fmaf(f[u], x[u][i], acc[i]);
        }
      }
#pragma unroll
    for (int i = 0; i < kVec; ++i) part[warp][lane * kVec + i] = acc[i];
    __syncthreads();
    if (threadIdx.x < D) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += part[w][threadIdx.x];
      out[bh * D + threadIdx.x] = from_f32<T>(sum);
    }
    if (lse && threadIdx.x == 0) lse[bh] = all * kLn2;
    return;
  }
  const int chunks = (p.k + kMergeEntries - 1) / kMergeEntries;
  const int bg = (blockIdx.x - p.B * p.Hq) / chunks;
  const int i = (blockIdx.x - p.B * p.Hq) % chunks * kMergeEntries + lane;
  const size_t head0 = (size_t)(bg / p.Hkv) * p.Hq + (size_t)(bg % p.Hkv) * p.G;
  const int blk = i < p.k ? sel[(size_t)bg * p.k + i] : -1;
  const bool there = blk >= 0 && blk < p.nB;
  float sum = 0.f;
  for (int h0 = warp; h0 - warp < p.G; h0 += 4 * kWarps) {
    float4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (there && h0 + u * kWarps < p.G)
        x[u] = *reinterpret_cast<const float4*>(
            ws_b + ((head0 + h0 + u * kWarps) * p.k + i) * kWarps);
    if (h0 == warp) {                                      // the first loads are in flight
      for (int h = warp; h < p.G; h += kWarps) {
        const float n = log_sum(ws_l + (head0 + h) * n_split, n_split, lane);
        if (lane == 0) norm[h] = n;
      }
      __syncwarp();                                        // read by the warp that wrote it
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int h = h0 + u * kWarps;
      if (there && h < p.G && norm[h] != -INFINITY)
        sum += (exp2f(x[u].x - norm[h]) + exp2f(x[u].y - norm[h])) +
               (exp2f(x[u].z - norm[h]) + exp2f(x[u].w - norm[h]));
    }
  }
  part[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && there) {
#pragma unroll
    for (int w = 1; w < kWarps; ++w) sum += part[w][lane];
    atomicAdd(mass + (size_t)bg * p.nB + blk, sum);
  }
}

// Heads of a CTA.  Few heads leave more CTAs and shorter tiles, many read the keys fewer times:
// 2 where that makes at most two CTAs an SM, 8 up to four, else 16.  Measured at 16 heads a KV
// head, fp32, head_dim 128, with 2, 8 and 16: 1 x 128 keys 10.3, 13.1 and 18.4 us, 4 x 8000 31.1,
// 21.9 and 24.0, 8 x 8000 53.8, 33.9 and 31.9.
int chunk_heads(const Dims& p) {
  const long long tiles = (long long)p.B * p.Hkv * min(p.k, p.nB);
  if (tiles * ((p.G + 1) / 2) <= 2 * 152 || p.G <= 2) return 2;
  return tiles * ((p.G + 7) / 8) <= 4 * 152 || p.G <= 8 ? 8 : 16;
}

template <typename T> int resident(const Dims& p) {
  const int h = chunk_heads(p);
  return p.d == 128 ? (h == 16 ? Layout<T, 128, 16>::kResident
                               : (h == 8 ? Layout<T, 128, 8>::kResident : Layout<T, 128, 2>::kResident))
                    : (h == 16 ? Layout<T, 64, 16>::kResident
                               : (h == 8 ? Layout<T, 64, 8>::kResident : Layout<T, 64, 2>::kResident));
}

// Splits of whole entries: the CTAs that run at once.
int mass_splits(const Dims& p, int* per) {
  const int h = chunk_heads(p), units = p.B * p.Hkv * ((p.G + h - 1) / h);
  const int slots = 152 * (p.dtype == 1 ? resident<__nv_bfloat16>(p) : resident<float>(p));
  const int want = max(1, min(p.k, slots / units));
  *per = (p.k + want - 1) / want;
  return (p.k + *per - 1) / *per;
}

size_t out_floats(const Dims& p, int n_split) {
  return (size_t)p.B * p.Hq * n_split * p.d;
}
size_t sum_floats(const Dims& p, int n_split) {
  return ((size_t)p.B * p.Hq * n_split + 3) / 4 * 4;
}

template <typename T, int D, int kH>
cudaError_t run_heads(const Dims& p, const void* q, const void* k, const void* v,
                      const int32_t* sel, void* out, float* lse, float* mass, float* ws,
                      cudaStream_t st) {
  int per;
  const int n_split = mass_splits(p, &per);
  float* ws_l = ws + out_floats(p, n_split);
  float* ws_b = ws_l + sum_floats(p, n_split);
  auto kern = decode_mass_partial<T, D, kH>;
  constexpr int smem = Layout<T, D, kH>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_after(kern, dim3(n_split, p.B * p.Hkv, (p.G + kH - 1) / kH), kThreads, smem, 0, st,
                   (const T*)q, (const T*)k, (const T*)v, sel, ws, ws_l, ws_b, p, n_split, per);
  if (e != cudaSuccess) return e;
  const unsigned chunks = (p.k + kMergeEntries - 1) / kMergeEntries;
  return launch_after(decode_mass_merge<T, D>, dim3(p.B * (p.Hq + p.Hkv * chunks)), kThreads, 0, 0,
                      st, ws, ws_l, ws_b, sel, (T*)out, lse, mass, p, n_split);
}

template <typename T, int D, typename... A>
cudaError_t run_mass(const Dims& p, A... a) {
  const int h = chunk_heads(p);
  return h == 16 ? run_heads<T, D, 16>(p, a...)
                 : (h == 8 ? run_heads<T, D, 8>(p, a...) : run_heads<T, D, 2>(p, a...));
}

}  // namespace

size_t decode_mass_workspace_bytes(const Dims& p) {
  // partial outputs, their log-sums and the selection entries' log-sums by warp
  const size_t entries = (size_t)p.B * p.Hq * p.k * kDecodeWarps;
  if (sparse_decode_mma_supported(p))
    return (decode_workspace_bytes(p) + 15) / 16 * 16 + sizeof(float) * entries;
  int per;
  const int n_split = mass_splits(p, &per);
  return sizeof(float) * (out_floats(p, n_split) + sum_floats(p, n_split) + entries);
}

cudaError_t launch_sparse_decode_mass(const Dims& p, const void* q, const void* k, const void* v,
                                      const int32_t* sel, void* out, float* lse, float* mass,
                                      float* ws, cudaStream_t st, int* dev_status) {
  if (sparse_decode_mma_supported(p))
    return launch_sparse_decode_mma_mass(p, q, k, v, sel, out, lse, mass, ws,
                                         ws + (decode_workspace_bytes(p) + 15) / 16 * 4, st,
                                         dev_status);
  if (p.dtype == 1)
    return p.d == 128 ? run_mass<__nv_bfloat16, 128>(p, q, k, v, sel, out, lse, mass, ws, st)
                      : run_mass<__nv_bfloat16, 64>(p, q, k, v, sel, out, lse, mass, ws, st);
  return p.d == 128 ? run_mass<float, 128>(p, q, k, v, sel, out, lse, mass, ws, st)
                    : run_mass<float, 64>(p, q, k, v, sel, out, lse, mass, ws, st);
}

}  // namespace msa
