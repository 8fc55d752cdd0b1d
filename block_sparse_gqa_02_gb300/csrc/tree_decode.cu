// Attention of a tree of drafted tokens over the selected blocks and its own tokens: the
// CUDA-core kernel (fp32, other block sizes) and the join of the splits.  (bf16 in blocks of 128:
// tree_decode_tc.cu.)
//
// CTA = (split of the token's selection, token x heads, sequence x KV head).  A warp takes 32 keys
// at a time and keeps the running maximum, sum and output of kH heads by itself: scores with a
// lane per key (K staged in shared memory, one read serves kH heads), output with a lane per
// D / 32 dims (V from memory, the weights broadcast); the four warps are joined at the end.  The
// tokens of a tree read the blocks that they share through L2.  fp32, 16 drafts of 64 heads on 4, 4 x 64K:
// 1.04 ms; a third of it would be its FMAs, the rest waits for K tiles (two CTAs a SM).
#include "launch.cuh"
#include "ptx.cuh"
#include "tree.cuh"
#include "tree_decode_tc.cuh"

namespace msa {

namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(dst)), "l"(src)
               : "memory");
}

template <int kH, int D, typename T> struct Layout {
  static constexpr int kKRow = D * (int)sizeof(T) + 16;    // bytes of a staged key: 16 mod 128
  static constexpr int kTile = 32 * kKRow;                 // K of a warp
  static constexpr int kOut = kH * D * 4;                  // its output at the end
  static constexpr int kWarp = kTile > kOut ? kTile : kOut;
  static constexpr int kQ = kWarps * kWarp;
  static constexpr int kP = kQ + kH * D * 4;               // [warp][32 keys][kH]
  static constexpr int kStat = kP + kWarps * 32 * kH * 4;  // [warp][2][kH]
  static constexpr int kBytes = kStat + kWarps * 2 * kH * 4;
};

template <typename T, int N> __device__ __forceinline__ void load_dims(const T* x, float* o) {
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = to_f32(x[i]);
}
template <> __device__ __forceinline__ void load_dims<float, 4>(const float* x, float* o) {
  const float4 y = *reinterpret_cast<const float4*>(x);
  o[0] = y.x; o[1] = y.y; o[2] = y.z; o[3] = y.w;
}
template <> __device__ __forceinline__ void load_dims<float, 2>(const float* x, float* o) {
  const float2 y = *reinterpret_cast<const float2*>(x);
  o[0] = y.x; o[1] = y.y;
}
template <>
__device__ __forceinline__ void load_dims<__nv_bfloat16, 4>(const __nv_bfloat16* x, float* o) {
  const uint2 y = *reinterpret_cast<const uint2*>(x);
  o[0] = __uint_as_float(y.x << 16); o[1] = __uint_as_float(y.x & 0xffff0000u);
  o[2] = __uint_as_float(y.y << 16); o[3] = __uint_as_float(y.y & 0xffff0000u);
}
template <>
__device__ __forceinline__ void load_dims<__nv_bfloat16, 2>(const __nv_bfloat16* x, float* o) {
  const uint32_t y = *reinterpret_cast<const uint32_t*>(x);
  o[0] = __uint_as_float(y << 16); o[1] = __uint_as_float(y & 0xffff0000u);
}

template <typename T, int D, int kH>
__global__ void __launch_bounds__(kThreads)
tree_decode_simt(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                 const T* __restrict__ kd, const T* __restrict__ vd,
                 const int32_t* __restrict__ sel, float* __restrict__ ws_o,
                 float* __restrict__ ws_l, Dims p, int n_split, int per) {
  using Lay = Layout<kH, D, T>;
  constexpr int kVec = D / 32;                             // dims of a lane
  constexpr int kChunk = 16 / (int)sizeof(T);
  extern __shared__ __align__(16) unsigned char smem[];
  ptx::grid_wait();
  ptx::launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int split = blockIdx.x, bg = blockIdx.z, b = bg / p.Hkv, g = bg % p.Hkv;
  const int node = blockIdx.y % p.nR, h0 = blockIdx.y / p.nR * kH;
  const int heads = min(kH, p.G - h0);
  const size_t row0 = ((size_t)b * p.nR + node) * p.Hq + (size_t)g * p.G + h0;
  const int L = seq_len_of(p, b);
  const TreeWord path = tree_path(p, b, node, L);
  unsigned char* ks = smem + warp * Lay::kWarp;
  float* qs = reinterpret_cast<float*>(smem + Lay::kQ);
  float* ps = reinterpret_cast<float*>(smem + Lay::kP) + warp * 32 * kH;
  float* stat = reinterpret_cast<float*>(smem + Lay::kStat);

  for (int e = threadIdx.x; e < kH * D; e += kThreads)     // in units of log2
    qs[e] = path && e / D < heads ? to_f32(q[row0 * D + e]) * p.sm_scale * kLog2e : 0.f;
  __syncthreads();

  float m[kH], l[kH], acc[kH][kVec];                       // m: the same in every lane; l: a lane's
#pragma unroll
  for (int h = 0; h < kH; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) acc[h][i] = 0.f;
  }

  // 32 keys from kr, vr on, of which the lanes in `seen` take part
  auto tile = [&](const T* kr, const T* vr, unsigned seen) {
    for (int c = lane; c < 32 * (D / kChunk); c += 32) {
      const int j = c / (D / kChunk);
      if (seen >> j & 1)
        copy16(ks + j * Lay::kKRow + c % (D / kChunk) * 16, kr + (size_t)j * D + c % (D / kChunk) * kChunk);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
    float s[kH];
#pragma unroll
    for (int h = 0; h < kH; ++h) s[h] = 0.f;
    const bool mine = seen >> lane & 1;
    if (mine) {
      const T* row = reinterpret_cast<const T*>(ks + lane * Lay::kKRow);
#pragma unroll 4
      for (int c = 0; c < D; c += kChunk) {
        float x[kChunk];
        Vec16<T>::load(row + c, x);
#pragma unroll
        for (int h = 0; h < kH; ++h)
#pragma unroll
          for (int e = 0; e < kChunk; e += 4) {
            const float4 y = *reinterpret_cast<const float4*>(qs + h * D + c + e);
            s[h] = fmaf(y.x, x[e], s[h]);
            s[h] = fmaf(y.y, x[e + 1], s[h]);
            s[h] = fmaf(y.z, x[e + 2], s[h]);
            s[h] = fmaf(y.w, x[e + 3], s[h]);
          }
      }
    }
#pragma unroll
    for (int h = 0; h < kH; ++h) {
      float top = mine ? s[h] : -INFINITY;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float to = fmaxf(m[h], top);
      const float base = to == -INFINITY ? 0.f : to;
      const float alpha = exp2f(m[h] - base);
      const float w = mine ? exp2f(s[h] - base) : 0.f;
      m[h] = to;
      l[h] = l[h] * alpha + w;
#pragma unroll
      for (int i = 0; i < kVec; ++i) acc[h][i] *= alpha;
      ps[lane * kH + h] = w;
    }
    __syncwarp();
#pragma unroll 8
    for (int j = 0; j < 32; ++j) {
      if (!(seen >> j & 1)) continue;                      // the same in all lanes
      float x[kVec];
      load_dims<T, kVec>(vr + (size_t)j * D + lane * kVec, x);
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        const float w = ps[j * kH + h];
#pragma unroll
        for (int i = 0; i < kVec; ++i) acc[h][i] = fmaf(w, x[i], acc[h][i]);
      }
    }
    __syncwarp();
  };
  auto first = [](int n) { return n >= 32 ? 0xffffffffu : (1u << n) - 1; };

  const int32_t* srow = sel + ((size_t)bg * p.nR + node) * p.k;
  const int e1 = min(p.k, (split + 1) * per);
  if (path) {
    for (int e = split * per; e < e1; ++e) {
      const int blk = srow[e];
      if (blk < 0 || blk >= p.nB) continue;
      const int seen = (int)min((long long)p.Bk, (long long)L - (long long)blk * p.Bk);
      if (seen > 0) {
        long long at;                                      // first row of the block
        if (p.block_table) {
          const int phys = p.block_table[(size_t)b * p.nB + blk];
          if (phys < 0 || phys >= p.n_phys) continue;
          at = ((long long)phys * p.Hkv + g) * p.Bk;
        } else {
          at = (long long)bg * p.Sk + (long long)blk * p.Bk;
        }
        for (int j = warp * 32; j < seen; j += kThreads)
          tile(k + (at + j) * D, v + (at + j) * D, first(seen - j));
      }
      // drafted keys of this block on the token's path: a warp takes every fourth half
      TreeWord in = 0;
      for (int i = lane; i < p.nR; i += 32) {
        const TreeWord other = tree_path(p, b, i, L);
        if ((path >> i & 1) && other && tree_pos(other, L) / p.Bk == blk) in |= 1ull << i;
      }
      const unsigned lo = __reduce_or_sync(0xffffffffu, (unsigned)in);
      const unsigned hi = __reduce_or_sync(0xffffffffu, (unsigned)(in >> 32));
      const size_t at = (size_t)bg * p.nR;
      if (lo && warp == (e & 1) * 2) tile(kd + at * D, vd + at * D, lo);
      if (hi && warp == (e & 1) * 2 + 1) tile(kd + (at + 32) * D, vd + (at + 32) * D, hi);
    }
  }
  __syncthreads();
  // the warp's state to shared memory, its output over its K
#pragma unroll
  for (int h = 0; h < kH; ++h) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], o);
    if (lane == 0) {
      stat[warp * 2 * kH + h] = m[h];
      stat[warp * 2 * kH + kH + h] = l[h];
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      reinterpret_cast<float*>(ks)[h * D + lane * kVec + i] = acc[h][i];
  }
  __syncthreads();
  for (int h = warp; h < heads; h += kWarps) {
    float top = -INFINITY, sum = 0.f, w[kWarps];
#pragma unroll
    for (int x = 0; x < kWarps; ++x) top = fmaxf(top, stat[x * 2 * kH + h]);
    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int x = 0; x < kWarps; ++x) {
      w[x] = exp2f(stat[x * 2 * kH + h] - base);
      sum += w[x] * stat[x * 2 * kH + kH + h];
    }
    const size_t slot = (row0 + h) * n_split + split;
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    for (int i = lane; i < D; i += 32) {
      float o = 0.f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x)
        o = fmaf(w[x], reinterpret_cast<const float*>(smem + x * Lay::kWarp)[h * D + i], o);
      ws_o[slot * D + i] = o * inv;
    }
    if (lane == 0) ws_l[slot] = sum > 0.f ? top / kLog2e + logf(sum) : -INFINITY;
  }
}

// o = sum_s exp(lse_s - lse) o_s with lse = log sum_s exp(lse_s), of a row of out [B, nR, Hq, D].
// kRowWarps warps a row take every kRowWarps-th split each, with the loads of eight in flight: one
// warp while there are few splits, all eight of the CTA when there are many (34 splits of 128 rows,
// cold: 17 us with one warp a row, 6 with eight).
template <typename T, int D, int kRowWarps>
__global__ void __launch_bounds__(256)
tree_combine(const float* __restrict__ ws_o, const float* __restrict__ ws_l, T* __restrict__ out,
             float* __restrict__ lse, Dims p, int n_split) {
  constexpr int kVec = D / 32, kRows = 8 / kRowWarps;
  __shared__ float part[kRowWarps > 1 ? kRowWarps : 1][D + 1];
  ptx::grid_wait();
  ptx::launch_dependents();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, sub = warp % kRowWarps;
  const long long row = (long long)blockIdx.x * kRows + warp / kRowWarps;
  if (row >= (long long)p.B * p.nR * p.Hq) return;         // whole CTAs where warps share a row
  constexpr int kFlight = 8;
  const float* l = ws_l + row * n_split;
  const float* o = ws_o + row * n_split * D + lane * kVec;
  float x[kFlight][kVec];
  auto load = [&](int s0) {
#pragma unroll
    for (int i = 0; i < kFlight; ++i)
      if (s0 + i * kRowWarps < n_split) load_dims<float, kVec>(o + (size_t)(s0 + i * kRowWarps) * D, x[i]);
  };
  float top = lane < n_split ? l[lane] : -INFINITY;
  load(sub);
  for (int s = lane + 32; s < n_split; s += 32) top = fmaxf(top, l[s]);
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
  float acc[kVec], den = 0.f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) acc[i] = 0.f;
  if (top != -INFINITY) {
    for (int s0 = sub; s0 < n_split; s0 += kFlight * kRowWarps) {
      if (s0 != sub) load(s0);
      const int mine = s0 + lane * kRowWarps;
      const float w = lane < kFlight && mine < n_split ? expf(l[mine] - top) : 0.f;
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, i);
        if (s0 + i * kRowWarps >= n_split) continue;
        den += wi;
#pragma unroll
        for (int e = 0; e < kVec; ++e) acc[e] = fmaf(wi, x[i][e], acc[e]);
      }
    }
  }
  if (kRowWarps > 1) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) part[sub][lane * kVec + i] = acc[i];
    if (lane == 0) part[sub][D] = den;
    __syncthreads();
    if (sub) return;
#pragma unroll
    for (int x = 1; x < kRowWarps; ++x) {
      den += part[x][D];
#pragma unroll
      for (int i = 0; i < kVec; ++i) acc[i] += part[x][lane * kVec + i];
    }
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) out[row * D + lane * kVec + i] = from_f32<T>(acc[i] * inv);
  if (lse && lane == 0) {
    const long long bt = row / p.Hq;
    const int h = (int)(row % p.Hq), t = (int)(bt % p.nR), b = (int)(bt / p.nR);
    lse[((size_t)b * p.Hq + h) * p.nR + t] = den > 0.f ? top + logf(den) : -INFINITY;
  }
}

// Splits of a token's selection on the CUDA cores: enough CTAs for two a SM.
int simt_splits(const Dims& p) {
  const long long units = (long long)p.B * p.Hkv * p.nR;
  long long s = (2 * 152 + units - 1) / units;
  if (s > p.k) s = p.k;
  return (int)(s < 1 ? 1 : s);
}

int splits(const Dims& p) {
  return tree_decode_tc_supported(p) ? tree_decode_tc_splits(p) : simt_splits(p);
}

template <typename T, int D, int kH>
cudaError_t launch_simt(const Dims& p, const void* q, const void* k, const void* v, const void* kd,
                        const void* vd, const int32_t* sel, float* ws_o, float* ws_l, int n_split,
                        cudaStream_t st) {
  constexpr int kBytes = Layout<kH, D, T>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(tree_decode_simt<T, D, kH>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != cudaSuccess) return e;
  const int per = (p.k + n_split - 1) / n_split;
  const dim3 grid((unsigned)n_split, (unsigned)(p.nR * ((p.G + kH - 1) / kH)),
                  (unsigned)(p.B * p.Hkv));
  return launch_after(tree_decode_simt<T, D, kH>, grid, kThreads, kBytes, 0, st, (const T*)q,
                      (const T*)k, (const T*)v, (const T*)kd, (const T*)vd, sel, ws_o, ws_l, p,
                      n_split, per);
}

template <typename T, int D>
cudaError_t decode(const Dims& p, const void* q, const void* k, const void* v, const void* kd,
                   const void* vd, const int32_t* sel, void* out, float* lse, float* ws,
                   cudaStream_t st, int* dev_status) {
  const int n_split = splits(p);
  const long long rows = (long long)p.B * p.nR * p.Hq;
  float* ws_o = ws;
  float* ws_l = ws + (size_t)rows * n_split * D;
  cudaError_t e;
  if (tree_decode_tc_supported(p)) {
    e = launch_tree_decode_tc(p, q, k, v, kd, vd, sel, ws_o, ws_l, st, dev_status);
  } else {
    // heads of a CTA: as many as the group has, up to 16 (each chunk reads K and V again)
    auto run = p.G <= 2   ? launch_simt<T, D, 2>
               : p.G <= 4 ? launch_simt<T, D, 4>
               : p.G <= 8 ? launch_simt<T, D, 8>
                          : launch_simt<T, D, 16>;
    e = run(p, q, k, v, kd, vd, sel, ws_o, ws_l, n_split, st);
  }
  if (e != cudaSuccess) return e;
  if (n_split <= 8)
    return launch_after(tree_combine<T, D, 1>, dim3((unsigned)((rows + 7) / 8)), 256, 0, 0, st, ws_o,
                        ws_l, (T*)out, lse, p, n_split);
  return launch_after(tree_combine<T, D, 8>, dim3((unsigned)rows), 256, 0, 0, st, ws_o, ws_l, (T*)out,
                      lse, p, n_split);
}

}  // namespace

size_t tree_workspace_bytes(const Dims& p) {
  return (size_t)p.B * p.nR * p.Hq * splits(p) * (p.d + 1) * sizeof(float);
}

cudaError_t launch_sparse_decode_tree(const Dims& p, const void* q, const void* k, const void* v,
                                      const void* k_draft, const void* v_draft,
                                      const int32_t* sel, void* out, float* lse, float* ws,
                                      cudaStream_t st, int* dev_status) {
  auto run = p.dtype == 1 ? (p.d == 128 ? decode<__nv_bfloat16, 128> : decode<__nv_bfloat16, 64>)
                          : (p.d == 128 ? decode<float, 128> : decode<float, 64>);
  return run(p, q, k, v, k_draft, v_draft, sel, out, lse, ws, st, dev_status);
}

}  // namespace msa
