// Decode attention over the 4-bit KV cache (format: include/msa.h, packed_cache.cuh): the new
// token's query heads of a group over the blocks that their KV head selected, as
// sparse_decode does over a 16- or 32-bit cache.
//
// A thread-block cluster takes one (sequence, KV head); its CTAs share the selected blocks out
// and meet through distributed shared memory: each reads the others' running maxima, sums and
// outputs of its slice of the heads, so one launch does the whole step without a workspace.
#include <cooperative_groups.h>

#include "packed_cache.cuh"

namespace cg = cooperative_groups;

namespace msa {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 16;              // query heads of a pass
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// CUDA-core kernel: fp32 arithmetic on the cache's values for fp32 queries.  A block's K, then
// its V, are expanded to fp32 in shared memory.
template <typename T, int D>
struct SimtSmem {
  float kv[kPackedBlock][D + 4];
  float o[kRows][D];                   // outputs of the pass, read by the cluster
  float q[kRows][D];
  float s[kRows][kPackedBlock];
  float m[kRows], l[kRows], alpha[kRows];
  float norm[kRows];                   // log2 of the softmax normaliser
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
packed_decode_simt(const T* __restrict__ q, const uint8_t* __restrict__ cache,
                   const int32_t* __restrict__ sel, T* __restrict__ out, float* __restrict__ lse,
                   float* __restrict__ mass, Dims p, int per) {
  using R = PackedRecord<D>;
  using S = SimtSmem<T, D>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  S& s = *reinterpret_cast<S*>(smem_raw);
  float* weights = reinterpret_cast<float*>(smem_raw + sizeof(S));   // [kRows][per], mass only
  cg::cluster_group cluster = cg::this_cluster();
  const int split = (int)cluster.block_rank(), n_split = (int)cluster.num_blocks();
  const int bg = blockIdx.y, b = bg / p.Hkv, g = bg % p.Hkv;
  const int L = seq_len_of(p, b), nB_b = (L + kPackedBlock - 1) / kPackedBlock;
  const int32_t* srow = sel + (size_t)bg * p.k;
  const int i0 = min(p.k, split * per), i1 = min(p.k, i0 + per);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float c1 = p.sm_scale * kLog2e;
  constexpr int kAcc = kRows * D / kThreads;               // outputs per thread
  const int od = tid % D, orow = tid / D * kAcc;

  // more than 16 heads of a group: one pass after the other, weights added up in order
  for (int h0 = 0; h0 < p.G; h0 += kRows) {
    const int rows = min(kRows, p.G - h0);
    for (int e = tid; e < kRows * D; e += kThreads) {
      const int r = e / D;
      s.q[r][e % D] = r < rows ? to_f32(q[((size_t)b * p.Hq + g * p.G + h0 + r) * D + e % D]) : 0.f;
    }
    if (tid < kRows) {
      s.m[tid] = -INFINITY;
      s.l[tid] = 0.f;
    }
    float acc[kAcc];
#pragma unroll
    for (int a = 0; a < kAcc; ++a) acc[a] = 0.f;
    __syncthreads();

    for (int i = i0; i < i1; ++i) {
      const int blk = srow[i];
      const int phys = blk >= 0 && blk < nB_b ? physical_block(p, b, blk) : -1;
      if (phys < 0) {                                      // same for the whole CTA
        if (mass && tid < kRows) weights[tid * per + i - i0] = -INFINITY;
        continue;
      }
      const uint8_t* rec = cache + ((size_t)phys * p.Hkv + g) * R::kPairBytes;
      const int seen = min(kPackedBlock, L - blk * kPackedBlock);
      // K: words of eight dims in memory order
      for (int e = tid; e < kPackedBlock * D / 8; e += kThreads) {
        const int j = e / (D / 8), w = e % (D / 8), c = w / R::kGroups, grp = w % R::kGroups;
        float* dst = &s.kv[j][grp * kPackedGroup + c * 8];
        const uint32_t x = j < seen ? *reinterpret_cast<const uint32_t*>(rec + e * 4) : 0;
        const float st = j < seen ? load_bf16(rec + R::plane(R::kStepOffset, j, grp)) : 0.f;
        const float md = j < seen ? load_bf16(rec + R::plane(R::kMidOffset, j, grp)) : 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u) dst[u] = packed_value((x >> (4 * u)) & 15u, st, md);
      }
      __syncthreads();
      {
        const int j = tid & (kPackedBlock - 1), r0 = (tid >> 7) * (kRows / 2);
        float dot[kRows / 2];
#pragma unroll
        for (int r = 0; r < kRows / 2; ++r) dot[r] = 0.f;
        for (int d0 = 0; d0 < D; d0 += 4) {
          const float4 kx = *reinterpret_cast<const float4*>(&s.kv[j][d0]);
#pragma unroll
          for (int r = 0; r < kRows / 2; ++r) {
            const float4 qx = *reinterpret_cast<const float4*>(&s.q[r0 + r][d0]);
            dot[r] = fmaf(qx.x, kx.x, dot[r]);
            dot[r] = fmaf(qx.y, kx.y, dot[r]);
            dot[r] = fmaf(qx.z, kx.z, dot[r]);
            dot[r] = fmaf(qx.w, kx.w, dot[r]);
          }
        }
#pragma unroll
        for (int r = 0; r < kRows / 2; ++r) s.s[r0 + r][j] = j < seen ? dot[r] * c1 : -INFINITY;
      }
      __syncthreads();
      // V over K's place; and the softmax of two heads per warp
      for (int e = tid; e < kPackedBlock * D / 4; e += kThreads) {
        const int grp = e % R::kGroups, place = e / R::kGroups % kPackedBlock;
        const int r = e / R::kGroups / kPackedBlock;
        const int j = 2 * ((place / 2) ^ (4 * (r & (R::kGroups == 4 ? 1 : 3)))) + (place & 1);
        float* dst = &s.kv[j][grp * kPackedGroup + r * 4];
        const uint8_t* vr = rec + R::kBytes;
        const uint32_t x = j < seen ? *reinterpret_cast<const uint16_t*>(vr + e * 2) : 0;
        const float st = j < seen ? load_bf16(vr + R::plane(R::kStepOffset, j, grp)) : 0.f;
        const float md = j < seen ? load_bf16(vr + R::plane(R::kMidOffset, j, grp)) : 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) dst[u] = packed_value((x >> (4 * u)) & 15u, st, md);
      }
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int r = warp * 2 + rr;
        float v[4], mx = -INFINITY, sum = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          v[u] = s.s[r][lane + 32 * u];
          mx = fmaxf(mx, v[u]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float m_old = s.m[r], m_new = fmaxf(m_old, mx);
        const float base = m_new == -INFINITY ? 0.f : m_new;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          v[u] = exp2f(v[u] - base);
          s.s[r][lane + 32 * u] = v[u];
          sum += v[u];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        __syncwarp();
        if (lane == 0) {
          const float al = exp2f(m_old - base);
          s.alpha[r] = al;
          s.m[r] = m_new;
          s.l[r] = s.l[r] * al + sum;
          if (mass) weights[r * per + i - i0] = base + log2f(sum);
        }
      }
      __syncthreads();
#pragma unroll
      for (int a = 0; a < kAcc; ++a) acc[a] *= s.alpha[orow + a];
      for (int j = 0; j < seen; ++j) {
        const float vx = s.kv[j][od];
#pragma unroll
        for (int a = 0; a < kAcc; ++a) acc[a] = fmaf(s.s[orow + a][j], vx, acc[a]);
      }
      __syncthreads();
    }
#pragma unroll
    for (int a = 0; a < kAcc; ++a) s.o[orow + a][od] = acc[a];
    cluster.sync();
    // every CTA forms the normalisers; each writes its share of the heads' outputs
    if (tid < kRows) {
      float mx = -INFINITY, sum = 0.f;
      for (int c = 0; c < n_split; ++c) mx = fmaxf(mx, *cluster.map_shared_rank(&s.m[tid], c));
      if (mx != -INFINITY)
        for (int c = 0; c < n_split; ++c)
          sum += exp2f(*cluster.map_shared_rank(&s.m[tid], c) - mx) *
                 *cluster.map_shared_rank(&s.l[tid], c);
      s.norm[tid] = mx == -INFINITY ? -INFINITY : mx + log2f(sum);
      const int h = g * p.G + h0 + tid;
      if (lse && split == 0 && tid < rows) lse[(size_t)b * p.Hq + h] = s.norm[tid] * kLn2;
    }
    __syncthreads();
    for (int e = split * kThreads + tid; e < rows * D; e += n_split * kThreads) {
      const int r = e / D, d = e % D;
      float sum = 0.f;
      if (s.norm[r] != -INFINITY)
        for (int c = 0; c < n_split; ++c)
          sum += exp2f(*cluster.map_shared_rank(&s.m[r], c) - s.norm[r]) *
                 *cluster.map_shared_rank(&s.o[r][d], c);
      out[((size_t)b * p.Hq + g * p.G + h0 + r) * D + d] = from_f32<T>(sum);
    }
    if (mass)
      for (int i = i0 + tid; i < i1; i += kThreads) {
        const int blk = srow[i];
        float sum = 0.f;
        for (int r = 0; r < rows; ++r)
          if (s.norm[r] != -INFINITY) sum += exp2f(weights[r * per + i - i0] - s.norm[r]);
        if (blk >= 0 && blk < nB_b) atomicAdd(mass + (size_t)bg * p.nB + blk, sum);
      }
    cluster.sync();                                        // the others have read this CTA's part
  }
}

template <typename T, int D>
cudaError_t decode_simt(const Dims& p, const void* q, const void* cache, const int32_t* sel,
                        void* out, float* lse, float* mass, cudaStream_t st) {
  auto kern = packed_decode_simt<T, D>;
  int n_split = 1;
  while (n_split < 8 && 2 * n_split <= p.k && 2 * n_split * p.B * p.Hkv <= 2 * 152) n_split *= 2;
  const int per = (p.k + n_split - 1) / n_split;
  const size_t smem = sizeof(SimtSmem<T, D>) + (mass ? sizeof(float) * kRows * per : 0);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n_split, p.B * p.Hkv);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = n_split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, (const T*)q, (const uint8_t*)cache, sel, (T*)out, lse,
                            mass, p, per);
}

}  // namespace

cudaError_t launch_sparse_decode_packed(const Dims& p, const void* q, const void* cache,
                                        const int32_t* sel, void* out, float* lse, float* mass,
                                        cudaStream_t st) {
  if (p.dtype == 1)
    return p.d == 128 ? decode_simt<__nv_bfloat16, 128>(p, q, cache, sel, out, lse, mass, st)
                      : decode_simt<__nv_bfloat16, 64>(p, q, cache, sel, out, lse, mass, st);
  return p.d == 128 ? decode_simt<float, 128>(p, q, cache, sel, out, lse, mass, st)
                    : decode_simt<float, 64>(p, q, cache, sel, out, lse, mass, st);
}

}  // namespace msa
