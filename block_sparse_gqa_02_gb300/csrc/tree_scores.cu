// Index scores of drafted tokens on the CUDA cores: fp32 queries, index_dim 64, other block
// sizes.  (bf16 of 128 dims in blocks of 128: tree_scores_tc.cu.)
//
// CTA = one block of one sequence.  A thread holds a key in registers (dequantised there when the
// cache is packed), a query row is a broadcast from shared memory, and the maximum over the keys
// is taken over the lanes for 32 queries at a time by halving (31 shuffles).  Each key is read
// once; with N tokens of H heads it is used for N H products of dI, so the FMA units bound it (8 x 128K
// tokens, 16 drafts, 8-bit keys: 640 us in fp32 of 128 dims, 295 in bf16 of 64).
#include "index_cache.cuh"
#include "launch.cuh"
#include "ptx.cuh"
#include "tree.cuh"
#include "tree_scores_tc.cuh"

namespace msa {

namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kCols = 32;              // queries (token, head) at a time

// Maximum over the lanes of each of 32 values; lane l returns that of value l.
__device__ __forceinline__ float lane_max(float (&v)[kCols], int lane) {
#pragma unroll
  for (int n = 16; n >= 1; n >>= 1) {
    const bool up = lane & n;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float mine = up ? v[i + n] : v[i], other = up ? v[i] : v[i + n];
      v[i] = fmaxf(mine, __shfl_xor_sync(0xffffffffu, other, n));
    }
  }
  return v[0];
}

// Eight values of a key from 8 codes and the row's scale, or from 16-bit or 32-bit values.
template <typename T> __device__ __forceinline__ void load_row8(const T* x, float* o);
template <> __device__ __forceinline__ void load_row8<float>(const float* x, float* o) {
  Vec16<float>::load(x, o);
  Vec16<float>::load(x + 4, o + 4);
}
template <> __device__ __forceinline__ void load_row8<__nv_bfloat16>(const __nv_bfloat16* x, float* o) {
  Vec16<__nv_bfloat16>::load(x, o);
}

template <int D, typename T>
__device__ __forceinline__ void load_key(const T* rows, long long r, float (&key)[D]) {
#pragma unroll
  for (int e = 0; e < D; e += 8) load_row8<T>(rows + r * D + e, key + e);
}
template <int D>
__device__ __forceinline__ void load_packed(const uint8_t* rec, int r, float (&key)[D]) {
  const float s = pow2_byte(rec[kIndexBlock * D + r]);
#pragma unroll
  for (int e = 0; e < D; e += 16) {
    const uint4 w = *reinterpret_cast<const uint4*>(rec + (size_t)r * D + e);
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 y = from_e4m3_pair(v[i >> 1] >> (i & 1) * 16 & 0xffffu);
      key[e + 2 * i] = y.x * s;
      key[e + 2 * i + 1] = y.y * s;
    }
  }
}

template <typename T, int D, bool kPacked>
__global__ void __launch_bounds__(kThreads)
tree_scores_simt(const T* __restrict__ iq, const void* __restrict__ idx_k,
                 const void* __restrict__ idx_draft, float* __restrict__ scores, Dims p) {
  extern __shared__ __align__(16) float smem[];
  __shared__ TreeWord path[64];
  const int cols = p.nR * p.Hkv;
  float* qs = smem;                                        // [kCols][D]
  float* best = smem + kCols * D;                          // [kWarps][cols rounded up to kCols]
  const int padded = (cols + kCols - 1) / kCols * kCols;
  ptx::grid_wait();
  ptx::launch_dependents();
  const int blk = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int L = seq_len_of(p, b);
  if (tid < 64) path[tid] = tid < p.nR ? tree_path(p, b, tid, L) : 0;
  for (int c = tid; c < kWarps * padded; c += kThreads) best[c] = -INFINITY;
  __syncthreads();

  const long long k0 = (long long)blk * p.Bk;
  const int keys = (int)min((long long)p.Bk, max(0ll, L - k0));   // of the cache in this block
  // a drafted key of this block, one a thread
  const bool drafted = tid < 64 && path[tid] != 0 && tree_pos(path[tid], L) / p.Bk == blk;
  const bool any_draft = __syncthreads_or(drafted);

  // a pass: up to one key a thread, seen by the tokens whose path has bit `bit` (-1: by all)
  auto pass = [&](const float (&key)[D], bool have, int bit) {
    for (int c0 = 0; c0 < cols; c0 += kCols) {
      __syncthreads();
      for (int e = tid * 8; e < kCols * D; e += kThreads * 8) {
        float* to = qs + e;
        if (c0 + e / D < cols) {
          load_row8<T>(iq + ((size_t)b * cols + c0) * D + e, to);
        } else {
#pragma unroll
          for (int x = 0; x < 8; ++x) to[x] = 0.f;
        }
      }
      __syncthreads();
      float v[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        const float4* q4 = reinterpret_cast<const float4*>(qs + c * D);
        float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
        for (int e = 0; e < D / 4; ++e) {
          const float4 x = q4[e];
          a0 = fmaf(x.x, key[4 * e], a0);
          a1 = fmaf(x.y, key[4 * e + 1], a1);
          a2 = fmaf(x.z, key[4 * e + 2], a2);
          a3 = fmaf(x.w, key[4 * e + 3], a3);
        }
        bool see = have && c0 + c < cols;
        if (bit >= 0 && see) see = path[(c0 + c) / p.Hkv] >> bit & 1;
        v[c] = see ? (a0 + a1) + (a2 + a3) : -INFINITY;
      }
      const float top = lane_max(v, lane);
      float& to = best[warp * padded + c0 + lane];
      to = fmaxf(to, top);
    }
  };

  float key[D];
  const int phys = p.block_table ? p.block_table[(size_t)b * p.nB + blk] : b * p.nB + blk;
  const bool there = !(p.block_table || kPacked) || (phys >= 0 && phys < p.n_phys);
  for (int j0 = 0; j0 < keys; j0 += kThreads) {
    const int j = j0 + tid;
    const bool have = j < keys;
#pragma unroll
    for (int e = 0; e < D; ++e) key[e] = 0.f;
    if (have && there) {
      if (kPacked)
        load_packed<D>(static_cast<const uint8_t*>(idx_k) + (size_t)phys * index_record(D), j, key);
      else
        load_key<D, T>(static_cast<const T*>(idx_k),
                       p.block_table ? (long long)phys * p.Bk + j : (long long)b * p.Sk + k0 + j, key);
    }
    pass(key, have, -1);
  }
  if (any_draft) {
#pragma unroll
    for (int e = 0; e < D; ++e) key[e] = 0.f;
    if (drafted) {
      if (kPacked)
        load_packed<D>(static_cast<const uint8_t*>(idx_draft) + (size_t)b * index_record(D), tid, key);
      else
        load_key<D, T>(static_cast<const T*>(idx_draft), (long long)b * p.nR + tid, key);
    }
    pass(key, drafted, tid < 64 ? tid : 0);
  }
  __syncthreads();
  for (int c = tid; c < cols; c += kThreads) {
    float x = best[c];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) x = fmaxf(x, best[w * padded + c]);
    const int node = c / p.Hkv, g = c % p.Hkv;
    scores[(((size_t)b * p.Hkv + g) * p.nR + node) * p.nB + blk] =
        path[node] ? x * p.index_scale : -INFINITY;
  }
}

template <typename T, int D, bool kPacked>
cudaError_t launch_simt(const Dims& p, const void* iq, const void* ik, const void* draft,
                        float* scores, cudaStream_t st) {
  const int padded = (p.nR * p.Hkv + kCols - 1) / kCols * kCols;
  const size_t smem = (size_t)(kCols * D + kWarps * padded) * sizeof(float);
  // the kernel's limit, the same in every call: host threads with other sizes share it
  cudaError_t e = cudaFuncSetAttribute(tree_scores_simt<T, D, kPacked>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
  if (e != cudaSuccess) return e;
  return launch_after(tree_scores_simt<T, D, kPacked>, dim3((unsigned)p.nB, (unsigned)p.B), kThreads,
                      smem, 0, st, (const T*)iq, ik, draft, scores, p);
}

template <typename T, bool kPacked>
cudaError_t launch_simt_dim(const Dims& p, const void* iq, const void* ik, const void* draft,
                            float* scores, cudaStream_t st) {
  return p.dI == 128 ? launch_simt<T, 128, kPacked>(p, iq, ik, draft, scores, st)
                     : launch_simt<T, 64, kPacked>(p, iq, ik, draft, scores, st);
}

}  // namespace

cudaError_t launch_index_scores_tree(const Dims& p, const void* idx_q, const void* idx_k,
                                     const void* idx_draft, int packed, float* scores,
                                     cudaStream_t st, int* dev_status) {
  if (tree_scores_tc_supported(p))
    return launch_tree_scores_tc(p, idx_q, idx_k, idx_draft, packed, scores, st, dev_status);
  if (p.dtype == 1)
    return packed ? launch_simt_dim<__nv_bfloat16, true>(p, idx_q, idx_k, idx_draft, scores, st)
                  : launch_simt_dim<__nv_bfloat16, false>(p, idx_q, idx_k, idx_draft, scores, st);
  return packed ? launch_simt_dim<float, true>(p, idx_q, idx_k, idx_draft, scores, st)
                : launch_simt_dim<float, false>(p, idx_q, idx_k, idx_draft, scores, st);
}

}  // namespace msa
