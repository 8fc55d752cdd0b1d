// The attention weight that every selected block of a decode step receives, added up per KV
// head: mass[b, g, blk] += sum over the group's heads h and the block's keys j of
// exp(z_hj - lse_h).
//
// Where decode runs on the tensor cores, its kernel writes each row's log-sum per block (k
// floats a warp, nothing beside the keys it reads) and the merge forms the weights in CTAs of its
// own: 30.7 us for 134 MB (8 ragged sequences, 64 blocks a head) against 32.7 for the same step
// without them, whose two launches do not overlap.  Other shapes (fp32, head_dim 64, other blocks,
// wide groups) take mass_kernel after the step: CTA = one selection entry of one (sequence, KV
// head), its keys' logits formed again in fp32 from K in shared memory, a thread per key, and
// weighed by the step's log-sum-exps.  A key read from shared memory serves eight heads: 4 x 50000
// keys, 48 blocks a head take 29 us more than the step's 277 (fp32, head_dim 128, 16 heads a KV
// head; 51 with a read per head) and 19 more than its 124 (bf16, head_dim 64; 31).  Either way a
// block's weight is one atomic addition, the only one to its address in a call, so results repeat
// bit for bit.
#include "common.cuh"
#include "sparse_decode_mma.cuh"

namespace msa {

namespace {

constexpr int kThreads = 128;
constexpr int kKeys = 128;             // keys of a pass, one thread each
constexpr float kLog2e = 1.4426950408889634f;

// kHeads: heads that share a read of a key from shared memory, 8 or 2.
template <typename T, int D, int kHeads>
__global__ void __launch_bounds__(kThreads)
mass_kernel(const T* __restrict__ q, const T* __restrict__ k, const int32_t* __restrict__ sel,
            const float* __restrict__ lse, float* __restrict__ mass, Dims p) {
  constexpr int kRow = D + 4;                              // floats of a staged key
  extern __shared__ float smem[];
  float* ks = smem;                                        // [kKeys][kRow]
  const int heads = (p.G + kHeads - 1) / kHeads * kHeads;  // rows past the last head stay zero
  float* qs = smem + kKeys * kRow;                         // [heads][D]
  float* ls = qs + heads * D;                              // [heads] lse in log2 units
  __shared__ float part[kThreads / 32];
  const int bg = blockIdx.y, b = bg / p.Hkv, g = bg % p.Hkv;
  const int L = seq_len_of(p, b), nB_b = (L + p.Bk - 1) / p.Bk;
  const int blk = sel[(size_t)bg * p.k + blockIdx.x];
  if (blk < 0 || blk >= nB_b) return;
  const T* kb = k + ((size_t)bg * p.Sk + (size_t)blk * p.Bk) * D;
  const int seen = min(p.Bk, L - blk * p.Bk);
  for (int e = threadIdx.x; e < heads * D; e += kThreads)
    qs[e] = e < p.G * D ? to_f32(q[((size_t)b * p.Hq + g * p.G) * D + e]) * (p.sm_scale * kLog2e)
                        : 0.f;
  for (int h = threadIdx.x; h < heads; h += kThreads)      // a head without keys adds nothing
    ls[h] = h < p.G ? lse[(size_t)b * p.Hq + g * p.G + h] * kLog2e : -INFINITY;
  float sum = 0.f;
  for (int j0 = 0; j0 < seen; j0 += kKeys) {
    const int n = min(kKeys, seen - j0);
    __syncthreads();
    for (int e = threadIdx.x * Vec16<T>::N; e < n * D; e += kThreads * Vec16<T>::N)
      Vec16<T>::load(kb + (size_t)j0 * D + e, ks + e / D * kRow + e % D);
    __syncthreads();
    const int j = threadIdx.x;
    if (j < n)
      for (int h0 = 0; h0 < p.G; h0 += kHeads) {           // a key's values serve kHeads heads
        float dot[kHeads];
#pragma unroll
        for (int h = 0; h < kHeads; ++h) dot[h] = 0.f;
#pragma unroll 4
        for (int d0 = 0; d0 < D; d0 += 4) {
          const float4 kx = *reinterpret_cast<const float4*>(ks + j * kRow + d0);
#pragma unroll
          for (int h = 0; h < kHeads; ++h) {
            const float4 qx = *reinterpret_cast<const float4*>(qs + (h0 + h) * D + d0);
            dot[h] = fmaf(qx.x, kx.x, dot[h]);
            dot[h] = fmaf(qx.y, kx.y, dot[h]);
            dot[h] = fmaf(qx.z, kx.z, dot[h]);
            dot[h] = fmaf(qx.w, kx.w, dot[h]);
          }
        }
#pragma unroll
        for (int h = 0; h < kHeads; ++h)
          if (ls[h0 + h] != -INFINITY) sum += exp2f(dot[h] - ls[h0 + h]);
      }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kThreads / 32; ++w) sum += part[w];
    atomicAdd(mass + (size_t)bg * p.nB + blk, sum);
  }
}

template <typename T, int D, int kHeads>
cudaError_t run_heads(const Dims& p, const void* q, const void* k, const int32_t* sel,
                     const float* lse, float* mass, cudaStream_t st) {
  auto kern = mass_kernel<T, D, kHeads>;
  const size_t heads = (size_t)(p.G + kHeads - 1) / kHeads * kHeads;
  const size_t smem = sizeof(float) * (kKeys * (D + 4) + heads * (D + 1));
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  kern<<<dim3(p.k, p.B * p.Hkv), kThreads, smem, st>>>((const T*)q, (const T*)k, sel, lse, mass,
                                                       p);
  return cudaGetLastError();
}

// Groups of up to two heads do no work for six that are not there.
template <typename T, int D>
cudaError_t run_mass(const Dims& p, const void* q, const void* k, const int32_t* sel,
                     const float* lse, float* mass, cudaStream_t st) {
  return p.G > 2 ? run_heads<T, D, 8>(p, q, k, sel, lse, mass, st)
                 : run_heads<T, D, 2>(p, q, k, sel, lse, mass, st);
}

}  // namespace

size_t decode_mass_workspace_bytes(const Dims& p) {
  // the decode's scratch, and the blocks' log-sums or (should the caller take none) the
  // log-sum-exps
  const size_t more = sparse_decode_mma_supported(p) ? (size_t)p.k * kDecodeWarps : 1;
  return (decode_workspace_bytes(p) + 15) / 16 * 16 + sizeof(float) * (size_t)p.B * p.Hq * more;
}

cudaError_t launch_sparse_decode_mass(const Dims& p, const void* q, const void* k, const void* v,
                                      const int32_t* sel, void* out, float* lse, float* mass,
                                      float* ws, cudaStream_t st, int* dev_status) {
  float* more = ws + (decode_workspace_bytes(p) + 15) / 16 * 4;
  if (sparse_decode_mma_supported(p))
    return launch_sparse_decode_mma_mass(p, q, k, v, sel, out, lse, mass, ws, more, st, dev_status);
  if (!lse) lse = more;
  cudaError_t e = launch_sparse_decode(p, q, k, v, sel, out, lse, ws, st, dev_status);
  if (e != cudaSuccess) return e;
  if (p.dtype == 1)
    return p.d == 128 ? run_mass<__nv_bfloat16, 128>(p, q, k, sel, lse, mass, st)
                      : run_mass<__nv_bfloat16, 64>(p, q, k, sel, lse, mass, st);
  return p.d == 128 ? run_mass<float, 128>(p, q, k, sel, lse, mass, st)
                    : run_mass<float, 64>(p, q, k, sel, lse, mass, st);
}

}  // namespace msa
