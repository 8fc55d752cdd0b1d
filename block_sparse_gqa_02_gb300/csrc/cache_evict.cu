// Eviction of cache blocks by accumulated attention weight: which blocks of each sequence stay
// (cache_evict_kernel), and moving them in contiguous caches (cache_gather_kernel).
//
// cache_evict_kernel, one CTA per sequence, is a chain of short steps and bound by their
// latency.  Block scores (the heads' weights summed in head order) become order-preserving
// 32-bit keys that stay in registers, a contiguous run of blocks a thread; the threshold, the
// largest key that at least the wanted number reach, is found bit by bit, each bit one count
// over the CTA with a single barrier (histograms in shared memory took longer: weights share
// few exponents, so their atomics collide).  A scan then turns "stays" and "goes" into a stable
// partition of the block indices.  Outputs may be the inputs: kept weights move towards the
// front, in chunks that are read whole before they are written, and the table's row goes
// through shared memory.
//
// cache_gather_kernel streams bytes: one CTA per kept block of one head of one cache.
#include "common.cuh"

namespace msa {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

// Larger float -> larger key; -0 as +0; NaN below everything.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum over the CTA of one value per thread.
__device__ __forceinline__ int scan(int v, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  // every warp adds up the warps before it
  const int before = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sums[lane] : 0);
  return before + x - v;
}

// kPer: blocks a thread owns, thread t those from t kPer on; kPer * kThreads >= nB.
template <int kPer>
__global__ void __launch_bounds__(kThreads)
cache_evict_kernel(const float* mass, const int32_t* table,
                   int32_t* __restrict__ kept, int32_t* new_lens, float* mass_out,
                   int32_t* table_out, Dims p, int keep, int n_first, int n_recent) {
  extern __shared__ uint32_t row[];                        // [nB]: keys, then the table's row
  uint16_t* order = reinterpret_cast<uint16_t*>(row + p.nB);    // [nB]: kept, then dropped
  __shared__ int counts[2][kWarps], sums[2][kWarps];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int L = seq_len_of(p, b), n = (L + p.Bk - 1) / p.Bk;
  const int nk = min(n, keep);
  const float* m0 = mass + (size_t)b * p.Hkv * p.nB;

  if (n <= keep) {
    for (int i = tid; i < n; i += kThreads) order[i] = (uint16_t)i;
  } else {
    const int lo = n_first, hi = n - n_recent;             // candidates [lo, hi)
    constexpr int kBatch = kPer < 8 ? kPer : 8;
    for (int i0 = tid; i0 < n; i0 += kThreads * kBatch) {
      float x[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * kThreads;
        x[u] = i < n ? m0[i] : 0.f;
      }
      for (int h = 1; h < p.Hkv; h += 3) {                 // three heads' loads in flight
        float y[3][kBatch];
#pragma unroll
        for (int v = 0; v < 3; ++v)
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            const int i = i0 + u * kThreads;
            y[v][u] = i < n && h + v < p.Hkv ? m0[(size_t)(h + v) * p.nB + i] : 0.f;
          }
#pragma unroll
        for (int v = 0; v < 3; ++v)
          if (h + v < p.Hkv) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) x[u] = __fadd_rn(x[u], y[v][u]);
          }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * kThreads;
        if (i < n) row[i] = score_key(x[u]);
      }
    }
    __syncthreads();
    // blocks outside [lo, hi) hold key 0 and never count: the thresholds below are above 0
    uint32_t key[kPer];
    const int i0 = tid * kPer;
#pragma unroll
    for (int u = 0; u < kPer; ++u) key[u] = i0 + u >= lo && i0 + u < hi ? row[i0 + u] : 0;
    const int want = keep - n_first - n_recent;
    // the largest threshold that at least `want` keys reach, and how many lie above it
    uint32_t tau = 0;
    int above = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t t = tau | 1u << bit;
      int cnt = 0;
#pragma unroll
      for (int u = 0; u < kPer; ++u) cnt += key[u] >= t;
      cnt = __reduce_add_sync(0xffffffffu, cnt);
      if (lane == 0) counts[bit & 1][warp] = cnt;
      __syncthreads();
      cnt = __reduce_add_sync(0xffffffffu, counts[bit & 1][lane]);
      if (cnt >= want)
        tau = t;
      else
        above = cnt;                                       // keys above the final threshold
    }
    // keys equal to it: the first want - above of them stay
    int n_eq = 0;
#pragma unroll
    for (int u = 0; u < kPer; ++u) n_eq += i0 + u >= lo && i0 + u < hi && key[u] == tau;
    int rank = scan(n_eq, sums[0]);
    uint32_t stays = 0;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int i = i0 + u;
      const bool candidate = i >= lo && i < hi;
      const bool s = !candidate || (want > 0 && (key[u] > tau ||
                                                 (key[u] == tau && rank < want - above)));
      rank += candidate && key[u] == tau;
      stays |= (uint32_t)(s && i < n) << u;
    }
    const int before = scan(__popc(stays), sums[1]);
    int stay = before, go = nk + min(i0, n) - before;
#pragma unroll
    for (int u = 0; u < kPer; ++u)
      if (i0 + u < n) order[(stays >> u & 1) ? stay++ : go++] = (uint16_t)(i0 + u);
  }
  __syncthreads();
  for (int i = tid; i < keep; i += kThreads)
    kept[(size_t)b * keep + i] = i < nk ? (int)order[i] : -1;
  if (tid == 0) new_lens[b] = L - (n - nk) * p.Bk;
  if (table)
    for (int i = tid; i < p.nB; i += kThreads) row[i] = (uint32_t)table[(size_t)b * p.nB + i];
  // weights: entry i comes from order[i] >= i, so a chunk that has been read may be written
  // before the next is read; four entries a thread and head in flight
  constexpr int kMove = 4;
  for (int h = 0; h < p.Hkv; h += 4)
    for (int c0 = 0; c0 < p.nB; c0 += kThreads * kMove) {
      const size_t at = ((size_t)b * p.Hkv + h) * p.nB;
      float x[4][kMove];
#pragma unroll
      for (int u = 0; u < kMove; ++u) {
        const int i = c0 + u * kThreads + tid;
        const int from = i < nk ? (int)order[i] : -1;
#pragma unroll
        for (int v = 0; v < 4; ++v)
          x[v][u] = from >= 0 && h + v < p.Hkv ? mass[at + (size_t)v * p.nB + from] : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kMove; ++u) {
        const int i = c0 + u * kThreads + tid;
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (i < p.nB && h + v < p.Hkv) mass_out[at + (size_t)v * p.nB + i] = x[v][u];
      }
    }
  if (table) {                                             // the row was read before the barriers
    for (int i = tid; i < p.nB; i += kThreads)
      table_out[(size_t)b * p.nB + i] = (int32_t)(i < n ? row[order[i]] : row[i]);
  }
}

constexpr int kGatherThreads = 256;

struct GatherArgs {
  msa_gather_tensor t[MSA_GATHER_MAX_TENSORS];
  long long first[MSA_GATHER_MAX_TENSORS];                 // number of the tensor's first CTA
  int n, keep, block;
};

__global__ void __launch_bounds__(kGatherThreads)
cache_gather_kernel(const __grid_constant__ GatherArgs a, const int32_t* __restrict__ kept) {
  int ti = 0;
  while (ti + 1 < a.n && (long long)blockIdx.x >= a.first[ti + 1]) ++ti;
  const msa_gather_tensor& t = a.t[ti];
  const long long e = (long long)blockIdx.x - a.first[ti];
  const int i = (int)(e % a.keep);
  const long long bh = e / a.keep, b = bh / t.n_heads;
  const int blk = kept[b * a.keep + i];
  if (blk < 0) return;
  const int64_t s0 = (int64_t)blk * a.block, d0 = (int64_t)i * a.block;
  int64_t rows = a.block;
  if (rows > t.src_rows - s0) rows = t.src_rows - s0;
  if (rows > t.dst_rows - d0) rows = t.dst_rows - d0;
  if (rows <= 0) return;
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(t.src) +
                                                    (bh * t.src_rows + s0) * t.row_bytes);
  uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(t.dst) +
                                        (bh * t.dst_rows + d0) * t.row_bytes);
  const int64_t n = rows * (t.row_bytes / 16);
  constexpr int kFlight = 8;                               // 16-byte loads in flight per thread
  for (int64_t x0 = threadIdx.x; x0 < n; x0 += kFlight * kGatherThreads) {
    uint4 v[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u)
      if (x0 + u * kGatherThreads < n) v[u] = __ldcs(src + x0 + u * kGatherThreads);
#pragma unroll
    for (int u = 0; u < kFlight; ++u)
      if (x0 + u * kGatherThreads < n) __stcs(dst + x0 + u * kGatherThreads, v[u]);
  }
}

}  // namespace

cudaError_t launch_cache_evict(const Dims& p, int keep, int n_first, int n_recent,
                               const float* mass, const int32_t* table, int32_t* kept,
                               int32_t* new_lens, float* mass_out, int32_t* table_out,
                               cudaStream_t st) {
  const size_t smem = (size_t)p.nB * 6;
  auto kern = p.nB <= 1024   ? cache_evict_kernel<1>
              : p.nB <= 8192 ? cache_evict_kernel<8>
                             : cache_evict_kernel<32>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  kern<<<p.B, kThreads, smem, st>>>(mass, table, kept, new_lens, mass_out, table_out, p, keep,
                                    n_first, n_recent);
  return cudaGetLastError();
}

cudaError_t launch_cache_gather(int batch, const msa_gather_tensor* tensors, int n,
                                const int32_t* kept, int keep, int block, cudaStream_t st) {
  GatherArgs a;
  a.n = n;
  a.keep = keep;
  a.block = block;
  long long ctas = 0;
  for (int i = 0; i < n; ++i) {
    a.t[i] = tensors[i];
    a.first[i] = ctas;
    ctas += (long long)batch * tensors[i].n_heads * keep;
  }
  if (ctas > 2147483647ll) return cudaErrorInvalidConfiguration;
  cache_gather_kernel<<<(unsigned)ctas, kGatherThreads, 0, st>>>(a, kept);
  return cudaGetLastError();
}

}  // namespace msa
