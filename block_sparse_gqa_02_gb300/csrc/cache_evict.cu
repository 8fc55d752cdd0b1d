// Eviction of cache blocks by accumulated attention weight: which blocks of each sequence stay
// (cache_evict_kernel), and moving them in contiguous caches (cache_gather_kernel).
//
// cache_evict_kernel, one CTA per sequence: block scores (the heads' weights summed in head
// order) become order-preserving 32-bit keys in shared memory, an 8-bit radix select finds the
// threshold, and a scan over the blocks turns "stays" and "goes" into a stable partition of
// the block indices.  Rows are read whole before they are written, so outputs may be the
// inputs.
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

// Exclusive prefix sum over the CTA of one value per thread; total receives the sum.
__device__ __forceinline__ int scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  const int before = (warp > 0 ? warp_sums[warp - 1] : 0) + x - v;
  total = warp_sums[kWarps - 1];
  __syncthreads();
  return before;
}

__global__ void __launch_bounds__(kThreads)
cache_evict_kernel(const float* mass, const int32_t* table, int32_t* __restrict__ kept,
                   int32_t* new_lens, float* mass_out, int32_t* table_out, Dims p, int keep,
                   int n_first, int n_recent) {
  extern __shared__ uint32_t keys[];                       // [nB]: keys, then a row being moved
  uint16_t* order = reinterpret_cast<uint16_t*>(keys + p.nB);   // [nB]: kept, then dropped
  __shared__ uint32_t hist[256];
  __shared__ int warp_sums[kWarps];
  __shared__ uint32_t s_digit;
  __shared__ int s_remaining;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int L = seq_len_of(p, b), n = (L + p.Bk - 1) / p.Bk;
  const int nk = min(n, keep);
  const float* m0 = mass + (size_t)b * p.Hkv * p.nB;

  if (n <= keep) {
    for (int i = tid; i < n; i += kThreads) order[i] = (uint16_t)i;
  } else {
    const int lo = n_first, hi = n - n_recent;             // candidates [lo, hi)
    for (int i = lo + tid; i < hi; i += kThreads) {
      float x = m0[i];
      for (int h = 1; h < p.Hkv; ++h) x = __fadd_rn(x, m0[(size_t)h * p.nB + i]);
      keys[i] = score_key(x);
    }
    const int want = keep - n_first - n_recent;
    uint32_t tau = 0xffffffffu;
    int take_eq = 0;
    if (want > 0) {
      uint32_t prefix = 0, mask = 0;
      int remaining = want;
      for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
        __syncthreads();
        for (int i = lo + tid; i < hi; i += kThreads)
          if ((keys[i] & mask) == prefix) atomicAdd(&hist[(keys[i] >> shift) & 255u], 1u);
        __syncthreads();
        if (tid < 32) {                                    // lane 0 holds bins 255..248
          int c[8], sum = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) sum += c[e] = (int)hist[255 - 8 * tid - e];
          int incl = sum;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (tid >= o) incl += y;
          }
          int cum = incl - sum;
          if (cum < remaining && remaining <= incl) {      // exactly one lane
            int e = 0;
            while (cum + c[e] < remaining) cum += c[e++];
            s_digit = 255u - 8u * tid - e;
            s_remaining = remaining - cum;
          }
        }
        __syncthreads();
        prefix |= s_digit << shift;
        mask |= 255u << shift;
        remaining = s_remaining;
        __syncthreads();
      }
      tau = prefix;
      take_eq = remaining;
    }
    // thread t owns the contiguous blocks [t c, t c + c)
    const int c = (n + kThreads - 1) / kThreads;
    const int i0 = min(n, tid * c), i1 = min(n, i0 + c);
    __syncthreads();
    auto candidate = [&](int i) { return i >= lo && i < hi; };
    int n_eq = 0, total;
    if (want > 0)
      for (int i = i0; i < i1; ++i) n_eq += candidate(i) && keys[i] == tau;
    int rank = scan(n_eq, warp_sums, total);
    auto stays = [&](int i, int& r) {
      if (!candidate(i)) return true;
      if (want <= 0) return false;
      return keys[i] > tau || (keys[i] == tau && r++ < take_eq);
    };
    int n_stay = 0;
    {
      int r = rank;
      for (int i = i0; i < i1; ++i) n_stay += stays(i, r);
    }
    const int before = scan(n_stay, warp_sums, total);
    int stay = before, go = nk + i0 - before;
    for (int i = i0; i < i1; ++i) order[stays(i, rank) ? stay++ : go++] = (uint16_t)i;
  }
  __syncthreads();
  for (int i = tid; i < keep; i += kThreads)
    kept[(size_t)b * keep + i] = i < nk ? (int)order[i] : -1;
  if (tid == 0) new_lens[b] = L - (n - nk) * p.Bk;
  // rows go through shared memory whole: outputs may be the inputs
  for (int h = 0; h < p.Hkv; ++h) {
    const size_t row = ((size_t)b * p.Hkv + h) * p.nB;
    float* buf = reinterpret_cast<float*>(keys);
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) buf[i] = mass[row + i];
    __syncthreads();
    for (int i = tid; i < p.nB; i += kThreads) mass_out[row + i] = i < nk ? buf[order[i]] : 0.f;
  }
  if (table) {
    const size_t row = (size_t)b * p.nB;
    int32_t* buf = reinterpret_cast<int32_t*>(keys);
    __syncthreads();
    for (int i = tid; i < p.nB; i += kThreads) buf[i] = table[row + i];
    __syncthreads();
    for (int i = tid; i < p.nB; i += kThreads) table_out[row + i] = i < n ? buf[order[i]] : buf[i];
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
  for (int64_t x = threadIdx.x; x < n; x += kGatherThreads) dst[x] = src[x];
}

}  // namespace

cudaError_t launch_cache_evict(const Dims& p, int keep, int n_first, int n_recent,
                               const float* mass, const int32_t* table, int32_t* kept,
                               int32_t* new_lens, float* mass_out, int32_t* table_out,
                               cudaStream_t st) {
  const size_t smem = (size_t)p.nB * 6;
  cudaError_t e = cudaFuncSetAttribute(cache_evict_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cache_evict_kernel<<<p.B, kThreads, smem, st>>>(mass, table, kept, new_lens, mass_out,
                                                  table_out, p, keep, n_first, n_recent);
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
