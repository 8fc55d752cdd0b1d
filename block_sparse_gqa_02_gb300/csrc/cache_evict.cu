// Eviction of cache blocks by accumulated attention weight: which blocks of each sequence stay
// (cache_evict_kernel), and moving them in contiguous caches (cache_gather_kernel).
//
// cache_evict_kernel is a chain of short steps and bound by their latency.  A cluster of CTAs
// takes one sequence.  Each CTA makes the whole choice for itself (no exchange, and the weights
// it reads are in L2 for the others): block scores (the heads' weights summed in head order)
// become order-preserving 32-bit keys, a contiguous run of blocks a thread; a radix select over
// 11, 11 and 10 bits finds the threshold; a scan turns "stays" and "goes" into a stable
// partition of the block indices.  Then the CTAs share the rows to be moved.  Outputs may be
// the inputs: all that a sequence's CTAs read lies before a cluster barrier, and what they
// write after it.  Measured: 11.2 us for 8 sequences of 8192 blocks and 4 heads (the choice takes
// about 7000 of 30000 clocks; finding the threshold bit by bit took 16700, one CTA a sequence
// with loads one after the other 24.6 us).
//
// cache_gather_kernel streams bytes: one CTA per kept block of one head of one cache, eight
// 16-byte loads in flight a thread (301 MB in 41 us, 7.3 TB/s with the writes still in L2).
#include <cooperative_groups.h>

#include "common.cuh"
#include "launch.cuh"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace msa {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMove = 4;               // entries of a row that a thread moves: 4096 a CTA
constexpr int kMaxParts = 8;           // CTAs of a sequence
static_assert(kMaxParts * kThreads * kMove >= kMaxBlocks, "a row is moved in one go");

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
  __shared__ int hist[2048], sums[2][kWarps], found[2];
  cg::cluster_group cluster = cg::this_cluster();
  const int part = (int)cluster.block_rank(), parts = (int)cluster.num_blocks();
  const int b = blockIdx.x / parts, tid = threadIdx.x;
  ptx::grid_wait();
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
    uint32_t key[kPer];
    const int i0 = tid * kPer;
#pragma unroll
    for (int u = 0; u < kPer; ++u) key[u] = i0 + u >= lo && i0 + u < hi ? row[i0 + u] : 0;
    const int want = keep - n_first - n_recent;
    // the want-th largest key (keys outside [lo, hi) are not counted), and how many are above it
    uint32_t tau = 0xffffffffu;
    int above = 0;
    if (want > 0) {
      uint32_t prefix = 0, mask = 0;
      for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digits = pass == 2 ? 1023u : 2047u;
        for (int i = tid; i < 2048; i += kThreads) hist[i] = 0;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kPer; ++u)
          if (i0 + u >= lo && i0 + u < hi && (key[u] & mask) == prefix)
            atomicAdd(&hist[(key[u] >> shift) & digits], 1);
        __syncthreads();
        // thread t: digits 2047 - 2 t and 2046 - 2 t
        const int a0 = hist[2047 - 2 * tid], a1 = hist[2046 - 2 * tid];
        const int before = above + scan(a0 + a1, sums[pass & 1]);
        if (before < want && want <= before + a0 + a1) {   // one thread
          const bool second = want > before + a0;
          found[0] = 2047 - 2 * tid - second;
          found[1] = before + (second ? a0 : 0);
        }
        __syncthreads();
        prefix |= (uint32_t)found[0] << shift;
        mask |= digits << shift;
        above = found[1];
      }
      tau = prefix;
    }
    // keys equal to it: the first want - above of them stay
    int n_eq = 0;
#pragma unroll
    for (int u = 0; u < kPer; ++u) n_eq += i0 + u >= lo && i0 + u < hi && key[u] == tau;
    int rank = scan(n_eq, sums[1]);
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
    const int before = scan(__popc(stays), sums[0]);
    int stay = before, go = nk + min(i0, n) - before;
#pragma unroll
    for (int u = 0; u < kPer; ++u)
      if (i0 + u < n) order[(stays >> u & 1) ? stay++ : go++] = (uint16_t)(i0 + u);
  }
  __syncthreads();
  // the CTA's share of the rows, four entries of four heads a thread at a time; entry i comes
  // from order[i]
  const int share = (p.nB + parts - 1) / parts, e0 = part * share, e1 = min(p.nB, e0 + share);
  const size_t trow = (size_t)b * p.nB;
  for (int i = part * kThreads + tid; i < keep; i += parts * kThreads)
    kept[(size_t)b * keep + i] = i < nk ? (int)order[i] : -1;
  if (table)
    for (int i = e0 + tid; i < e1; i += kThreads)
      row[i] = (uint32_t)table[trow + (i < n ? (int)order[i] : i)];
  for (int h = 0; h < p.Hkv; h += 4) {
    const size_t at = ((size_t)b * p.Hkv + h) * p.nB;
    float x[4][kMove];
#pragma unroll
    for (int u = 0; u < kMove; ++u) {
      const int i = e0 + u * kThreads + tid;
      const int from = i < e1 && i < nk ? (int)order[i] : -1;
#pragma unroll
      for (int v = 0; v < 4; ++v)
        x[v][u] = from >= 0 && h + v < p.Hkv ? mass[at + (size_t)v * p.nB + from] : 0.f;
    }
    cluster.sync();
#pragma unroll
    for (int u = 0; u < kMove; ++u) {
      const int i = e0 + u * kThreads + tid;
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (i < e1 && h + v < p.Hkv) mass_out[at + (size_t)v * p.nB + i] = x[v][u];
    }
  }
  if (part == 0 && tid == 0) new_lens[b] = L - (n - nk) * p.Bk;
  if (table)
    for (int i = e0 + tid; i < e1; i += kThreads) table_out[trow + i] = (int32_t)row[i];
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
  ptx::grid_wait();
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
  const int per = p.nB <= 1024 ? 1 : p.nB <= 8192 ? 8 : 32;
  auto kern = per == 1 ? cache_evict_kernel<1> : per == 8 ? cache_evict_kernel<8>
                                                          : cache_evict_kernel<32>;
  // the kernel's limit, the same in every call: host threads with other sizes share it
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       per * kThreads * 6);
  if (e != cudaSuccess) return e;
  int parts = (p.nB + kThreads - 1) / kThreads;            // at most an entry a thread, or all
  if (parts > kMaxParts) parts = kMaxParts;
  return launch_after(kern, dim3((unsigned)p.B * parts), kThreads, smem, parts, st, mass, table, kept,
                      new_lens, mass_out, table_out, p, keep, n_first, n_recent);
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
  return launch_after(cache_gather_kernel, dim3((unsigned)ctas), kGatherThreads, 0, 0, st, a, kept);
}

}  // namespace msa
