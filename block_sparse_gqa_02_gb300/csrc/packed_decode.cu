// Decode attention over the 4-bit KV cache (format: include/msa.h, packed_cache.cuh): the new
// token's query heads of a group over the blocks that their KV head selected, as
// sparse_decode does over a 16- or 32-bit cache.
//
// A thread-block cluster takes one (sequence, KV head); its CTAs share the selected blocks out
// and meet through distributed shared memory: each reads the others' running maxima, sums and
// outputs of its slice of the heads, so one launch does the whole step without a workspace.
//
// bf16 queries run on the tensor cores (packed_decode_mma), fp32 ones, and rows of more blocks
// than its list holds, on the CUDA cores (packed_decode_simt).
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "launch.cuh"
#include "packed_cache.cuh"
#include "ptx.cuh"

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
  extern __shared__ __align__(128) uint8_t smem_raw[];
  S& s = *reinterpret_cast<S*>(smem_raw);
  float* weights = reinterpret_cast<float*>(smem_raw + sizeof(S));   // [kRows][per], mass only
  cg::cluster_group cluster = cg::this_cluster();
  ptx::grid_wait();
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

// ------------------------------------------------------------------ tensor-core kernel
//
// The G <= 16 heads of a group (16 of them a pass) are the M rows of mma.sync.m16n8k16.  The
// codes become exact fp16 integers c = code - 8: a code or-ed into the mantissa of 1024 (or, four
// bits further up, of 64) with 1032 (72) subtracted, so that two of them share a shift.  Steps
// and mids enter apart from them:
//   z_j = sum_g step_jg (q_g . c_jg) + sum_g mid_jg (sum of q_g),
//   o_g = sum_j (p_j step_jg) c_jg + sum_j p_j mid_jg.
// Scores: q is brought to fp16 by a power of two per row (exact but for values below 2^-14 of
// the row's largest, whose error is 2^-25 of that); the accumulators, one per group of dims, are
// scaled by the steps in fp32; the mid term is one bf16 MMA whose A operand is the group sums
// of q, split in three parts (24 bits).
// Outputs: p and the steps are fp16 (steps relative to the largest of their group that the warp
// has met, times 2^10), and so is their product: roundings of 2^-11, an eighth of what bf16 would
// cost; products below 2^-24 of the largest step lose digits.  The mid term is a bf16 MMA with
// the mids as four more columns.
//
// CTA = one split of a (sequence, KV head), three groups of four warps that take its blocks in
// turn, 32 keys a warp, each warp with a softmax base of its own that moves only when a row's
// maximum passes it by more than 4 (log2 units).  Whole records (K and V of a block, 160 D
// contiguous bytes) come through a ring, one bulk copy each; a group's first warp refills a
// stage in the middle of its next block, when the other warps have left the stage.  Twelve
// warps leave a thread 168 registers, which hold Q's operands and the outputs.
//
// The CTAs of a cluster end by writing their partial outputs, maxima and sums into each
// other's shared memory (each owns a share of the rows), so after one cluster barrier
// everything is local.

constexpr int kMmaGroups = 3;                              // groups of warps
constexpr int kGroupWarps = 4;
constexpr int kMmaWarps = kMmaGroups * kGroupWarps;
constexpr int kMmaThreads = kMmaWarps * 32;
constexpr int kMaxSplits = 8;          // CTAs of a cluster
constexpr int kMaxList = 1024;         // blocks of a split
constexpr int kMaxMassList = 128;      // blocks of a split whose weights are kept
constexpr float kSlack = 4.f;          // p <= 2^4
constexpr int kStepShift = 10;         // steps below 2^11: p * step < 2^15 in fp16
constexpr uint32_t kMinStepExp = 27;   // biased exponent of the smallest step, 2^-100

struct Entry {
  int phys, seen, blk;
};

template <int D>
struct MmaSmem {
  static constexpr int kStages = D == 128 ? 8 : 16;
  static constexpr int kGroups = PackedRecord<D>::kGroups;
  static_assert(kStages <= 32, "the first copies are issued a lane each");
  union {
    __align__(128) uint8_t ring[kStages][PackedRecord<D>::kPairBytes];
    float part[kMmaWarps][kRows][D + 4];                   // the warps' outputs, after the ring
  };
  // from every CTA of the cluster: its outputs of this CTA's rows, its rows' maxima and sums
  float o[kRows][D];                   // [split][row of this CTA][D]
  float m[kMaxSplits][kRows], l[kMaxSplits][kRows];
  float norm[kRows];
  uint4 qf[kGroups][2][32];            // Q as A operands, per lane
  float qsum[kGroups][kRows];          // sums of q over a group of dims
  float cr[kRows];                     // score units to log2 units
  __half vstep[kMmaWarps][kGroups][32];                    // V's steps of a warp's keys
  float wm[kMmaWarps][kRows], wl[kMmaWarps][kRows];
  uint64_t full[kStages], empty[kStages];
  int last[kStages];                   // a stage's last copy
  int abort, count;
};

// d = a b, d += a b
template <bool kBf16>
__device__ __forceinline__ void mma_new(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  if (kBf16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
template <bool kBf16>
__device__ __forceinline__ void mma_add(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  if (kBf16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Pairs of fp32 in a 64-bit register for the paired instructions.
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split_f32x2(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Pairs of fp16.
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// (x & mask) | magic in one instruction: the magic comes in a register that the compiler does not
// know, as it would split the pair of constants into two instructions.
template <uint32_t kMask>
__device__ __forceinline__ uint32_t mask_or(uint32_t x, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "n"(kMask), "r"(magic));
  return r;
}
__device__ __forceinline__ uint32_t opaque(uint32_t x) {
  uint32_t r;
  asm volatile("mov.b32 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// Codes in bits 0-3 and 16-19 (low) or 4-7 and 20-23 (high) of x as integers -8 .. 7; the magics
// are the fp16 pairs 1024 and 64.
struct CodeMagic {
  uint32_t low = opaque(0x64006400u), high = opaque(0x54005400u);
  __device__ __forceinline__ uint32_t lows(uint32_t x) const {
    return sub_f16x2(mask_or<0x000f000fu>(x, low), 0x64086408u);     // 1024 + code - 1032
  }
  __device__ __forceinline__ uint32_t highs(uint32_t x) const {
    return sub_f16x2(mask_or<0x00f000f0u>(x, high), 0x54805480u);    // 64 + code - 72
  }
};

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float lo_bf16(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

__device__ __forceinline__ uint32_t load_u32(const void* p) {
  return *reinterpret_cast<const uint32_t*>(p);
}

// N = 2 or 4 consecutive words.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if (N == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x, w[1] = u.y, w[2 % N] = u.z, w[3 % N] = u.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x, w[1] = u.y;
  }
}

template <int D, bool kMass>
__global__ void __launch_bounds__(kMmaThreads, 1)
packed_decode_mma(const __nv_bfloat16* __restrict__ q, const uint8_t* __restrict__ cache,
                  const int32_t* __restrict__ sel, __nv_bfloat16* __restrict__ out,
                  float* __restrict__ lse, float* __restrict__ mass, Dims p, int per,
                  int* status) {
  using R = PackedRecord<D>;
  using S = MmaSmem<D>;
  constexpr int NG = R::kGroups, kStages = S::kStages;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  S& s = *reinterpret_cast<S*>(smem_raw);
  Entry* list = reinterpret_cast<Entry*>(smem_raw + sizeof(S));                  // [per]
  float* weights = reinterpret_cast<float*>(list + per);   // [kGroupWarps][kRows][per], kMass only
  cg::cluster_group cluster = cg::this_cluster();
  const int split = (int)cluster.block_rank(), n_split = (int)cluster.num_blocks();
  const int own = kRows / n_split;                         // rows that a CTA of the cluster ends
  const int bg = blockIdx.y, b = bg / p.Hkv, g = bg % p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / kGroupWarps, gw = warp % kGroupWarps;
  const int gr = lane >> 2, c = lane & 3;
  const volatile int* abort = &s.abort;
  const float c1 = p.sm_scale * kLog2e;
  // the other CTAs have started before anything is written into their shared memory
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  ptx::grid_wait();

  // Copy number x (block x - first of the list) into its stage, once its last block has left it.
  auto issue = [&](int x, int i) {
    const int st = x % kStages;
    if (!ptx::mbar_wait(&s.empty[st], ((x / kStages) & 1) ^ 1, abort)) return false;
    if (lane == 0) {
      s.last[st] = x;
      ptx::mbar_arrive_expect_tx(&s.full[st], R::kPairBytes);
      ptx::bulk_load(s.ring[st], cache + ((size_t)list[i].phys * p.Hkv + g) * R::kPairBytes,
                     R::kPairBytes, &s.full[st]);
    }
    __syncwarp();
    return true;
  };

  if (warp == kMmaWarps - 1) {
    // the split's blocks, in order, without entries that are no block of the sequence
    const int i0 = min(p.k, split * per), i1 = min(p.k, i0 + per);
    int blk = i0 + lane < i1 ? sel[(size_t)bg * p.k + i0 + lane] : -1;
    const int L = seq_len_of(p, b), nB_b = (L + kPackedBlock - 1) / kPackedBlock;
    if (lane == 0) {
      for (int i = 0; i < kStages; ++i) {
        ptx::mbar_init(&s.full[i], 1);
        ptx::mbar_init(&s.empty[i], kGroupWarps);
        s.last[i] = -1;
      }
      s.abort = 0;
      ptx::fence_barrier_init();
    }
    int n = 0;
    for (int i = i0; i < i1; i += 32) {
      const int phys = blk >= 0 && blk < nB_b ? physical_block(p, b, blk) : -1;
      const uint32_t there = __ballot_sync(0xffffffffu, phys >= 0);
      if (phys >= 0)
        list[n + __popc(there & ((1u << lane) - 1))] =
            Entry{phys, min(kPackedBlock, L - blk * kPackedBlock), blk};
      n += __popc(there);
      blk = i + 32 + lane < i1 ? sel[(size_t)bg * p.k + i + 32 + lane] : -1;
    }
    if (lane == 0) s.count = n;
    __syncwarp();
  }

  // more than 16 heads of a group: one pass after the other, weights added up in order
  int first = 0;                                           // copies of the passes before
  for (int h0 = 0; h0 < p.G; h0 += kRows) {
    const int rows = min(kRows, p.G - h0);
    if (warp == kMmaWarps - 1 && lane < min(s.count, kStages) && !*abort) {
      // the first copies, a lane each; every stage is empty here
      const int x = first + lane, st = x % kStages;
      s.last[st] = x;
      ptx::mbar_arrive_expect_tx(&s.full[st], R::kPairBytes);
      ptx::bulk_load(s.ring[st], cache + ((size_t)list[lane].phys * p.Hkv + g) * R::kPairBytes,
                     R::kPairBytes, &s.full[st]);
    }
    // Q as A operands, dims in the order of the codes in K's words: of group x, k-step kk holds
    // dims 32 x + 8 c + (2 kk, 2 kk + 4) and (2 kk + 1, 2 kk + 5); rows gr and gr + 8
    if (warp < NG) {
      const __nv_bfloat16* q0 = q + ((size_t)b * p.Hq + (size_t)g * p.G + h0) * D;
      uint32_t f0[4], f1[4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = gr + 8 * r;
        uint4 w[NG];
#pragma unroll
        for (int x = 0; x < NG; ++x)
          w[x] = row < rows ? *reinterpret_cast<const uint4*>(q0 + (size_t)row * D +
                                                              x * kPackedGroup + c * 8)
                            : make_uint4(0, 0, 0, 0);
        uint32_t top = 0;                                  // largest |q| of the row, bf16 bits
#pragma unroll
        for (int x = 0; x < NG; ++x) {
          const uint32_t v[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
          for (int u = 0; u < 4; ++u) top = max(top, max(v[u] & 0x7fffu, (v[u] >> 16) & 0x7fffu));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t e = min(max(top >> 7, 1u), 253u);
        const float f = __uint_as_float((254u - e) << 23);
        uint4 own = w[0];
#pragma unroll
        for (int x = 1; x < NG; ++x)
          if (warp == x) own = w[x];
        const float d0 = lo_bf16(own.x) * f, d1 = hi_bf16(own.x) * f;
        const float d2 = lo_bf16(own.y) * f, d3 = hi_bf16(own.y) * f;
        const float d4 = lo_bf16(own.z) * f, d5 = hi_bf16(own.z) * f;
        const float d6 = lo_bf16(own.w) * f, d7 = hi_bf16(own.w) * f;
        f0[r] = f16_pair(d0, d4);
        f0[2 + r] = f16_pair(d1, d5);
        f1[r] = f16_pair(d2, d6);
        f1[2 + r] = f16_pair(d3, d7);
        float t = ((d0 + d1) + (d2 + d3)) + ((d4 + d5) + (d6 + d7));
        t += __shfl_xor_sync(0xffffffffu, t, 1);
        t += __shfl_xor_sync(0xffffffffu, t, 2);
        if (c == 0) s.qsum[warp][row] = t;
        if (warp == 0 && c == 0) s.cr[row] = c1 * __uint_as_float(e << 23);
      }
      s.qf[warp][0][lane] = make_uint4(f0[0], f0[1], f0[2], f0[3]);
      s.qf[warp][1][lane] = make_uint4(f1[0], f1[1], f1[2], f1[3]);
    }
    __syncthreads();
    const int n_blocks = s.count;
    const float cr[2] = {s.cr[gr], s.cr[gr + 8]};
    // the group sums of q in three bf16 parts: k = part * NG + group
    uint32_t qs[4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int x = NG == 4 ? 2 * (c & 1) : 0;
      const float t0 = s.qsum[x][gr + 8 * r], t1 = s.qsum[x + 1][gr + 8 * r];
      const float a0 = __bfloat162float(__float2bfloat16_rn(t0));
      const float a1 = __bfloat162float(__float2bfloat16_rn(t1));
      const float b0 = __bfloat162float(__float2bfloat16_rn(t0 - a0));
      const float b1 = __bfloat162float(__float2bfloat16_rn(t1 - a1));
      const uint32_t hi = bf16_pair(a0, a1), md = bf16_pair(b0, b1);
      const uint32_t lo = bf16_pair(t0 - a0 - b0, t1 - a1 - b1);
      if (NG == 4) {
        qs[r] = c < 2 ? hi : md;
        qs[2 + r] = c < 2 ? lo : 0u;
      } else {
        qs[r] = c == 0 ? hi : c == 1 ? md : c == 2 ? lo : 0u;
        qs[2 + r] = 0u;
      }
    }
    float o[4 * NG][4], om[4];
    float base[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    uint32_t vexp[NG];                                     // exponent of V's largest step so far
#pragma unroll
    for (int t = 0; t < 4 * NG; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
    om[0] = om[1] = om[2] = om[3] = 0.f;
#pragma unroll
    for (int x = 0; x < NG; ++x) vexp[x] = kMinStepExp;

    const int key0 = gw * 32;
    const CodeMagic codes;
    bool ok = !*abort;
    for (int i = group; ok && i < n_blocks; i += kMmaGroups) {
      const int st = (first + i) % kStages;
      ok = ptx::mbar_wait(&s.full[st], ((first + i) / kStages) & 1, abort);
      if (!ok) break;
      uint8_t* kr = s.ring[st];
      uint8_t* vr = kr + R::kBytes;
      const int seen = list[i].seen;
      if (seen < kPackedBlock) {
        // keys past the sequence: whatever their bytes hold counts as zero
        if (key0 + lane >= seen)
#pragma unroll
          for (int y = 0; y < 2 * NG; ++y) {
            *reinterpret_cast<uint16_t*>(kr + R::plane(R::kStepOffset, key0 + lane, y)) = 0;
            *reinterpret_cast<uint16_t*>(vr + R::plane(R::kStepOffset, key0 + lane, y)) = 0;
          }
        ptx::fence_proxy_async_smem();                     // before the stage's next copy
        __syncwarp();
      }
      // V's steps of the warp's keys (one a lane) in fp16, relative to the largest of their group
      {
        uint32_t t[NG], e[NG];
        bool grows = false;
#pragma unroll
        for (int x = 0; x < NG; ++x) {
          t[x] = *reinterpret_cast<const uint16_t*>(vr + R::plane(R::kStepOffset, key0 + lane, x));
          e[x] = __reduce_max_sync(0xffffffffu, t[x]) >> 7;
          grows |= e[x] > vexp[x];
        }
        if (grows) {                                       // the same in all lanes
#pragma unroll
          for (int x = 0; x < NG; ++x) {
            const float f = e[x] > vexp[x] ? ex2((float)vexp[x] - (float)e[x]) : 1.f;
            vexp[x] = max(vexp[x], e[x]);
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
              for (int v = 0; v < 4; ++v) o[4 * x + u][v] *= f;
          }
        }
#pragma unroll
        for (int x = 0; x < NG; ++x)
          s.vstep[warp][x][lane] = __float2half_rn(
              lo_bf16(t[x]) * __uint_as_float((254 + kStepShift - vexp[x]) << 23));
        __syncwarp();
      }
      // scores of 16 rows x 32 keys, two n-tiles (16 keys) at a time
      float sc[4][4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t w[2][NG];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int key = key0 + (2 * half + u) * 8 + gr;  // this lane's key as a B column
          load_words<NG>(kr + R::k_word(key, 0, c), w[u]);
          const int x = NG == 4 ? 2 * (c & 1) : 0;
          const uint32_t mids =
              *reinterpret_cast<const uint16_t*>(kr + R::plane(R::kMidOffset, key, x)) |
              (uint32_t)*reinterpret_cast<const uint16_t*>(kr + R::plane(R::kMidOffset, key, x + 1))
                  << 16;
          mma_new<true>(sc[2 * half + u], qs, mids, mids);
        }
#pragma unroll
        for (int y = 0; y < NG; ++y) {
          const uint4 v0 = s.qf[y][0][lane], v1 = s.qf[y][1][lane];
          const uint32_t a0[4] = {v0.x, v0.y, v0.z, v0.w}, a1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float acc[4];
            const uint32_t w8 = w[u][y] >> 8;
            mma_new<false>(acc, a0, codes.lows(w[u][y]), codes.highs(w[u][y]));
            mma_add<false>(acc, a1, codes.lows(w8), codes.highs(w8));
            // its keys as accumulator columns: 2 c and 2 c + 1
            const uint32_t st2 = load_u32(
                kr + R::plane(R::kStepOffset, key0 + (2 * half + u) * 8 + 2 * c, y));
            const uint64_t step = f32x2(lo_bf16(st2), hi_bf16(st2));
            float(&t)[4] = sc[2 * half + u];
            split_f32x2(fma_f32x2(f32x2(acc[0], acc[1]), step, f32x2(t[0], t[1])), t[0], t[1]);
            split_f32x2(fma_f32x2(f32x2(acc[2], acc[3]), step, f32x2(t[2], t[3])), t[2], t[3]);
          }
        }
      }
      // the stage of this group's block before: its other warps have most likely left it
      if (gw == 0 && i >= kMmaGroups && i - kMmaGroups + kStages < n_blocks) {
        ok = issue(first + i - kMmaGroups + kStages, i - kMmaGroups + kStages);
        if (!ok) break;
      }
      if (seen < kPackedBlock) {
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          const int col = key0 + nt * 8 + 2 * c;
          if (col >= seen) sc[nt][0] = sc[nt][2] = -INFINITY;
          if (col + 1 >= seen) sc[nt][1] = sc[nt][3] = -INFINITY;
        }
      }
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        mx[0] = fmaxf(mx[0], fmaxf(sc[nt][0], sc[nt][1]));
        mx[1] = fmaxf(mx[1], fmaxf(sc[nt][2], sc[nt][3]));
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2)) * cr[r];
      }
      if (__any_sync(0xffffffffu, mx[0] > base[0] + kSlack || mx[1] > base[1] + kSlack)) {
        float alpha[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float up = fmaxf(base[r], mx[r]);
          alpha[r] = up == -INFINITY ? 1.f : ex2(base[r] - up);
          base[r] = up;
          l_run[r] *= alpha[r];
        }
#pragma unroll
        for (int t = 0; t < 4 * NG; ++t) {
          o[t][0] *= alpha[0];
          o[t][1] *= alpha[0];
          o[t][2] *= alpha[1];
          o[t][3] *= alpha[1];
        }
        om[0] *= alpha[0];
        om[1] *= alpha[0];
        om[2] *= alpha[1];
        om[3] *= alpha[1];
      }
      float sum[2] = {0.f, 0.f};
      {
        const float b0 = base[0] == -INFINITY ? 0.f : base[0];
        const float b1 = base[1] == -INFINITY ? 0.f : base[1];
        const uint64_t r0 = f32x2(cr[0], cr[0]), r1 = f32x2(cr[1], cr[1]);
        const uint64_t n0 = f32x2(-b0, -b0), n1 = f32x2(-b1, -b1);
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          split_f32x2(fma_f32x2(f32x2(sc[nt][0], sc[nt][1]), r0, n0), sc[nt][0], sc[nt][1]);
          split_f32x2(fma_f32x2(f32x2(sc[nt][2], sc[nt][3]), r1, n1), sc[nt][2], sc[nt][3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[nt][e] = ex2(sc[nt][e]);
          sum[0] += sc[nt][0] + sc[nt][1];
          sum[1] += sc[nt][2] + sc[nt][3];
        }
      }
      l_run[0] += sum[0];
      l_run[1] += sum[1];
      if (kMass) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
          sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
        }
        const float bs = c ? base[1] : base[0], sm = c ? sum[1] : sum[0];
        if (c < 2)
          weights[(gw * kRows + gr + 8 * c) * per + i] =
              bs == -INFINITY ? -INFINITY : bs + __log2f(sm);
      }
      // outputs: 16 keys a step
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const int key = key0 + ks * 16 + 2 * c;            // keys key, key + 1, key + 8, key + 9
        const int pair = key / 2;
        uint32_t va[NG], vb[NG];                           // NG / 2 words of each key of the pair
        load_words<NG>(vr + R::v_half(2 * pair, 0, gr), va);
        load_words<NG>(vr + R::v_half(2 * (pair + 4), 0, gr), vb);
        const float* p0 = sc[2 * ks];
        const float* p1 = sc[2 * ks + 1];
        {
          uint32_t m0 = 0, m1 = 0;                         // mids of group gr as column gr
          if (gr < NG) {
            m0 = load_u32(vr + R::plane(R::kMidOffset, key, gr));
            m1 = load_u32(vr + R::plane(R::kMidOffset, key + 8, gr));
          }
          const uint32_t pb[4] = {bf16_pair(p0[0], p0[1]), bf16_pair(p0[2], p0[3]),
                                  bf16_pair(p1[0], p1[1]), bf16_pair(p1[2], p1[3])};
          mma_add<true>(om, pb, m0, m1);
        }
        const uint32_t ph[4] = {f16_pair(p0[0], p0[1]), f16_pair(p0[2], p0[3]),
                                f16_pair(p1[0], p1[1]), f16_pair(p1[2], p1[3])};
#pragma unroll
        for (int x = 0; x < NG; ++x) {
          const uint32_t s0 = load_u32(&s.vstep[warp][x][ks * 16 + 2 * c]);
          const uint32_t s1 = load_u32(&s.vstep[warp][x][ks * 16 + 8 + 2 * c]);
          const uint32_t pa[4] = {mul_f16x2(ph[0], s0), mul_f16x2(ph[1], s0),
                                  mul_f16x2(ph[2], s1), mul_f16x2(ph[3], s1)};
          // the group's 16 bits of the two keys of each pair, a byte (two dims) at a time
          const int word = x / 2, byte = 2 * (x & 1);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t pick = (uint32_t)(byte + y) * 0x0011u | (uint32_t)(4 + byte + y) * 0x1100u;
            const uint32_t a = __byte_perm(va[word], va[NG / 2 + word], pick);
            const uint32_t e = __byte_perm(vb[word], vb[NG / 2 + word], pick);
            mma_add<false>(o[4 * x + 2 * y], pa, codes.lows(a), codes.lows(e));
            mma_add<false>(o[4 * x + 2 * y + 1], pa, codes.highs(a), codes.highs(e));
          }
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&s.empty[st]);
    }
    if (!ok && lane == 0) {
      s.abort = 1;
      if (status) atomicExch(status, 0x412);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l_run[r] += __shfl_xor_sync(0xffffffffu, l_run[r], 1);
      l_run[r] += __shfl_xor_sync(0xffffffffu, l_run[r], 2);
    }
    if (c == 0) {
      s.wm[warp][gr] = base[0];
      s.wm[warp][gr + 8] = base[1];
      s.wl[warp][gr] = l_run[0];
      s.wl[warp][gr + 8] = l_run[1];
    }
    // Every warp has left its loop.  Without an abort every copy has been consumed; after one,
    // a warp waits for the last copy of every stage before the memory is used again.
    __syncthreads();
    if (*abort) {
      if (warp == 0)
        for (int x = 0; x < kStages; ++x)
          if (s.last[x] >= 0) ptx::mbar_wait_timed(&s.full[x], (s.last[x] / kStages) & 1);
      __syncthreads();
    }
    // the warp's outputs relative to the CTA's maxima.  Columns 2 c, 2 c + 1 of n-tile 4 x + i
    // are dims 32 x + 4 column + i; the mid term of group x is in lane x / 2 of the quad,
    // element x % 2
    float rel[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kMmaWarps; ++w) top = fmaxf(top, s.wm[w][gr + 8 * r]);
      rel[r] = base[r] == -INFINITY ? 0.f : ex2(base[r] - top);
    }
#pragma unroll
    for (int x = 0; x < NG; ++x) {
      const float f = __uint_as_float((vexp[x] - kStepShift) << 23);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float mid = rel[r] * __shfl_sync(0xffffffffu, om[2 * r + (x & 1)],
                                               (lane & ~3) | (x >> 1));
        const float fr = f * rel[r];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 v = make_float4(
              fmaf(o[4 * x][2 * r + e], fr, mid), fmaf(o[4 * x + 1][2 * r + e], fr, mid),
              fmaf(o[4 * x + 2][2 * r + e], fr, mid), fmaf(o[4 * x + 3][2 * r + e], fr, mid));
          *reinterpret_cast<float4*>(
              &s.part[warp][gr + 8 * r][x * kPackedGroup + 4 * (2 * c + e)]) = v;
        }
      }
    }
    if (h0 == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    __syncthreads();
    // the CTA's maxima and sums to every CTA of the cluster, its outputs to the rows' owners
    if (threadIdx.x < kRows * n_split) {
      const int r = threadIdx.x % kRows, to = threadIdx.x / kRows;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kMmaWarps; ++w) top = fmaxf(top, s.wm[w][r]);
      if (top != -INFINITY)
#pragma unroll
        for (int w = 0; w < kMmaWarps; ++w) sum += ex2(s.wm[w][r] - top) * s.wl[w][r];
      *cluster.map_shared_rank(&s.m[split][r], to) = top;
      *cluster.map_shared_rank(&s.l[split][r], to) = sum;
    }
    for (int e = threadIdx.x; e < kRows * D / 4; e += kMmaThreads) {
      const int r = e / (D / 4), d0 = e % (D / 4) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kMmaWarps; ++w) {
        const float4 u = *reinterpret_cast<const float4*>(&s.part[w][r][d0]);
        v.x += u.x;
        v.y += u.y;
        v.z += u.z;
        v.w += u.w;
      }
      *reinterpret_cast<float4*>(
          cluster.map_shared_rank(&s.o[split * own + r % own][d0], r / own)) = v;
    }
    cluster.sync();
    if (threadIdx.x < kRows) {
      const int r = threadIdx.x;
      float top = -INFINITY, sum = 0.f;
      for (int x = 0; x < n_split; ++x) top = fmaxf(top, s.m[x][r]);
      if (top != -INFINITY)
        for (int x = 0; x < n_split; ++x) sum += ex2(s.m[x][r] - top) * s.l[x][r];
      s.norm[r] = top == -INFINITY ? -INFINITY : top + __log2f(sum);
      if (lse && split == 0 && r < rows) lse[(size_t)b * p.Hq + g * p.G + h0 + r] = s.norm[r] * kLn2;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < own * D / 2; e += kMmaThreads) {
      const int ro = e / (D / 2), r = split * own + ro, d0 = e % (D / 2) * 2;
      if (r >= rows) break;
      float2 v = make_float2(0.f, 0.f);
      if (s.norm[r] != -INFINITY)
        for (int x = 0; x < n_split; ++x) {
          const float f = ex2(s.m[x][r] - s.norm[r]);
          const float2 u = *reinterpret_cast<const float2*>(&s.o[x * own + ro][d0]);
          v.x = fmaf(f, u.x, v.x);
          v.y = fmaf(f, u.y, v.y);
        }
      *reinterpret_cast<__nv_bfloat162*>(out + ((size_t)b * p.Hq + g * p.G + h0 + r) * D + d0) =
          __floats2bfloat162_rn(v.x, v.y);
    }
    if (kMass)
      for (int i = threadIdx.x; i < n_blocks; i += kMmaThreads) {
        float sum = 0.f;
        for (int r = 0; r < rows; ++r)
          if (s.norm[r] != -INFINITY)
            for (int w = 0; w < kGroupWarps; ++w)
              sum += ex2(weights[(w * kRows + r) * per + i] - s.norm[r]);
        if (!*abort) atomicAdd(mass + (size_t)bg * p.nB + list[i].blk, sum);
      }
    first += n_blocks;
    if (h0 + kRows < p.G) {
      // the next pass copies into the memory that held the warps' outputs, and the others
      // write into this CTA's
      ptx::fence_proxy_async_smem();
      cluster.sync();
    }
  }
}

template <int D, bool kMass>
cudaError_t decode_mma(const Dims& p, int n_split, const void* q, const void* cache,
                       const int32_t* sel, void* out, float* lse, float* mass, cudaStream_t st,
                       int* status) {
  auto kern = packed_decode_mma<D, kMass>;
  const int per = (p.k + n_split - 1) / n_split;
  const size_t smem = sizeof(MmaSmem<D>) + sizeof(Entry) * per +
                      (kMass ? sizeof(float) * kGroupWarps * kRows * per : 0);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  return launch_after(kern, dim3(n_split, p.B * p.Hkv), kMmaThreads, smem, n_split, st, (const __nv_bfloat16*)q, (const uint8_t*)cache, sel, (__nv_bfloat16*)out, lse, mass, p, per, status);
}

// CTAs that share a (sequence, KV head): doubled while they fit on the SMs two at a time
// and have a block each; with weights, as many as their lists need.
int packed_splits(const Dims& p, bool mass) {
  int n = 1;
  while (n < kMaxSplits && 2 * n <= p.k && 2 * n * p.B * p.Hkv <= 152) n *= 2;
  while (n < kMaxSplits && (p.k + n - 1) / n > (mass ? kMaxMassList : kMaxList)) n *= 2;
  return n;
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
  return launch_after(kern, dim3(n_split, p.B * p.Hkv), kThreads, smem, n_split, st, (const T*)q, (const uint8_t*)cache, sel, (T*)out, lse, mass, p, per);
}

}  // namespace

cudaError_t launch_sparse_decode_packed(const Dims& p, const void* q, const void* cache,
                                        const int32_t* sel, void* out, float* lse, float* mass,
                                        cudaStream_t st, int* dev_status) {
  const int n = packed_splits(p, mass != nullptr);
  if (p.dtype == 1 && (p.k + n - 1) / n <= kMaxList) {
    if (p.d == 128)
      return mass ? decode_mma<128, true>(p, n, q, cache, sel, out, lse, mass, st, dev_status)
                  : decode_mma<128, false>(p, n, q, cache, sel, out, lse, mass, st, dev_status);
    return mass ? decode_mma<64, true>(p, n, q, cache, sel, out, lse, mass, st, dev_status)
                : decode_mma<64, false>(p, n, q, cache, sel, out, lse, mass, st, dev_status);
  }
  if (p.dtype == 1)
    return p.d == 128 ? decode_simt<__nv_bfloat16, 128>(p, q, cache, sel, out, lse, mass, st)
                      : decode_simt<__nv_bfloat16, 64>(p, q, cache, sel, out, lse, mass, st);
  return p.d == 128 ? decode_simt<float, 128>(p, q, cache, sel, out, lse, mass, st)
                    : decode_simt<float, 64>(p, q, cache, sel, out, lse, mass, st);
}

}  // namespace msa
