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
// codes become exact bf16 integers, so products with them lose nothing, and steps and mids
// enter in fp32:
//   z_j = sum_g step_jg (q_g . c_jg) + sum_g mid_jg (sum of q_g),
//   o_g = sum_j (p_j step_jg) c_jg + sum_j p_j mid_jg,      c = code - 8.
// K's codes are or-ed into the mantissa of 16, and the accumulators (one per group of dims) start
// at -24 times the rows' group sums of q, which takes the 16 and the 8 away without an
// instruction per operand; V's are or-ed into that of 128 and 136 is subtracted (its sums run
// over thousands of keys, where the offset would cost digits).  The scores' mid term is one MMA
// whose A operand is the group sums of q, split in three bf16 parts (24 bits).  For the output
// p_j step_jg is formed in fp32 and rounded once to bf16, as the 16-bit cache's kernel rounds
// p_j; the mid term is an MMA with the mids as four more columns.
//
// CTA = one split of a (sequence, KV head), two groups of four warps that take its blocks in
// turn, 32 keys a warp, each warp with a softmax base of its own that moves only when a row's
// maximum passes it by more than 8 (log2 units).  Whole records (K and V of a block, 160 D
// contiguous bytes) come through a ring, one bulk copy each; a group's first warp refills a
// stage in the middle of its next block, when the other warps have left the stage.  Q's
// operands stay in shared memory: at 128 registers a thread two CTAs fit an SM.

constexpr int kMmaGroups = 4;                              // groups of warps
constexpr int kGroupWarps = 4;
constexpr int kMmaWarps = kMmaGroups * kGroupWarps;
constexpr int kMmaThreads = kMmaWarps * 32;
constexpr int kMaxList = 1024;         // blocks of a split
constexpr int kMaxMassList = 128;      // blocks of a split whose weights are kept
constexpr float kSlack = 8.f;

struct Entry {
  int phys, seen, blk;
};

template <int D>
struct MmaSmem {
  static constexpr int kStages = D == 128 ? 8 : 16;
  static constexpr int kGroups = PackedRecord<D>::kGroups;
  union {
    __align__(128) uint8_t ring[kStages][PackedRecord<D>::kPairBytes];
    float part[kMmaWarps][kRows][D + 4];                   // the warps' outputs, after the ring
  };
  float o[kRows][D];                   // the CTA's outputs, relative to m
  uint4 qf[kGroups][2][32];            // Q as A operands, per lane
  float qsum[kGroups][kRows];          // sums of q over a group of dims
  float m[kRows], l[kRows], norm[kRows];
  float wm[kMmaWarps][kRows], wl[kMmaWarps][kRows];
  uint64_t full[kStages], empty[kStages];
  int last[kStages];                   // a stage's last copy
  int abort, count;
};

// d = a b + c
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1,
                                          float c0, float c1, float c2, float c3) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2),
        "f"(c3));
}
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint4& a, uint32_t b0,
                                          uint32_t b1) {
  mma_16816(d, a, b0, b1, d[0], d[1], d[2], d[3]);
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
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Codes in bits 3-6 and 19-22 of x as a pair of bf16 integers 16 + code.
__device__ __forceinline__ uint32_t code_pair_16(uint32_t x) {
  return (x & 0x00780078u) | 0x41804180u;
}

// Codes in bits 0-3 and 16-19 of x as a pair of bf16 integers -8 .. 7.
__device__ __forceinline__ uint32_t code_pair(uint32_t x) {
  const uint32_t v = (x & 0x000f000fu) | 0x43004300u;     // 128 + code
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x43084308u));
  return r;
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t bf16_pair(uint64_t x) {
  float lo, hi;
  split_f32x2(x, lo, hi);
  return bf16_pair(lo, hi);
}

__device__ __forceinline__ float lo_bf16(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
__device__ __forceinline__ uint64_t widen_bf16(uint32_t x) {
  return f32x2(lo_bf16(x), hi_bf16(x));
}

__device__ __forceinline__ uint32_t load_u32(const uint8_t* p) {
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
  const int bg = blockIdx.y, b = bg / p.Hkv, g = bg % p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / kGroupWarps, gw = warp % kGroupWarps;
  const int gr = lane >> 2, c = lane & 3;
  const volatile int* abort = &s.abort;
  const float c1 = p.sm_scale * kLog2e;

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
    if (lane == 0) {
      for (int i = 0; i < kStages; ++i) {
        ptx::mbar_init(&s.full[i], 1);
        ptx::mbar_init(&s.empty[i], kGroupWarps);
        s.last[i] = -1;
      }
      s.abort = 0;
      ptx::fence_barrier_init();
    }
    // the split's blocks, in order, without entries that are no block of the sequence
    const int L = seq_len_of(p, b), nB_b = (L + kPackedBlock - 1) / kPackedBlock;
    const int i0 = min(p.k, split * per), i1 = min(p.k, i0 + per);
    int n = 0;
    for (int i = i0; i < i1; i += 32) {
      const int blk = i + lane < i1 ? sel[(size_t)bg * p.k + i + lane] : -1;
      const int phys = blk >= 0 && blk < nB_b ? physical_block(p, b, blk) : -1;
      const uint32_t there = __ballot_sync(0xffffffffu, phys >= 0);
      if (phys >= 0)
        list[n + __popc(there & ((1u << lane) - 1))] =
            Entry{phys, min(kPackedBlock, L - blk * kPackedBlock), blk};
      n += __popc(there);
    }
    if (lane == 0) s.count = n;
    __syncwarp();
  }

  // more than 16 heads of a group: one pass after the other, weights added up in order
  int first = 0;                                           // copies of the passes before
  for (int h0 = 0; h0 < p.G; h0 += kRows) {
    const int rows = min(kRows, p.G - h0);
    if (warp == kMmaWarps - 1) {
      const int n = s.count;
      for (int i = 0; i < min(n, kStages) && !*abort; ++i)
        if (!issue(first + i, i)) {
          if (lane == 0) {
            s.abort = 1;
            if (status) atomicExch(status, 0x411);
          }
          break;
        }
    } else if (warp < NG) {
      // Q as A operands, dims in the order of the codes in K's words: of group x, k-step kk
      // holds dims 32 x + 8 c + (2 kk, 2 kk + 4) and (2 kk + 1, 2 kk + 5)
      const __nv_bfloat16* q0 = q + ((size_t)b * p.Hq + (size_t)g * p.G + h0) * D;
      uint4 w[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = gr + 8 * r;
        w[r] = row < rows ? *reinterpret_cast<const uint4*>(q0 + (size_t)row * D +
                                                            warp * kPackedGroup + c * 8)
                          : make_uint4(0, 0, 0, 0);
        float t = lo_bf16(w[r].x) + hi_bf16(w[r].x) + lo_bf16(w[r].y) + hi_bf16(w[r].y) +
                  lo_bf16(w[r].z) + hi_bf16(w[r].z) + lo_bf16(w[r].w) + hi_bf16(w[r].w);
        t += __shfl_xor_sync(0xffffffffu, t, 1);
        t += __shfl_xor_sync(0xffffffffu, t, 2);
        if (c == 0) s.qsum[warp][row] = t;
      }
      // dims (0,1) (2,3) (4,5) (6,7) -> (0,4) (1,5) and (2,6) (3,7)
      s.qf[warp][0][lane] =
          make_uint4(__byte_perm(w[0].x, w[0].z, 0x5410), __byte_perm(w[1].x, w[1].z, 0x5410),
                     __byte_perm(w[0].x, w[0].z, 0x7632), __byte_perm(w[1].x, w[1].z, 0x7632));
      s.qf[warp][1][lane] =
          make_uint4(__byte_perm(w[0].y, w[0].w, 0x5410), __byte_perm(w[1].y, w[1].w, 0x5410),
                     __byte_perm(w[0].y, w[0].w, 0x7632), __byte_perm(w[1].y, w[1].w, 0x7632));
    }
    __syncthreads();
    const int n_blocks = s.count;
    // the group sums of q in three bf16 parts: k = part * NG + group
    uint4 qs;
    {
      uint32_t w[4];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float v[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int k = 8 * u + 2 * c + e, part = k / NG;
            float t = s.qsum[k % NG][gr + 8 * r];
            for (int y = 0; y < part; ++y) t -= __bfloat162float(__float2bfloat16_rn(t));
            v[e] = part < 3 ? t : 0.f;
          }
          w[2 * u + r] = bf16_pair(v[0], v[1]);
        }
      qs = make_uint4(w[0], w[1], w[2], w[3]);
    }
    float o[4 * NG][4], om[4];
    float base[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 4 * NG; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
    om[0] = om[1] = om[2] = om[3] = 0.f;

    const int key0 = gw * 32;
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
          mma_16816(sc[2 * half + u], qs, mids, mids, 0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int y = 0; y < NG; ++y) {
          const uint4 a0 = s.qf[y][0][lane], a1 = s.qf[y][1][lane];
          const float i0 = -24.f * s.qsum[y][gr], i1 = -24.f * s.qsum[y][gr + 8];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float acc[4];
            mma_16816(acc, a0, code_pair_16(w[u][y] << 3), code_pair_16(w[u][y] >> 1), i0, i0, i1,
                      i1);
            mma_16816(acc, a1, code_pair_16(w[u][y] >> 5), code_pair_16(w[u][y] >> 9));
            // its keys as accumulator columns: 2 c and 2 c + 1
            const uint64_t step = widen_bf16(load_u32(
                kr + R::plane(R::kStepOffset, key0 + (2 * half + u) * 8 + 2 * c, y)));
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
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2)) * c1;
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
        const uint64_t c2 = f32x2(c1, c1), n0 = f32x2(-b0, -b0), n1 = f32x2(-b1, -b1);
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          split_f32x2(fma_f32x2(f32x2(sc[nt][0], sc[nt][1]), c2, n0), sc[nt][0], sc[nt][1]);
          split_f32x2(fma_f32x2(f32x2(sc[nt][2], sc[nt][3]), c2, n1), sc[nt][2], sc[nt][3]);
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
        const uint64_t p00 = f32x2(p0[0], p0[1]), p01 = f32x2(p0[2], p0[3]);
        const uint64_t p10 = f32x2(p1[0], p1[1]), p11 = f32x2(p1[2], p1[3]);
        {
          uint32_t m0 = 0, m1 = 0;                         // mids of group gr as column gr
          if (gr < NG) {
            m0 = load_u32(vr + R::plane(R::kMidOffset, key, gr));
            m1 = load_u32(vr + R::plane(R::kMidOffset, key + 8, gr));
          }
          mma_16816(om, make_uint4(bf16_pair(p00), bf16_pair(p01), bf16_pair(p10), bf16_pair(p11)),
                    m0, m1);
        }
#pragma unroll
        for (int x = 0; x < NG; ++x) {
          const uint64_t s0 = widen_bf16(load_u32(vr + R::plane(R::kStepOffset, key, x)));
          const uint64_t s1 = widen_bf16(load_u32(vr + R::plane(R::kStepOffset, key + 8, x)));
          const uint4 pa = make_uint4(bf16_pair(mul_f32x2(p00, s0)), bf16_pair(mul_f32x2(p01, s0)),
                                      bf16_pair(mul_f32x2(p10, s1)), bf16_pair(mul_f32x2(p11, s1)));
          // the group's 16 bits of the two keys of each pair, a byte (two dims) at a time
          const int word = x / 2, byte = 2 * (x & 1);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t pick = (uint32_t)(byte + y) * 0x0011u | (uint32_t)(4 + byte + y) * 0x1100u;
            const uint32_t a = __byte_perm(va[word], va[NG / 2 + word], pick);
            const uint32_t e = __byte_perm(vb[word], vb[NG / 2 + word], pick);
            mma_16816(o[4 * x + 2 * y], pa, code_pair(a), code_pair(e));
            mma_16816(o[4 * x + 2 * y + 1], pa, code_pair(a >> 4), code_pair(e >> 4));
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
    // Every warp has left its loop.  Without an abort every copy has been consumed; after one,
    // a warp waits for the last copy of every stage before the memory is used again.
    __syncthreads();
    if (*abort && warp == 0)
      for (int x = 0; x < kStages; ++x)
        if (s.last[x] >= 0) ptx::mbar_wait_timed(&s.full[x], (s.last[x] / kStages) & 1);
    __syncthreads();
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
    // columns 2 c, 2 c + 1 of n-tile 4 x + i are dims 32 x + 4 column + i; the mid term of
    // group x is in lane x / 2 of the quad, element x % 2
#pragma unroll
    for (int x = 0; x < NG; ++x)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float mid = __shfl_sync(0xffffffffu, om[2 * r + (x & 1)], (lane & ~3) | (x >> 1));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 v = make_float4(o[4 * x][2 * r + e] + mid, o[4 * x + 1][2 * r + e] + mid,
                                       o[4 * x + 2][2 * r + e] + mid,
                                       o[4 * x + 3][2 * r + e] + mid);
          *reinterpret_cast<float4*>(
              &s.part[warp][gr + 8 * r][x * kPackedGroup + 4 * (2 * c + e)]) = v;
        }
      }
    __syncthreads();
    // the CTA's outputs, sums and maxima
    if (threadIdx.x < kRows) {
      float top = -INFINITY, sum = 0.f;
      for (int w = 0; w < kMmaWarps; ++w) top = fmaxf(top, s.wm[w][threadIdx.x]);
      if (top != -INFINITY)
        for (int w = 0; w < kMmaWarps; ++w)
          sum += ex2(s.wm[w][threadIdx.x] - top) * s.wl[w][threadIdx.x];
      s.m[threadIdx.x] = top;
      s.l[threadIdx.x] = sum;
    }
    for (int e = threadIdx.x; e < kRows * D / 4; e += kMmaThreads) {
      const int r = e / (D / 4), d0 = e % (D / 4) * 4;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kMmaWarps; ++w) top = fmaxf(top, s.wm[w][r]);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (top != -INFINITY)
#pragma unroll
        for (int w = 0; w < kMmaWarps; ++w) {
          const float f = ex2(s.wm[w][r] - top);
          const float4 u = *reinterpret_cast<const float4*>(&s.part[w][r][d0]);
          v.x = fmaf(f, u.x, v.x);
          v.y = fmaf(f, u.y, v.y);
          v.z = fmaf(f, u.z, v.z);
          v.w = fmaf(f, u.w, v.w);
        }
      *reinterpret_cast<float4*>(&s.o[r][d0]) = v;
    }
    cluster.sync();
    // every CTA forms the normalisers; each writes its share of the heads' outputs
    if (threadIdx.x < kRows) {
      const int r = threadIdx.x;
      float top = -INFINITY, sum = 0.f;
      for (int x = 0; x < n_split; ++x) top = fmaxf(top, *cluster.map_shared_rank(&s.m[r], x));
      if (top != -INFINITY)
        for (int x = 0; x < n_split; ++x)
          sum += ex2(*cluster.map_shared_rank(&s.m[r], x) - top) *
                 *cluster.map_shared_rank(&s.l[r], x);
      s.norm[r] = top == -INFINITY ? -INFINITY : top + __log2f(sum);
      if (lse && split == 0 && r < rows) lse[(size_t)b * p.Hq + g * p.G + h0 + r] = s.norm[r] * kLn2;
    }
    __syncthreads();
    for (int e = split * kMmaThreads + threadIdx.x; e < rows * D / 2; e += n_split * kMmaThreads) {
      const int r = e / (D / 2), d0 = e % (D / 2) * 2;
      float2 v = make_float2(0.f, 0.f);
      if (s.norm[r] != -INFINITY)
        for (int x = 0; x < n_split; ++x) {
          const float f = ex2(*cluster.map_shared_rank(&s.m[r], x) - s.norm[r]);
          const float2 u = *reinterpret_cast<const float2*>(cluster.map_shared_rank(&s.o[r][d0], x));
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
    // the next pass copies into the memory that held the warps' outputs
    if (h0 + kRows < p.G) ptx::fence_proxy_async_smem();
    first += n_blocks;
    cluster.sync();                                        // the others have read this CTA's part
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
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n_split, p.B * p.Hkv);
  cfg.blockDim = dim3(kMmaThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = n_split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, (const __nv_bfloat16*)q, (const uint8_t*)cache, sel,
                            (__nv_bfloat16*)out, lse, mass, p, per, status);
}

// CTAs that share a (sequence, KV head): doubled while they fit on the SMs two at a time
// and have a block each; with weights, as many as their lists need.
int packed_splits(const Dims& p, bool mass) {
  int n = 1;
  while (n < 8 && 2 * n <= p.k && 2 * n * p.B * p.Hkv <= 152) n *= 2;
  while (n < 8 && (p.k + n - 1) / n > (mass ? kMaxMassList : kMaxList)) n *= 2;
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
