// Decode attention over the 4-bit KV cache (format: include/msa.h, packed_cache.cuh): the new
// token's query heads of a group over the blocks that their KV head selected, as
// sparse_decode does over a 16- or 32-bit cache.
//
// A thread-block cluster takes one (sequence, KV head); its CTAs share the selected blocks out
// and meet through distributed shared memory, so one launch does the whole step without a
// workspace.
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
// of q, split in three parts (24 bits).  The row's power of two joins the softmax scale, so a
// score is formed at up to 2^9 times a step and steps above 2^118 would overflow.
// Outputs: p and the steps are fp16 (steps relative to the largest of their group that the warp
// has met, times 2^10), and so is their product: two roundings of 2^-11 (a step's 8 bits are exact),
// each an eighth of what bf16 would cost; products below 2^-24 of the largest step lose digits.  The
// mid term is a bf16 MMA with the mids, which are bf16, as four more columns, and p rounded to
// bf16: 2^-8 of each key's share, against a row sum of unrounded p.  Where V has channels with
// offsets the mids carry most of the value, so this is the largest rounding of the call (fp16 has no
// room for mids, whose range is bf16's).  The roundings of different keys are independent and add up
// to less than the output's own to bf16: against fp64 the outputs of the measured cases are off as
// much as fp32 sums rounded to bf16 are.
// fp32 queries take the same kernel with q, p and p * step split in two fp16 parts (22 bits) and
// the mid term's p in three of bf16 (24 bits), a product each: 24.9 us where bf16 takes 17.5 (8 x
// 128K, 16 heads a group); fp32 arithmetic on the CUDA cores took 158.
//
// CTA = one split of a (sequence, KV head), three groups of four warps that take its blocks in
// turn, 32 keys a warp, each warp with a softmax base of its own that moves only when a row's
// maximum passes it by more than 4 (log2 units).  Whole records (K and V of a block, 160 D
// contiguous bytes) come through a ring, one bulk copy each; a group's first warp refills a
// stage in the middle of its next block, when the other warps have left the stage.  Q's
// operands are read from shared memory for every 16 keys; the outputs stay in registers, which
// twelve warps leave enough of (168 a thread; sixteen warps of 128 spilled and gained nothing).
//
// What bounds it (8 x 1M, 64 blocks a head, 18.7 us, 42 MB, 2.3 TB/s): of a CTA's 17 us, with
// sixteen blocks each, 2.5 pass before its first block has arrived, 11.5 in the loop and 3 in
// the merge.  The loop issues some 900 instructions a warp and block; 62 % of the issue slots
// are used, the tensor pipe (mma.sync) 38 % and the ALUs 44 %: without the second product the
// call takes 14.9 us, without the first 14.3, so about 10.5 are the memory's and the ends'.
//
// The CTAs of a cluster end by writing their partial outputs, maxima and sums into each
// other's shared memory (each owns a share of the rows), so after one cluster barrier
// everything is local.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "launch.cuh"
#include "packed_cache.cuh"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace msa {

namespace {

constexpr int kRows = 16;              // query heads of a pass
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kMmaGroups = 3;                              // groups of warps
constexpr int kGroupWarps = 4;
constexpr int kMmaWarps = kMmaGroups * kGroupWarps;
constexpr int kMmaThreads = kMmaWarps * 32;
constexpr int kMaxSplits = 16;         // CTAs of a cluster
constexpr int kMaxList = 1024;         // selection entries of a split that are listed at once
constexpr int kMaxMassList = 128;      // blocks of a split whose weights are kept
constexpr float kSlack = 4.f;          // p <= 2^4
constexpr int kStepShift = 10;         // steps below 2^11: p * step < 2^15 in fp16
constexpr uint32_t kMinStepExp = 27;   // biased exponent of the smallest step, 2^-100

struct Entry {
  int phys, seen, blk;
};

// kParts: fp16 parts of q (1 for bf16 queries, 2 for fp32).
template <int D, int kParts>
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
  uint4 qf[kParts][kGroups][2][32];    // Q as A operands, per lane
  float qsum[kGroups][kRows];          // sums of q over a group of dims
  float cr[kRows];                     // score units to log2 units
  __half vstep[kMmaWarps][kGroups][32];                    // V's steps of a warp's keys
  float wm[kMmaWarps][kRows], wl[kMmaWarps][kRows];
  uint64_t full[kStages], empty[kStages];
  int last[kStages];                   // a stage's last copy
  int abort, count, lost;              // lost: some CTA of the cluster gave up a wait
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

__device__ __forceinline__ uint32_t load_u16(const void* p) {
  return *reinterpret_cast<const uint16_t*>(p);
}
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

// A lane's part of a query row: of each group of dims eight values (all loads in flight together),
// the largest magnitude's fp32 bits, and the eight of one group.
template <typename T, int NG> struct RowPart;
template <int NG> struct RowPart<__nv_bfloat16, NG> {
  uint4 w[NG];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
#pragma unroll
    for (int x = 0; x < NG; ++x) w[x] = *reinterpret_cast<const uint4*>(p + x * kPackedGroup);
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int x = 0; x < NG; ++x) {
      const uint32_t v[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
      for (int u = 0; u < 4; ++u) m = max(m, max(v[u] & 0x7fffu, (v[u] >> 16) & 0x7fffu));
    }
    return m << 16;
  }
  __device__ __forceinline__ void group(int g, float* x) const {
    uint4 v = w[0];
#pragma unroll
    for (int y = 1; y < NG; ++y)
      if (g == y) v = w[y];
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = lo_bf16(u[i]);
      x[2 * i + 1] = hi_bf16(u[i]);
    }
  }
};
template <int NG> struct RowPart<float, NG> {
  float w[NG][8];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int x = 0; x < NG; ++x) {
      Vec16<float>::load(p + x * kPackedGroup, w[x]);
      Vec16<float>::load(p + x * kPackedGroup + 4, w[x] + 4);
    }
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
#pragma unroll
    for (int x = 0; x < NG; ++x)
#pragma unroll
      for (int u = 0; u < 8; ++u) m = max(m, __float_as_uint(w[x][u]) & 0x7fffffffu);
    return m;
  }
  __device__ __forceinline__ void group(int g, float* x) const {
#pragma unroll
    for (int y = 0; y < NG; ++y)
      if (g == y)
#pragma unroll
        for (int u = 0; u < 8; ++u) x[u] = w[y][u];
  }
};
__device__ __forceinline__ void store_pair(__nv_bfloat16* p, float2 v) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
}
__device__ __forceinline__ void store_pair(float* p, float2 v) {
  *reinterpret_cast<float2*>(p) = v;
}
// What fp16 leaves of a pair.
__device__ __forceinline__ uint32_t f16_rest(float lo, float hi, uint32_t pair) {
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&pair));
  return f16_pair(lo - v.x, hi - v.y);
}

template <typename T, int D, bool kMass>
__global__ void __launch_bounds__(kMmaThreads, 1)
packed_decode_mma(const T* __restrict__ q, const uint8_t* __restrict__ cache,
                  const int32_t* __restrict__ sel, T* __restrict__ out, float* __restrict__ lse,
                  float* __restrict__ mass, Dims p, int per, int* status) {
  constexpr bool kWide = sizeof(T) == 4;                   // fp32 queries
  using R = PackedRecord<D>;
  using S = MmaSmem<D, kWide ? 2 : 1>;
  constexpr int NG = R::kGroups, kStages = S::kStages;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  S& s = *reinterpret_cast<S*>(smem_raw);
  Entry* list = reinterpret_cast<Entry*>(smem_raw + sizeof(S));   // [min(per, kMaxList)]
  // kMass only: log-sums [kGroupWarps][per][kRows], and the blocks' weights so far [per]
  float* weights = reinterpret_cast<float*>(list + per);
  float* total = weights + kGroupWarps * per * kRows;
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

  // more than 16 heads of a group: one pass after the other, weights added up in order and to mass
  // in the last
  int first = 0;                                           // copies made so far
  for (int h0 = 0; h0 < p.G; h0 += kRows) {
    const int rows = min(kRows, p.G - h0);
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
    bool ok = true;
    int n_blocks = 0;
    float cr[2];
    uint32_t qs[4];
    // the split's selection entries, kMaxList a round (one round but for rows of thousands)
    for (int round = 0;; ++round) {
      if (warp == kMmaWarps - 1) {
        // the blocks, in order, without entries that are no block of the sequence
        const int from = split * per + round * kMaxList;
        const int32_t* entry = sel + (size_t)bg * p.k + from;
        const int entries = min(min(p.k - split * per, per) - round * kMaxList, kMaxList);
        int blk = lane < entries ? entry[lane] : -1;
        const int L = seq_len_of(p, b), nB_b = (L + kPackedBlock - 1) / kPackedBlock;
        if (h0 == 0 && round == 0 && lane == 0) {          // while the loads are in flight
          for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(&s.full[i], 1);
            ptx::mbar_init(&s.empty[i], kGroupWarps);
            s.last[i] = -1;
          }
          s.abort = s.lost = 0;
          ptx::fence_barrier_init();
        }
        int n = 0;
        for (int i = 0; i < entries; i += 32) {
          const int phys = blk >= 0 && blk < nB_b ? physical_block(p, b, blk) : -1;
          const uint32_t there = __ballot_sync(0xffffffffu, phys >= 0);
          if (phys >= 0)
            list[n + __popc(there & ((1u << lane) - 1))] =
                Entry{phys, min(kPackedBlock, L - blk * kPackedBlock), blk};
          n += __popc(there);
          blk = i + 32 + lane < entries ? entry[i + 32 + lane] : -1;
        }
        if (lane == 0) s.count = n;
        __syncwarp();
        const int now = p.inject == 2 && split == 0 ? min(n, 1) : n;   // test hook: one copy
        if (lane < min(now, kStages) && !*abort) {
          // the first copies, a lane each; every stage is empty here
          const int x = first + lane, st = x % kStages;
          s.last[st] = x;
          ptx::mbar_arrive_expect_tx(&s.full[st], R::kPairBytes);
          ptx::bulk_load(s.ring[st], cache + ((size_t)list[lane].phys * p.Hkv + g) * R::kPairBytes,
                         R::kPairBytes, &s.full[st]);
        }
        __syncwarp();
      }
      // Q as A operands, dims in the order of the codes in K's words: of group x, k-step kk holds
      // dims 32 x + 8 c + (2 kk, 2 kk + 4) and (2 kk + 1, 2 kk + 5); rows gr and gr + 8
      if (round == 0 && warp < NG) {
        const T* q0 = q + ((size_t)b * p.Hq + (size_t)g * p.G + h0) * D;
        uint32_t f[2][2][4];                                 // [part][k-step][register]
        RowPart<T, NG> part[2];
        // rows past the last head repeat it and count as zero
#pragma unroll
        for (int r = 0; r < 2; ++r)
          part[r].load(q0 + (size_t)min(gr + 8 * r, rows - 1) * D + c * 8);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = gr + 8 * r;
          uint32_t top = row < rows ? part[r].top() : 0u;  // largest |q| of the row
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const uint32_t e = min(max(top >> 23, 1u), 253u);
          const float down = __uint_as_float((254u - e) << 23);
          float w[8];
          part[r].group(warp, w);
#pragma unroll
          for (int u = 0; u < 8; ++u) w[u] = row < rows ? w[u] * down : 0.f;
          // dims (0, 4) (1, 5) and (2, 6) (3, 7)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint32_t hi = f16_pair(w[u], w[u + 4]);
            f[0][u / 2][2 * (u & 1) + r] = hi;
            f[1][u / 2][2 * (u & 1) + r] = kWide ? f16_rest(w[u], w[u + 4], hi) : 0u;
          }
          float t = ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
          t += __shfl_xor_sync(0xffffffffu, t, 1);
          t += __shfl_xor_sync(0xffffffffu, t, 2);
          if (c == 0) s.qsum[warp][row] = t;
          if (warp == 0 && c == 0) s.cr[row] = c1 * __uint_as_float(e << 23);
        }
#pragma unroll
        for (int u = 0; u < (kWide ? 2 : 1); ++u)
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
            s.qf[u][warp][kk][lane] =
                make_uint4(f[u][kk][0], f[u][kk][1], f[u][kk][2], f[u][kk][3]);
      }
      __syncthreads();
      n_blocks = s.count;
      if (round == 0) {
        cr[0] = s.cr[gr];
        cr[1] = s.cr[gr + 8];
        // the group sums of q in three bf16 parts: k = part * NG + group
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
      }
      ok = !*abort;
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
            t[x] = load_u16(vr + R::plane(R::kStepOffset, key0 + lane, x));
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
            const uint32_t mids = load_u16(kr + R::plane(R::kMidOffset, key, x)) |
                                  load_u16(kr + R::plane(R::kMidOffset, key, x + 1)) << 16;
            mma_new<true>(sc[2 * half + u], qs, mids, mids);
          }
#pragma unroll
          for (int y = 0; y < NG; ++y) {
            const uint4 v0 = s.qf[0][y][0][lane], v1 = s.qf[0][y][1][lane];
            const uint32_t a0[4] = {v0.x, v0.y, v0.z, v0.w}, a1[4] = {v1.x, v1.y, v1.z, v1.w};
            const uint4 z0 = s.qf[kWide][y][0][lane], z1 = s.qf[kWide][y][1][lane];
            const uint32_t b0[4] = {z0.x, z0.y, z0.z, z0.w}, b1[4] = {z1.x, z1.y, z1.z, z1.w};
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              float acc[4];
              const uint32_t w8 = w[u][y] >> 8;
              mma_new<false>(acc, a0, codes.lows(w[u][y]), codes.highs(w[u][y]));
              mma_add<false>(acc, a1, codes.lows(w8), codes.highs(w8));
              if (kWide) {
                mma_add<false>(acc, b0, codes.lows(w[u][y]), codes.highs(w[u][y]));
                mma_add<false>(acc, b1, codes.lows(w8), codes.highs(w8));
              }
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
            weights[(gw * per + i) * kRows + gr + 8 * c] =
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
            uint32_t pb[4] = {bf16_pair(p0[0], p0[1]), bf16_pair(p0[2], p0[3]),
                              bf16_pair(p1[0], p1[1]), bf16_pair(p1[2], p1[3])};
            mma_add<true>(om, pb, m0, m1);
            if (kWide) {                                     // p in two more parts
              float rest[8] = {p0[0], p0[1], p0[2], p0[3], p1[0], p1[1], p1[2], p1[3]};
#pragma unroll
              for (int part = 0; part < 2; ++part) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                  rest[2 * u] -= lo_bf16(pb[u]);
                  rest[2 * u + 1] -= hi_bf16(pb[u]);
                  pb[u] = bf16_pair(rest[2 * u], rest[2 * u + 1]);
                }
                mma_add<true>(om, pb, m0, m1);
              }
            }
          }
          const uint32_t ph[4] = {f16_pair(p0[0], p0[1]), f16_pair(p0[2], p0[3]),
                                  f16_pair(p1[0], p1[1]), f16_pair(p1[2], p1[3])};
#pragma unroll
          for (int x = 0; x < NG; ++x) {
            const uint32_t s0 = load_u32(&s.vstep[warp][x][ks * 16 + 2 * c]);
            const uint32_t s1 = load_u32(&s.vstep[warp][x][ks * 16 + 8 + 2 * c]);
            uint32_t pa[4], pr[4];                           // p * step, and what fp16 leaves of it
            if (kWide) {
              const float2 t0 = __half22float2(*reinterpret_cast<const __half2*>(&s0));
              const float2 t1 = __half22float2(*reinterpret_cast<const __half2*>(&s1));
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const float* pu = u < 2 ? p0 + 2 * u : p1 + 2 * (u - 2);
                const float2 tu = u < 2 ? t0 : t1;
                const float lo = pu[0] * tu.x, hi = pu[1] * tu.y;
                pa[u] = f16_pair(lo, hi);
                pr[u] = f16_rest(lo, hi, pa[u]);
              }
            } else {
              pa[0] = mul_f16x2(ph[0], s0);
              pa[1] = mul_f16x2(ph[1], s0);
              pa[2] = mul_f16x2(ph[2], s1);
              pa[3] = mul_f16x2(ph[3], s1);
            }
            // the group's 16 bits of the two keys of each pair, a byte (two dims) at a time
            const int word = x / 2, byte = 2 * (x & 1);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t pick =
                  (uint32_t)(byte + y) * 0x0011u | (uint32_t)(4 + byte + y) * 0x1100u;
              const uint32_t a = __byte_perm(va[word], va[NG / 2 + word], pick);
              const uint32_t e = __byte_perm(vb[word], vb[NG / 2 + word], pick);
              mma_add<false>(o[4 * x + 2 * y], pa, codes.lows(a), codes.lows(e));
              mma_add<false>(o[4 * x + 2 * y + 1], pa, codes.highs(a), codes.highs(e));
              if (kWide) {
                mma_add<false>(o[4 * x + 2 * y], pr, codes.lows(a), codes.lows(e));
                mma_add<false>(o[4 * x + 2 * y + 1], pr, codes.highs(a), codes.highs(e));
              }
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
      first += n_blocks;
      if (min(p.k - split * per, per) - round * kMaxList <= kMaxList) break;
      __syncthreads();                                       // the list is made anew
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
      // a warp without a base has a sum of 0, or NaN when all its scores are no numbers
      const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int w = 0; w < kMmaWarps; ++w) sum += ex2(s.wm[w][r] - ref) * s.wl[w][r];
      *cluster.map_shared_rank(&s.m[split][r], to) = top;
      // a sum below zero: this CTA gave up a wait
      *cluster.map_shared_rank(&s.l[split][r], to) = *abort ? -1.f : sum;
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
      bool gave_up = false;
      for (int x = 0; x < n_split; ++x) {
        top = fmaxf(top, s.m[x][r]);
        gave_up |= s.l[x][r] < 0.f;
      }
      const float ref = top == -INFINITY ? 0.f : top;
      for (int x = 0; x < n_split; ++x) sum += ex2(s.m[x][r] - ref) * s.l[x][r];
      // without all of the row's blocks: output 0, lse -inf, no weights
      s.norm[r] = sum == 0.f || gave_up ? -INFINITY : ref + __log2f(sum);
      if (gave_up) s.lost = 1;
      if (lse && split == 0 && r < rows)
        lse[(size_t)b * p.Hq + g * p.G + h0 + r] = s.norm[r] * kLn2;
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
      store_pair(out + ((size_t)b * p.Hq + g * p.G + h0 + r) * D + d0, v);
    }
    if (kMass)                                             // sixteen lanes a block, one a row; a
                                                           // lane meets its block in every pass
      for (int e0 = 0; e0 < n_blocks * kRows; e0 += kMmaThreads) {
        const int e = e0 + (int)threadIdx.x, i = e / kRows, r = e % kRows;
        float sum = 0.f;
        if (i < n_blocks && r < rows && s.norm[r] != -INFINITY)
#pragma unroll
          for (int w = 0; w < kGroupWarps; ++w)
            sum += ex2(weights[(w * per + i) * kRows + r] - s.norm[r]);
#pragma unroll
        for (int x = kRows / 2; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        if (r == 0 && i < n_blocks) {
          if (h0 > 0) sum += total[i];
          if (h0 + kRows < p.G) total[i] = sum;
          else if (!s.lost) atomicAdd(mass + (size_t)bg * p.nB + list[i].blk, sum);
        }
      }
    if (h0 + kRows < p.G) {
      // the next pass copies into the memory that held the warps' outputs, and the others
      // write into this CTA's
      ptx::fence_proxy_async_smem();
      cluster.sync();
    }
  }
}

template <typename T, int D, bool kMass>
cudaError_t decode_mma(const Dims& p, const void* q, const void* cache, const int32_t* sel,
                       void* out, float* lse, float* mass, cudaStream_t st, int* status) {
  // CTAs that share a (sequence, KV head): as many as leave each an entry while all clusters run
  // at once.  One CTA fills an SM, and 76, 36, 15 and 7 clusters of 2, 4, 8 and 16 of them fit
  // this GPU's processor clusters (the occupancy calculator's figures).  16 clusters of 8 ran in
  // two waves and took 21.9 us where 16 of 4 take 17.2; 4 of 16 take 9.2 where 4 of 8 took 11.4.
  const int units = p.B * p.Hkv;
  int n_split = units <= 7 ? 16 : units <= 15 ? 8 : units <= 36 ? 4 : units <= 76 ? 2 : 1;
  while (n_split > p.k) n_split /= 2;
  // with weights, as many as their lists need
  if (kMass)
    while (n_split < kMaxSplits && (p.k - 1) / n_split >= kMaxMassList) n_split *= 2;
  static_assert(kMaxPackedMassBlocks <= kMaxSplits * kMaxMassList, "lists of weights");
  const int per = (p.k - 1) / n_split + 1, listed = per < kMaxList ? per : kMaxList;
  const size_t smem = sizeof(MmaSmem<D, sizeof(T) == 4 ? 2 : 1>) + sizeof(Entry) * listed +
                      (kMass ? sizeof(float) * (kGroupWarps * kRows + 1) * per : 0);
  // the kernel's limit is set to the same value by every call: host threads share it, and one with
  // short lists must not lower it between another's setting and its launch
  constexpr size_t kLargest = sizeof(MmaSmem<D, sizeof(T) == 4 ? 2 : 1>) +
                              (kMass ? kMaxMassList * (sizeof(Entry) + 4 * kGroupWarps * kRows + 4)
                                     : kMaxList * sizeof(Entry));
  static_assert(kLargest <= 227 * 1024, "shared memory of a CTA");
  auto kern = packed_decode_mma<T, D, kMass>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)kLargest);
  if (e == cudaSuccess && n_split > 8)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  return launch_after(kern, dim3(n_split, p.B * p.Hkv), kMmaThreads, smem, n_split, st,
                      (const T*)q, (const uint8_t*)cache, sel, (T*)out, lse, mass, p, per, status);
}

template <typename T>
cudaError_t decode(const Dims& p, const void* q, const void* cache, const int32_t* sel, void* out,
                   float* lse, float* mass, cudaStream_t st, int* status) {
  if (p.d == 128)
    return mass ? decode_mma<T, 128, true>(p, q, cache, sel, out, lse, mass, st, status)
                : decode_mma<T, 128, false>(p, q, cache, sel, out, lse, mass, st, status);
  return mass ? decode_mma<T, 64, true>(p, q, cache, sel, out, lse, mass, st, status)
              : decode_mma<T, 64, false>(p, q, cache, sel, out, lse, mass, st, status);
}

}  // namespace

cudaError_t launch_sparse_decode_packed(const Dims& p, const void* q, const void* cache,
                                        const int32_t* sel, void* out, float* lse, float* mass,
                                        cudaStream_t st, int* dev_status) {
  if (p.dtype == 1)
    return decode<__nv_bfloat16>(p, q, cache, sel, out, lse, mass, st, dev_status);
  return decode<float>(p, q, cache, sel, out, lse, mass, st, dev_status);
}

}  // namespace msa
