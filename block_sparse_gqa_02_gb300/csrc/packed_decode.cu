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
// codes become exact bf16 integers -8 .. 7 (a code or-ed into the mantissa of 128 and 136 taken
// away), so products with them lose nothing, and steps and mids enter in fp32:
//   z_j = sum_g step_jg (q_g . c_jg) + sum_g mid_jg (sum of q_g),
//   o_g = sum_j (p_j step_jg) c_jg + sum_j p_j mid_jg.
// The scores take one accumulator per group of dims; their mid term is one more MMA whose A
// operand is the rows' group sums of q, split in three bf16 parts (24 bits).  For the output
// p_j step_jg is formed in fp32 and rounded once to bf16, as the 16-bit cache's kernel rounds
// p_j; the mid term is an MMA with the mids as four more columns.
//
// CTA = one split of a (sequence, KV head): a producer warp lists the split's blocks and keeps a
// ring of whole records (K and V of a block, 160 D contiguous bytes, one bulk copy) filled;
// four warps take 32 keys of every block each, with a softmax base of their own that moves only
// when a row's maximum passes it by more than 8 (log2 units).

constexpr int kMmaWarps = 4;
constexpr int kMmaThreads = (kMmaWarps + 1) * 32;
constexpr int kMaxList = 1024;         // blocks of a split
constexpr int kMaxMassList = 128;      // blocks of a split whose weights are kept
constexpr float kSlack = 8.f;

struct Entry {
  int phys, seen, blk;
};

template <int D>
struct MmaSmem {
  static constexpr int kStages = D == 128 ? 5 : 8;
  union {
    __align__(128) uint8_t ring[kStages][PackedRecord<D>::kPairBytes];
    float part[kMmaWarps][kRows][D + 4];                   // the warps' outputs, after the ring
  };
  float o[kRows][D];                   // the CTA's outputs, relative to m
  float m[kRows], l[kRows], norm[kRows];
  float wm[kMmaWarps][kRows], wl[kMmaWarps][kRows];
  uint64_t full[kStages], empty[kStages];
  int abort, count;
};

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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

__device__ __forceinline__ float lo_bf16(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// Keeps the halves of a pair of keys (j, j + 1) that lie before `seen`.
__device__ __forceinline__ uint32_t keep_seen(uint32_t pair, int j, int seen) {
  return pair & ((j < seen ? 0xffffu : 0u) | (j + 1 < seen ? 0xffff0000u : 0u));
}

template <int D, bool kMass>
__global__ void __launch_bounds__(kMmaThreads)
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
  float* weights = reinterpret_cast<float*>(list + per);   // [kMmaWarps][kRows][per], kMass only
  cg::cluster_group cluster = cg::this_cluster();
  const int split = (int)cluster.block_rank(), n_split = (int)cluster.num_blocks();
  const int bg = blockIdx.y, b = bg / p.Hkv, g = bg % p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gr = lane >> 2, c = lane & 3;
  const volatile int* abort = &s.abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&s.full[i], 1);
      ptx::mbar_init(&s.empty[i], kMmaWarps);
    }
    s.abort = 0;
    ptx::fence_barrier_init();
  }
  if (warp == kMmaWarps) {
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
  }
  __syncthreads();
  const int n_blocks = s.count;
  const float c1 = p.sm_scale * kLog2e;
  int issued = 0, taken = 0;                               // blocks copied, blocks consumed

  // more than 16 heads of a group: one pass after the other, weights added up in order
  for (int h0 = 0; h0 < p.G; h0 += kRows) {
    const int rows = min(kRows, p.G - h0);
    float o[4 * NG][4], om[4];
    float base[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 4 * NG; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
    om[0] = om[1] = om[2] = om[3] = 0.f;

    if (warp == kMmaWarps) {
      // ------------------------------------------------------------------- producer
      bool ok = !*abort;
      for (int i = 0; ok && i < n_blocks; ++i) {
        const int st = issued % kStages;
        ok = ptx::mbar_wait(&s.empty[st], ((issued / kStages) & 1) ^ 1, abort);
        if (!ok) break;
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(&s.full[st], R::kPairBytes);
          ptx::bulk_load(s.ring[st], cache + ((size_t)list[i].phys * p.Hkv + g) * R::kPairBytes,
                         R::kPairBytes, &s.full[st]);
        }
        ++issued;
        __syncwarp();
      }
      if (!ok && lane == 0) {
        s.abort = 1;
        if (status) atomicExch(status, 0x411);
      }
    } else {
      // -------------------------------------------------------------- compute warps
      // Q as A operands, dims in the order of the codes in K's words: of group x, k-step kk
      // holds dims 32 x + 8 c + (2 kk, 2 kk + 4) and (2 kk + 1, 2 kk + 5)
      uint32_t qa[NG][2][4], qs[4];
      {
        float sum[2][NG];
        const __nv_bfloat16* q0 = q + ((size_t)b * p.Hq + (size_t)g * p.G + h0) * D;
#pragma unroll
        for (int x = 0; x < NG; ++x)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int row = gr + 8 * r;
            const uint4 w = row < rows ? *reinterpret_cast<const uint4*>(q0 + (size_t)row * D +
                                                                        x * kPackedGroup + c * 8)
                                       : make_uint4(0, 0, 0, 0);
            // dims (0,1) (2,3) (4,5) (6,7) -> (0,4) (1,5) (2,6) (3,7)
            qa[x][0][r] = __byte_perm(w.x, w.z, 0x5410);
            qa[x][0][2 + r] = __byte_perm(w.x, w.z, 0x7632);
            qa[x][1][r] = __byte_perm(w.y, w.w, 0x5410);
            qa[x][1][2 + r] = __byte_perm(w.y, w.w, 0x7632);
            float t = lo_bf16(w.x) + hi_bf16(w.x) + lo_bf16(w.y) + hi_bf16(w.y) + lo_bf16(w.z) +
                      hi_bf16(w.z) + lo_bf16(w.w) + hi_bf16(w.w);
            t += __shfl_xor_sync(0xffffffffu, t, 1);
            t += __shfl_xor_sync(0xffffffffu, t, 2);
            sum[r][x] = t;
          }
        // the three parts of the sums: k = part * NG + group
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float part[3][NG];
#pragma unroll
          for (int x = 0; x < NG; ++x) {
            part[0][x] = __bfloat162float(__float2bfloat16_rn(sum[r][x]));
            part[1][x] = __bfloat162float(__float2bfloat16_rn(sum[r][x] - part[0][x]));
            part[2][x] = sum[r][x] - part[0][x] - part[1][x];
          }
          if (NG == 4) {
            const int x = 2 * (c & 1);
            const float lo = c < 2 ? (x ? part[0][2 % NG] : part[0][0])
                                   : (x ? part[1][2 % NG] : part[1][0]);
            const float hi = c < 2 ? (x ? part[0][3 % NG] : part[0][1])
                                   : (x ? part[1][3 % NG] : part[1][1]);
            qs[r] = bf16_pair(lo, hi);
            qs[2 + r] = c < 2 ? bf16_pair(x ? part[2][2 % NG] : part[2][0],
                                          x ? part[2][3 % NG] : part[2][1])
                              : 0u;
          } else {
            qs[r] = c == 0 ? bf16_pair(part[0][0], part[0][1])
                    : c == 1 ? bf16_pair(part[1][0], part[1][1])
                    : c == 2 ? bf16_pair(part[2][0], part[2][1]) : 0u;
            qs[2 + r] = 0u;
          }
        }
      }
      bool ok = !*abort;
      for (int i = 0; ok && i < n_blocks; ++i) {
        const int st = taken % kStages;
        ok = ptx::mbar_wait(&s.full[st], (taken / kStages) & 1, abort);
        if (!ok) break;
        const uint8_t* kr = s.ring[st];
        const uint8_t* vr = kr + R::kBytes;
        const int seen = list[i].seen;
        const int key0 = warp * 32;
        // scores of 16 rows x 32 keys
        float sc[4][4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          const int key = key0 + nt * 8 + gr;              // this lane's key as a B column
          const int col = key0 + nt * 8 + 2 * c;           // its keys as accumulator columns
          uint32_t w[NG];
          if (NG == 4) {
            const uint4 u = *reinterpret_cast<const uint4*>(kr + R::k_word(key, 0, c));
            w[0] = u.x, w[1] = u.y, w[2 % NG] = u.z, w[3 % NG] = u.w;
          } else {
            const uint2 u = *reinterpret_cast<const uint2*>(kr + R::k_word(key, 0, c));
            w[0] = u.x, w[1] = u.y;
          }
          const int x = NG == 4 ? 2 * (c & 1) : 0;
          const uint32_t mids =
              *reinterpret_cast<const uint16_t*>(kr + R::plane(R::kMidOffset, key, x)) |
              (uint32_t)*reinterpret_cast<const uint16_t*>(kr + R::plane(R::kMidOffset, key, x + 1))
                  << 16;
          float acc[NG][4];
          sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
          mma_16816(sc[nt], qs, mids, mids);
#pragma unroll
          for (int y = 0; y < NG; ++y) {
            acc[y][0] = acc[y][1] = acc[y][2] = acc[y][3] = 0.f;
            mma_16816(acc[y], qa[y][0], code_pair(w[y]), code_pair(w[y] >> 4));
            mma_16816(acc[y], qa[y][1], code_pair(w[y] >> 8), code_pair(w[y] >> 12));
          }
#pragma unroll
          for (int y = 0; y < NG; ++y) {
            const uint32_t st2 =
                *reinterpret_cast<const uint32_t*>(kr + R::plane(R::kStepOffset, col, y));
            const float s0 = lo_bf16(st2), s1 = hi_bf16(st2);
            sc[nt][0] = fmaf(acc[y][0], s0, sc[nt][0]);
            sc[nt][1] = fmaf(acc[y][1], s1, sc[nt][1]);
            sc[nt][2] = fmaf(acc[y][2], s0, sc[nt][2]);
            sc[nt][3] = fmaf(acc[y][3], s1, sc[nt][3]);
          }
          if (seen < kPackedBlock) {                       // whatever the unused bytes held
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
        // -inf * 0 of a zero scale is no number: such rows stay at -inf
        if (!(mx[0] > -INFINITY)) mx[0] = -INFINITY;
        if (!(mx[1] > -INFINITY)) mx[1] = -INFINITY;
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
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            sc[nt][0] = ex2(fmaf(sc[nt][0], c1, -b0));
            sc[nt][1] = ex2(fmaf(sc[nt][1], c1, -b0));
            sc[nt][2] = ex2(fmaf(sc[nt][2], c1, -b1));
            sc[nt][3] = ex2(fmaf(sc[nt][3], c1, -b1));
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
            weights[(warp * kRows + gr + 8 * c) * per + i] =
                bs == -INFINITY ? -INFINITY : bs + __log2f(sm);
        }
        // outputs: 16 keys a step
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const int key = key0 + ks * 16 + 2 * c;          // keys key, key + 1, key + 8, key + 9
          const int pair = key / 2;
          const uint8_t* v0 = vr + R::v_half(2 * pair, 0, gr);
          const uint8_t* v1 = vr + R::v_half(2 * (pair + 4), 0, gr);
          uint32_t va[NG], vb[NG];                         // NG / 2 words of each key of the pair
          if (NG == 4) {
            const uint4 u = *reinterpret_cast<const uint4*>(v0);
            const uint4 t = *reinterpret_cast<const uint4*>(v1);
            va[0] = u.x, va[1] = u.y, va[2 % NG] = u.z, va[3 % NG] = u.w;
            vb[0] = t.x, vb[1] = t.y, vb[2 % NG] = t.z, vb[3 % NG] = t.w;
          } else {
            const uint2 u = *reinterpret_cast<const uint2*>(v0);
            const uint2 t = *reinterpret_cast<const uint2*>(v1);
            va[0] = u.x, va[1] = u.y;
            vb[0] = t.x, vb[1] = t.y;
          }
          const float* p0 = sc[2 * ks];
          const float* p1 = sc[2 * ks + 1];
          {
            uint32_t m0 = 0, m1 = 0;                       // mids of group gr as column gr
            if (gr < NG) {
              m0 = *reinterpret_cast<const uint32_t*>(vr + R::plane(R::kMidOffset, key, gr));
              m1 = *reinterpret_cast<const uint32_t*>(vr + R::plane(R::kMidOffset, key + 8, gr));
              if (seen < kPackedBlock) {
                m0 = keep_seen(m0, key, seen);
                m1 = keep_seen(m1, key + 8, seen);
              }
            }
            const uint32_t pa[4] = {bf16_pair(p0[0], p0[1]), bf16_pair(p0[2], p0[3]),
                                    bf16_pair(p1[0], p1[1]), bf16_pair(p1[2], p1[3])};
            mma_16816(om, pa, m0, m1);
          }
#pragma unroll
          for (int x = 0; x < NG; ++x) {
            uint32_t w0 = *reinterpret_cast<const uint32_t*>(vr + R::plane(R::kStepOffset, key, x));
            uint32_t w1 =
                *reinterpret_cast<const uint32_t*>(vr + R::plane(R::kStepOffset, key + 8, x));
            if (seen < kPackedBlock) {
              w0 = keep_seen(w0, key, seen);
              w1 = keep_seen(w1, key + 8, seen);
            }
            const float s0 = lo_bf16(w0), s1 = hi_bf16(w0), s2 = lo_bf16(w1), s3 = hi_bf16(w1);
            const uint32_t pa[4] = {
                bf16_pair(p0[0] * s0, p0[1] * s1), bf16_pair(p0[2] * s0, p0[3] * s1),
                bf16_pair(p1[0] * s2, p1[1] * s3), bf16_pair(p1[2] * s2, p1[3] * s3)};
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
        ++taken;
      }
      if (!ok && lane == 0) {
        s.abort = 1;
        if (status) atomicExch(status, 0x412);
      }
    }
    // Every warp has left its loop.  Without an abort every copy has been consumed; after one,
    // the producer waits for its last copies before the ring's memory is used again.
    __syncthreads();
    if (warp == kMmaWarps && lane == 0 && *abort)
      for (int x = issued > kStages ? issued - kStages : 0; x < issued; ++x)
        ptx::mbar_wait_timed(&s.full[x % kStages], (x / kStages) & 1);
    __syncthreads();
    if (warp < kMmaWarps) {
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
            for (int w = 0; w < kMmaWarps; ++w)
              sum += ex2(weights[(w * kRows + r) * per + i] - s.norm[r]);
        if (!*abort) atomicAdd(mass + (size_t)bg * p.nB + list[i].blk, sum);
      }
    // the next pass copies into the memory that held the warps' outputs
    if (h0 + kRows < p.G) ptx::fence_proxy_async_smem();
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
                      (kMass ? sizeof(float) * kMmaWarps * kRows * per : 0);
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
  while (n < 8 && 2 * n <= p.k && 2 * n * p.B * p.Hkv <= 2 * 152) n *= 2;
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
