// Index scores of drafted tokens on the tcgen05 tensor cores (bf16 queries, index_dim 128, blocks
// of 128 keys, 8-bit or 16-bit index keys): every token's index queries against every cached index
// key, max-pooled per block, and against the keys of its path.
//
// The scan is to be bound by HBM: a key is read once for all tokens, 129 bytes in 8 bits.  Each CTA
// streams a contiguous range of one sequence's blocks through a TMA ring; a thread issues a
// block's products with the 128 keys as M and the columns (token, head) as N, so that the cost
// follows the number of tokens.  8-bit keys are operands as they lie in the cache: a key's scale is
// a power of two of its own and is applied to the products.  The queries keep their precision by
// being split in three 8-bit parts, x 2^-e = hi + mid + lo, each the nearest e5m2 value (3 significant
// bits, 2^-16 to 57344) to what the ones before leave.  A bf16 value is m units of its last bit,
// m < 2^8: hi leaves at most 16 units, mid at most one, lo nothing.  That holds while the last bit
// is 2^-16 or more; with the largest dim scaled to (28672, 57344] it is so for dims of at least 2^-9,
// 2^-23.8 of the largest.  A smaller dim is off by at most 2^-17, 2^-31.8 of the largest.  (Two e4m3
// parts, a third less of products, keep the digits to 2^-9.8 of the largest only: one large dim then
// costs the others theirs.)  All parts accumulate in the same TMEM columns.
//
// Two groups of four epilogue warps take the blocks in turn (one group's chain of waits and loads
// is longer than a block's share of the bandwidth).  They read the accumulator as fragments of 16
// keys x 8 columns, in which a thread holds four keys of a column: scale, maximum over the four,
// then over the lanes by halving (4 shuffles for 16 columns).  The maxima of eight blocks collect in
// one of two buffers, which two further warps write out, 32 bytes of a score row at a time.
// Warps: 0-7 epilogue (group warp / 4, TMEM lane quadrant warp % 4), 8 TMA producer, 9-10 MMA
// issuers (every other block: one alone takes 58 us more), 11-12 writers.  Every wait is bounded.
// Measured: 16 drafts, 8-bit keys, 8 x 1M tokens 192 us (5.7 TB/s, 85 % of the copy bandwidth; two parts
// of the queries: 189; shared memory serves operands in 66 % of the cycles, the issue slots are 40 %
// busy); 32 drafts 258, 64 drafts 508; 12 drafts, 16-bit keys, ragged 8 x 128K 32 us (5.2 TB/s with 5 us
// of set-up); 5 drafts, 1 x 8K 10.5 us, of which a CTA's work is 5.
#include "index_cache.cuh"
#include "launch.cuh"
#include "ptx.cuh"
#include "tma_host.cuh"
#include "tree.cuh"
#include "tree_scores_tc.cuh"

namespace msa {

namespace {

constexpr int kBk = 128, kDI = 128, kRowBytes = 128;
constexpr int kAcc = 4;                // accumulators in TMEM
constexpr int kGroups = 2;             // of epilogue warps (four: 6 us more at 8 x 1M, 16 drafts)
constexpr int kIssuers = 2;            // warps that issue products
// A barrier's phases are told apart by parity, so each waiter has to see them one by one: what
// completes an accumulator's phases is waited for by one group and issued by one warp, and so is
// a stage's (the number of stages is a multiple of the issuers').
static_assert(kAcc % kGroups == 0 && kAcc % kIssuers == 0, "one group and issuer an accumulator");
constexpr int kProducerWarp = 4 * kGroups, kMmaWarp = kProducerWarp + 1;
constexpr int kWriterWarp = kMmaWarp + kIssuers, kWriters = 2;
constexpr int kWarps = kWriterWarp + kWriters, kThreads = kWarps * 32;
constexpr int kMaxCols = 128;          // UMMA N: four accumulators fill TMEM
constexpr int kMaxStages = 12;
constexpr int kScaleSlots = 16;        // a power of two, kMaxStages + kAcc or more: see the producer
static_assert(kScaleSlots >= kMaxStages + kAcc && (kScaleSlots & (kScaleSlots - 1)) == 0, "slots");
constexpr int kSmemLimit = 232448;
constexpr int kParts = 3;              // of a query beside 8-bit keys; 16-bit ones: two halves of the dims

// The small part of shared memory; the ring, the queries and the results lie before it.
struct Small {
  TreeWord path[64];
  TreeWord late;                       // tokens whose position is in the block after the first's
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full[kAcc], acc_empty[kAcc];
  uint64_t res_full[2], res_empty[2], dres_full;
  int b, blk0, nblk, rank, cnt;        // the CTA's range, and its place among the sequence's CTAs
  uint32_t tmem_base;
  int abort;
};

// Bytes of each part, all multiples of 16; cols: padded to 16.
struct Plan {
  int cols, stages, stage_bytes, q_tiles;                  // q_tiles: of cols x 128 bytes of queries
  __host__ __device__ int q_at() const { return stages * stage_bytes; }
  __host__ __device__ int ex_at() const { return q_at() + cols * q_tiles * kRowBytes; }
  __host__ __device__ int res_at() const { return ex_at() + kScaleSlots * kBk; }
  __host__ __device__ int res_row() const { return cols + 4; }          // spreads the banks
  __host__ __device__ int dres_at() const { return res_at() + 16 * res_row() * 4; }
  __host__ __device__ int scale_at() const { return dres_at() + 2 * cols * 4; }
  __host__ __device__ int row_at() const { return scale_at() + cols * 4; }
  __host__ __device__ int small_at() const { return row_at() + cols * 4; }
  __host__ __device__ int bytes() const { return small_at() + (int)sizeof(Small); }
};

__device__ __forceinline__ void raise_abort(Small& s, int* status, int code) {
  s.abort = 1;
  if (status) atomicExch(status, code);
}

__device__ __forceinline__ void arrive_n(uint64_t* bar, int n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(ptx::smem_u32(bar)), "r"(n)
               : "memory");
}

// The CTA's blocks: the CTAs are shared out in proportion to the sequences' block counts, each
// sequence getting at least one.  One warp.
__device__ __forceinline__ void find_range(const Dims& p, Small& s, int lane) {
  const int ctas = gridDim.x, c = blockIdx.x;              // ctas >= p.B
  if (lane == 0) {                                         // nothing, where every sequence is empty
    s.b = p.B - 1;
    s.blk0 = s.nblk = 0;
    s.rank = s.cnt = 1;
  }
  __syncwarp();
  if (ctas == p.B) {                                       // a CTA a sequence
    if (lane == 0) {
      s.b = c;
      s.rank = 0;
      s.nblk = (seq_len_of(p, c) + kBk - 1) / kBk;
    }
    return;
  }
  long long total = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    long long nb = b0 + lane < p.B ? (seq_len_of(p, b0 + lane) + kBk - 1) / kBk : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) nb += __shfl_xor_sync(0xffffffffu, nb, o);
    total += nb;
  }
  if (total < 1) total = 1;
  long long before = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    const int nb = b < p.B ? (seq_len_of(p, b) + kBk - 1) / kBk : 0;
    long long incl = nb;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const long long prefix = before + incl - nb;
    const int lo = b + (int)((ctas - p.B) * prefix / total);
    const int hi = b + 1 + (int)((ctas - p.B) * (prefix + nb) / total);
    if (b < p.B && c >= lo && c < hi) {                    // one lane of all
      const int cnt = hi - lo, per = (nb + cnt - 1) / cnt;
      s.b = b;
      s.rank = c - lo;
      s.cnt = cnt;
      s.blk0 = min(nb, s.rank * per);
      s.nblk = min(nb - s.blk0, per);
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
}

// Maximum over lane / 4 (the rows of a fragment) of values v[4 c + j], c < N (1, 2 or 4), of the
// columns 16 c + 2 (lane % 4) + {0, 1, 8, 9}[j].  Each step halves the values: the lane ends with
// those of column frag_col(lane) of chunk 2 i + (lane & 4 ? 1 : 0) in v[i] (one chunk: all lanes).
__device__ __forceinline__ int frag_col(int lane) {
  return (lane & 16 ? 8 : 0) + 2 * (lane & 3) + (lane & 8 ? 1 : 0);
}
template <int N>
__device__ __forceinline__ void frag_max(float (&v)[4 * N], int lane) {
  const bool u16 = lane & 16, u8 = lane & 8, u4 = lane & 4;
#pragma unroll
  for (int c = 0; c < N; ++c) {
    const float a = __shfl_xor_sync(0xffffffffu, u16 ? v[4 * c] : v[4 * c + 2], 16);
    const float b = __shfl_xor_sync(0xffffffffu, u16 ? v[4 * c + 1] : v[4 * c + 3], 16);
    v[4 * c] = fmaxf(u16 ? v[4 * c + 2] : v[4 * c], a);
    v[4 * c + 1] = fmaxf(u16 ? v[4 * c + 3] : v[4 * c + 1], b);
  }
#pragma unroll
  for (int c = 0; c < N; ++c) {
    const float a = __shfl_xor_sync(0xffffffffu, u8 ? v[4 * c] : v[4 * c + 1], 8);
    v[4 * c] = fmaxf(u8 ? v[4 * c + 1] : v[4 * c], a);
  }
  if (N == 1) {
    v[0] = fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], 4));
  } else {
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      const float a = __shfl_xor_sync(0xffffffffu, u4 ? v[4 * c] : v[4 * c + 4], 4);
      v[c / 2] = fmaxf(u4 ? v[4 * c + 4] : v[4 * c], a);
    }
  }
}

// Integers in the order of the floats, and back.
__device__ __forceinline__ int order_key(float x) {
  const int i = __float_as_int(x);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float from_order_key(int k) {
  return __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
}
constexpr int kNothing = (int)0x807fffff;                  // of -inf

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Two fp32 products with one factor.
__device__ __forceinline__ float2 mul2(uint32_t a, uint32_t b, uint64_t ss) {
  uint64_t x;
  float2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "r"(a), "r"(b));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(x) : "l"(ss));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}

// Maxima over a quadrant's 32 keys of N x 16 accumulator columns from `at` on, each key's products
// times its scale, joined into to[0 .. 16 N) (a maximum: no order of the warps shows).
template <int N, bool kScaled>
__device__ __forceinline__ void block_max(uint32_t at, const float (&sc)[4], int* to, int lane) {
  uint32_t a[N][8], d[N][8];                               // keys 0-15 and 16-31
#pragma unroll
  for (int c = 0; c < N; ++c) {
    ptx::tmem_ld_frag16(at + 16 * c, a[c]);
    ptx::tmem_ld_frag16(at + (16u << 16) + 16 * c, d[c]);
  }
  uint64_t ss[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) asm("mov.b64 %0, {%1, %1};" : "=l"(ss[r]) : "f"(sc[r]));
  ptx::tmem_ld_wait();
  float v[4 * N];
#pragma unroll
  for (int c = 0; c < N; ++c)
#pragma unroll
    for (int h = 0; h < 2; ++h) {                          // eight columns each
      float2 x[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t* f = r < 2 ? a[c] : d[c];
        const uint32_t lo = f[4 * h + 2 * (r & 1)], hi = f[4 * h + 2 * (r & 1) + 1];
        x[r] = kScaled ? mul2(lo, hi, ss[r]) : make_float2(__uint_as_float(lo), __uint_as_float(hi));
      }
      v[4 * c + 2 * h] = max3(x[0].x, x[1].x, fmaxf(x[2].x, x[3].x));
      v[4 * c + 2 * h + 1] = max3(x[0].y, x[1].y, fmaxf(x[2].y, x[3].y));
    }
  frag_max<N>(v, lane);
  if (N == 1) {
    if (!(lane & 4)) atomicMax(to + frag_col(lane), order_key(v[0]));
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) atomicMax(to + 32 * i + (lane & 4 ? 16 : 0) + frag_col(lane), order_key(v[i]));
  }
}

template <bool kPacked>
__global__ void __launch_bounds__(kThreads, 1)
tree_scores_tc_kernel(const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_d,
                      const __nv_bfloat16* __restrict__ iq, const uint8_t* __restrict__ cache,
                      const uint8_t* __restrict__ drafts, float* __restrict__ scores, Dims p,
                      Plan plan, int per_group, uint32_t tmem_cols, int* status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* qs = smem + plan.q_at();
  uint8_t* ex = smem + plan.ex_at();
  int* res = reinterpret_cast<int*>(smem + plan.res_at());         // [2][8 blocks][cols], order_key
  int* dres = reinterpret_cast<int*>(smem + plan.dres_at());       // [2 blocks][cols]
  float* qscale = reinterpret_cast<float*>(smem + plan.scale_at());
  int* rows = reinterpret_cast<int*>(smem + plan.row_at());        // score row of a column
  Small& s = *reinterpret_cast<Small*>(smem + plan.small_at());
  ptx::grid_wait();
  ptx::launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int node0 = blockIdx.y * per_group;
  const int n_nodes = min(per_group, p.nR - node0);
  const int C = n_nodes * p.Hkv, Cp = plan.cols, stages = plan.stages;
  const volatile int* abort = &s.abort;

  if (warp == 0) find_range(p, s, lane);
  if (tid == 32) {
    for (int i = 0; i < stages; ++i) {
      ptx::mbar_init(&s.full[i], 1);
      ptx::mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < kAcc; ++i) {
      ptx::mbar_init(&s.acc_full[i], 2);                   // products done; their issuer
      ptx::mbar_init(&s.acc_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&s.res_full[i], 8 * 4);               // four warps a block
      ptx::mbar_init(&s.res_empty[i], kWriters);
    }
    ptx::mbar_init(&s.dres_full, 4);
    s.abort = 0;
    s.late = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 2) {
    ptx::tmem_alloc(&s.tmem_base, tmem_cols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before_sync();
  __syncthreads();
  ptx::tc_fence_after_sync();
  const uint32_t tmem = s.tmem_base;
  const int b = s.b, blk0 = s.blk0, nblk = s.nblk;
  const int L = seq_len_of(p, b);
  const int nB_b = (L + kBk - 1) / kBk;                    // blocks with cached keys
  const int first = L / kBk;                               // block of the first drafted position
  // the sequence's last range takes the drafted keys too, before its blocks
  const int drafted = blk0 + nblk == nB_b && (nblk > 0 || s.rank == 0) ? 1 : 0;
  const int items = nblk + drafted;
  if (warp == kProducerWarp) {
    // ------------------------------------------------------------- TMA producer
    // (The loops of this kernel turn once in 700 cycles: stages and phases are counted, not divided
    // out, and a table's entries are read 32 at a time.)
    int issued = 0, st = 0, entry = 0;
    uint32_t phase = 1;
    bool ok = true;
    if (lane == 0) ptx::tma_prefetch_desc(&tm_k);
    const int32_t* table = p.block_table ? p.block_table + (size_t)b * p.nB + blk0 : nullptr;
    for (int i = 0; i < items; ++i) {
      if (p.inject == 2 && s.rank == 0 && i > 0) break;     // test hook: no copies any more
      const bool draft = drafted && i == 0;
      const int n = i - drafted;                           // block of the range
      if (table && !draft && (n & 31) == 0) entry = n + lane < nblk ? table[n + lane] : 0;
      int y = 0, z = b;                                    // row and outer index of the tile
      if (!draft) {
        if (table) z = __shfl_sync(0xffffffffu, entry, n & 31);
        else if (kPacked) z = b * p.nB + blk0 + n;
        else y = (blk0 + n) * kBk;
        debug_check(z >= 0 && z < (table || kPacked ? p.n_phys : p.B), status, kDbgCoord);
      }
      if (!ptx::mbar_wait(&s.empty[st], phase, abort)) { ok = false; break; }
      if (lane == 0) {
        uint8_t* to = smem + st * plan.stage_bytes;
        const CUtensorMap* tm = draft ? &tm_d : &tm_k;
        ptx::mbar_arrive_expect_tx(&s.full[st], plan.stage_bytes + (kPacked ? kBk : 0));
        if (kPacked) {
          ptx::tma_load_3d(to, tm, &s.full[st], 0, 0, z);
          // a table entry that is no block: zeros for the codes, some block's exponents.  The slot was
          // read kScaleSlots items ago: the stage is free since the products of the item `stages`
          // before this one, whose accumulator was free since the epilogue of kAcc items before that
          const int zc = draft ? z : min(max(z, 0), p.n_phys - 1);
          ptx::bulk_load(ex + (i & (kScaleSlots - 1)) * kBk,
                         (draft ? drafts : cache) + (size_t)zc * index_record(kDI) + kBk * kDI, kBk,
                         &s.full[st]);
        } else {
          ptx::tma_load_3d(to, tm, &s.full[st], 0, y, z);
          ptx::tma_load_3d(to + kBk * kRowBytes, tm, &s.full[st], 64, y, z);
        }
      }
      issued = i + 1;
      if (++st == stages) st = 0, phase ^= 1;
      __syncwarp();
    }
    if (!ok && lane == 0) raise_abort(s, status, 0x501);
    // copies in flight land before the CTA leaves (after a full run they have been used)
    if (lane == 0)
      for (int i = issued > stages ? issued - stages : 0; i < issued; ++i)
        ptx::mbar_wait_timed(&s.full[i % stages], (i / stages) & 1);
  } else {
    // the producer has started; the other warps set up the tree and the results first
    // (all the queries' loads in flight together: one column after the other they took 7 us beside
    // the copies)
    const int me = warp > kProducerWarp ? tid - 32 : tid;
    const int wq = warp > kProducerWarp ? warp - 1 : warp;
    constexpr int kPass = 2 * (kWarps - 1);                // columns at a time, half a warp each
    constexpr int kOwn = (kMaxCols + kPass - 1) / kPass;
    const int sub = lane & 15, c_own = 2 * wq + (lane >> 4);
    uint4 qv[kOwn];                                        // dims 8 sub .. 8 sub + 7
#pragma unroll
    for (int x = 0; x < kOwn; ++x) {
      const int c = c_own + x * kPass;
      qv[x] = make_uint4(0, 0, 0, 0);
      if (c < C)
        qv[x] = *reinterpret_cast<const uint4*>(iq + (((size_t)b * p.nR + node0) * p.Hkv + c) * kDI + sub * 8);
    }
    for (int e = me; e < 16 * plan.res_row(); e += kThreads - 32) res[e] = kNothing;
    for (int e = me; e < 2 * Cp; e += kThreads - 32) dres[e] = kNothing;
    if (me < 64) {
      const TreeWord path = me < p.nR ? tree_path(p, b, me, L) : 0;
      s.path[me] = path;
      if (path && tree_pos(path, L) / kBk == first + 1) atomicOr(&s.late, 1ull << me);
    }
    asm volatile("bar.sync 4, %0;" ::"n"(kThreads - 32) : "memory");
    // ---- the queries as the B operand, K-major with the 128-byte swizzle (16-byte unit u of row c
    // lies at unit u ^ (c % 8)); half a warp a column, and Cp is even, so a warp leaves as a whole
#pragma unroll
    for (int x = 0; x < kOwn; ++x) {
      const int c = c_own + x * kPass;
      if (c >= Cp) break;
      const int node = node0 + c / p.Hkv;
      const bool there = c < C && s.path[node] != 0;
      const uint4 w = there ? qv[x] : make_uint4(0, 0, 0, 0);
      float scale = p.index_scale;
      if (kPacked) {
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
        uint32_t amax = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = max(amax, max(v[e] << 16 & 0x7fffffffu, v[e] & 0x7fff0000u));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const uint32_t byte = index_exponent<15>(amax);
        const float inv = pow2_byte(254 - byte);
        scale *= pow2_byte(byte);
        // fp16 holds the scaled dims and what the parts leave of them: 8 bits, the last at 2^-24 or more
        __half2 rest[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          rest[e] = __floats2half2_rn(__uint_as_float(v[e] << 16) * inv, __uint_as_float(v[e] & 0xffff0000u) * inv);
        uint8_t* to = qs + c * kRowBytes + (((sub >> 1) ^ (c & 7)) << 4) + (sub & 1) * 8;
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          uint32_t code[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            code[e] = e5m2_pair(rest[e]);
            rest[e] = __hsub2(rest[e], from_e5m2_pair(code[e]));
          }
          *reinterpret_cast<uint2*>(to + part * Cp * kRowBytes) =
              make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
        }
      } else {
        *reinterpret_cast<uint4*>(qs + (sub >> 3) * Cp * kRowBytes + c * kRowBytes +
                                  (((sub & 7) ^ (c & 7)) << 4)) = w;
      }
      if (sub == 0) {
        qscale[c] = scale;
        // the column's score row; of an absent token (scores -inf) its complement
        const int row = (b * p.Hkv + c % p.Hkv) * p.nR + node;
        rows[c] = there ? row : ~row;
      }
    }
    // blocks that no key of this sequence can be in: its CTAs share them out
    const int f0 = min(p.nB, first + 2);
    for (int c = s.rank * (kWarps - 1) + wq; c < C; c += s.cnt * (kWarps - 1)) {
      float* to = scores + (size_t)((b * p.Hkv + c % p.Hkv) * p.nR + node0 + c / p.Hkv) * p.nB;
      for (int e = f0 + lane; e < p.nB; e += 32) to[e] = -INFINITY;
    }
    ptx::fence_proxy_async_smem();
    asm volatile("bar.sync 2, %0;" ::"n"(kThreads - 32) : "memory");

    if (warp >= kMmaWarp && warp < kWriterWarp) {
      // ---------------------------------------------------------- MMA issuers
      const int m = warp - kMmaWarp;
      int issued = -1;                                     // the last item issued here
      bool ok = true;
      int st = m;
      uint32_t phase = 0;
      const uint64_t a_desc = ptx::smem_desc_k_sw128(ptx::smem_u32(smem));
      const uint64_t q_desc = ptx::smem_desc_k_sw128(ptx::smem_u32(qs));
      const int q_tile = Cp * kRowBytes;                   // 8-bit: a part; 16-bit: half of the dims
      const uint32_t idesc = kPacked ? ptx::idesc_e4m3_e5m2_f32(kBk, Cp) : ptx::idesc_bf16_f32(kBk, Cp);
      for (int i = m; i < items; i += kIssuers) {
        const int buf = i % kAcc;
        if (!ptx::mbar_wait(&s.full[st], phase, abort) ||
            !ptx::mbar_wait(&s.acc_empty[buf], ((i / kAcc) & 1) ^ 1, abort)) { ok = false; break; }
        ptx::tc_fence_after_sync();
        if (lane == 0) {
          const uint32_t d = tmem + buf * Cp;
          const uint64_t a = a_desc + ((uint32_t)(st * plan.stage_bytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < 4 * (kPacked ? kParts : 2); ++kk) {
            const uint64_t q = q_desc + ((uint32_t)((kk >> 2) * q_tile + (kk & 3) * 32) >> 4);
            if (kPacked)                                   // all parts against the same 128 dims
              ptx::umma_f8_ss(d, a + ((kk & 3) * 32 >> 4), q, idesc, kk > 0 ? 1u : 0u);
            else
              ptx::umma_bf16_ss(d, a + (((kk >> 2) * kBk * kRowBytes + (kk & 3) * 32) >> 4), q, idesc,
                                kk > 0 ? 1u : 0u);
          }
          ptx::umma_commit(&s.empty[st]);
          ptx::umma_commit(&s.acc_full[buf]);
          // this thread has seen the copies land: passes on what the epilogue reads of them
          ptx::mbar_arrive(&s.acc_full[buf]);
        }
        issued = i;
        st += kIssuers;
        if (st >= stages) st -= stages, phase ^= 1;
        __syncwarp();
      }
      if (!ok && lane == 0) raise_abort(s, status, 0x502);
      if (lane == 0 && issued >= 0)                        // the last products here are complete
        ptx::mbar_wait_timed(&s.acc_full[issued % kAcc], (issued / kAcc) & 1);
    } else if (warp >= kWriterWarp) {
      // -------------------------------------------------------------- writers
      const int wt = tid - kWriterWarp * 32;
      const int grp0 = blk0 >> 3, groups = nblk > 0 ? ((blk0 + nblk - 1) >> 3) - grp0 + 1 : 0;
      bool ok = true;
      // maxima of block `to` in column c, from the group's buffer (left empty for the next) and from
      // the drafted keys; -inf once a wait was given up
      auto write = [&](int c, int to, bool cached) {
        int key = kNothing;
        if (ok && cached) {
          int* r = res + ((((to >> 3) - grp0) & 1) * 8 + (to & 7)) * plan.res_row() + c;
          key = *r;
          *r = kNothing;
        }
        if (ok && drafted && to >= first) key = max(key, dres[(to - first) * Cp + c]);
        float v = from_order_key(key);
        const int row = rows[c];
        v = row < 0 || v == -INFINITY ? -INFINITY : v * qscale[c];
        scores[(size_t)(row < 0 ? ~row : row) * p.nB + to] = v;
      };
      for (int o = 0; o < groups; ++o) {
        const int base = (grp0 + o) * 8;
        const int lo = max(base, blk0), hi = min(base + 8, blk0 + nblk);
        if (ok) {
          if (wt == 0 && hi - lo < 8) arrive_n(&s.res_full[o & 1], (8 - (hi - lo)) * 4);
          __syncwarp();
          ok = ptx::mbar_wait(&s.res_full[o & 1], (o >> 1) & 1, abort);
          if (ok && drafted && o + 1 == groups) ok = ptx::mbar_wait(&s.dres_full, 0, abort);
          ok = __all_sync(0xffffffffu, ok);
        }
        for (int e = wt; e < C * 8; e += kWriters * 32)
          if (base + (e & 7) >= lo && base + (e & 7) < hi) write(e >> 3, base + (e & 7), true);
        __syncwarp();
        if (ok && lane == 0) ptx::mbar_arrive(&s.res_empty[o & 1]);
      }
      if (ok && drafted && groups == 0)
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(&s.dres_full, 0, abort));
      if (drafted) {                                       // blocks of drafted keys alone
        const int n1 = min(p.nB, first + 2);
        for (int e = wt; e < C * 2; e += kWriters * 32)
          if (nB_b + (e & 1) < n1) write(e >> 1, nB_b + (e & 1), false);
      }
      if (!ok && lane == 0) raise_abort(s, status, 0x504);
    } else {
      // ------------------------------------------------------------- epilogue
      const int quad = warp & 3, gr = lane >> 2;
      bool ok = true;
      for (int i = warp >> 2; i < items; i += kGroups) {
        const int buf = i % kAcc;
        const bool draft = drafted && i == 0;
        const int blk = blk0 + i - drafted;
        const int o = (blk >> 3) - (blk0 >> 3);            // group of eight blocks
        if (!ptx::mbar_wait(&s.acc_full[buf], (i / kAcc) & 1, abort)) { ok = false; break; }
        ptx::tc_fence_after_sync();
        float sc[4] = {1.f, 1.f, 1.f, 1.f};
        if (kPacked)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            sc[r] = pow2_byte(ex[(i & (kScaleSlots - 1)) * kBk + quad * 32 + r * 8 + gr]);
        if (!draft && !ptx::mbar_wait(&s.res_empty[o & 1], ((o >> 1) & 1) ^ 1, abort)) { ok = false; break; }
        const uint32_t at = tmem + ((uint32_t)(quad * 32) << 16) + buf * Cp;
        const int seen = L - blk * kBk - quad * 32;        // keys of this warp's 32 (blocks only)
        int* to = res + ((o & 1) * 8 + (blk & 7)) * plan.res_row();
        if (!draft && seen >= 32) {
          int c0 = 0;
          for (; c0 + 64 <= Cp; c0 += 64) block_max<4, kPacked>(at + c0, sc, to + c0, lane);
          if (Cp & 32) block_max<2, kPacked>(at + c0, sc, to + c0, lane), c0 += 32;
          if (Cp & 16) block_max<1, kPacked>(at + c0, sc, to + c0, lane);
        } else {
          // some keys only: those before the sequence's end, or drafted keys that are on the
          // column's path, in the first position's block and (second turn) in the next
#pragma unroll 1
          for (int e = 0; e < Cp / 16 * (draft ? 2 : 1); ++e) {
            const int c0 = (draft ? e >> 1 : e) * 16, late = draft ? e & 1 : 0;
            uint32_t a[8], d[8];
            ptx::tmem_ld_frag16(at + c0, a);
            ptx::tmem_ld_frag16(at + (16u << 16) + c0, d);
            ptx::tmem_ld_wait();
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int col = c0 + (j >> 1) * 8 + 2 * (lane & 3) + (j & 1);
              TreeWord in = draft && col < C ? s.path[node0 + col / p.Hkv] : 0;
              in &= late ? s.late : ~s.late;
              v[j] = -INFINITY;
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const int t = quad * 32 + r * 8 + gr;      // drafted token of the key
                const bool see = draft ? t < 64 && (in >> t & 1) && s.path[t] != 0 : gr + 8 * r < seen;
                const uint32_t raw = r < 2 ? a[(j >> 1) * 4 + (j & 1) + 2 * r] : d[(j >> 1) * 4 + (j & 1) + 2 * (r - 2)];
                if (see) v[j] = fmaxf(v[j], __uint_as_float(raw) * sc[r]);
              }
            }
            frag_max<1>(v, lane);
            if (!(lane & 4)) atomicMax((draft ? dres + late * Cp : to) + c0 + frag_col(lane), order_key(v[0]));
          }
        }
        ptx::tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(&s.acc_empty[buf]);
          ptx::mbar_arrive(draft ? &s.dres_full : &s.res_full[o & 1]);
        }
      }
      if (!ok && lane == 0) raise_abort(s, status, 0x503);
    }
  }

  ptx::tc_fence_before_sync();
  __syncthreads();
  if (warp == 2) {
    ptx::tc_fence_after_sync();
    ptx::tmem_dealloc(tmem, tmem_cols);
  }
}

template <bool kPacked>
cudaError_t launch(const Dims& p, const void* idx_q, const void* idx_k, const void* idx_draft,
                   float* scores, cudaStream_t st, int* status, int sms) {
  CUtensorMap tk, td;
  cudaError_t e;
  if (kPacked) {
    // records as (128 dims, 128 keys, block), 129 * 128 bytes apart
    const uint64_t stride[2] = {kRowBytes, index_record(kDI)};
    const uint32_t box[3] = {kDI, kBk, 1};
    uint64_t dims[3] = {kDI, kBk, (uint64_t)p.n_phys};
    e = make_tensor_map(CU_TENSOR_MAP_DATA_TYPE_UINT8, &tk, idx_k, 3, dims, stride, box);
    dims[2] = (uint64_t)p.B;
    if (e == cudaSuccess)
      e = make_tensor_map(CU_TENSOR_MAP_DATA_TYPE_UINT8, &td, idx_draft, 3, dims, stride, box);
  } else {
    const uint32_t box[3] = {64, kBk, 1};
    const uint64_t r = p.block_table ? (uint64_t)kBk : (uint64_t)p.Sk;
    const uint64_t kd[3] = {kDI, r, p.block_table ? (uint64_t)p.n_phys : (uint64_t)p.B};
    const uint64_t ks[2] = {kDI * 2, r * kDI * 2};
    const uint64_t dd[3] = {kDI, (uint64_t)p.nR, (uint64_t)p.B};
    const uint64_t ds[2] = {kDI * 2, (uint64_t)p.nR * kDI * 2};
    e = make_tensor_map_bf16(&tk, idx_k, 3, kd, ks, box);
    if (e == cudaSuccess) e = make_tensor_map_bf16(&td, idx_draft, 3, dd, ds, box);
  }
  if (e != cudaSuccess) return e;
  // tokens of a CTA: as many as give 128 columns (more tokens: several CTAs read the same keys at
  // about the same time, through L2)
  const int groups = (p.nR * p.Hkv + kMaxCols - 1) / kMaxCols;
  int per = (p.nR + groups - 1) / groups;
  if (per > kMaxCols / p.Hkv) per = kMaxCols / p.Hkv;
  const int n_groups = (p.nR + per - 1) / per;
  Plan plan;
  plan.cols = (per * p.Hkv + 15) / 16 * 16;
  plan.stage_bytes = kPacked ? kBk * kRowBytes : 2 * kBk * kRowBytes;
  plan.q_tiles = kPacked ? kParts : 2;
  plan.stages = kMaxStages;
  while (plan.stages > kIssuers && plan.bytes() + 1024 > kSmemLimit) plan.stages -= kIssuers;
  uint32_t cols = 32;
  while (cols < (uint32_t)(kAcc * plan.cols)) cols *= 2;
  // the kernel's limit, the same in every call: host threads with other sizes share it
  e = cudaFuncSetAttribute(tree_scores_tc_kernel<kPacked>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  if (e != cudaSuccess) return e;
  int ctas = sms / n_groups;
  if (ctas < p.B) ctas = p.B;
  return launch_after(tree_scores_tc_kernel<kPacked>, dim3((unsigned)ctas, (unsigned)n_groups), kThreads,
                      (size_t)plan.bytes() + 1024, 0, st, tk, td, (const __nv_bfloat16*)idx_q,
                      (const uint8_t*)idx_k, (const uint8_t*)idx_draft, scores, p, plan, per, cols,
                      status);
}

}  // namespace

bool tree_scores_tc_supported(const Dims& p) {
  return p.dtype == 1 && p.dI == kDI && p.Bk == kBk && p.Hkv <= 64;
}

cudaError_t launch_tree_scores_tc(const Dims& p, const void* idx_q, const void* idx_k,
                                  const void* idx_draft, int packed, float* scores,
                                  cudaStream_t st, int* status) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  return packed ? launch<true>(p, idx_q, idx_k, idx_draft, scores, st, status, sms)
                : launch<false>(p, idx_q, idx_k, idx_draft, scores, st, status, sms);
}

}  // namespace msa
