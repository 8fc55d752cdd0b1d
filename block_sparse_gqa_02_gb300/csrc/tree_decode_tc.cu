// Attention of a tree of drafted tokens on the tcgen05 tensor cores (bf16 inputs, fp32 softmax and
// accumulation; head_dim 64 or 128, blocks of 128 keys).
//
// The tokens of a tree select mostly the same blocks, so a block is read once for all of
// them.  CTA = (split, up to 256 rows, sequence x KV head), a row being a (token, query head)
// of the KV head's group.  It forms the union of its tokens' selections (a bitmap of blocks in
// shared memory), takes the split's share of it in order, streams these blocks through a TMA ring,
// and multiplies all rows with each; rows whose token did not select a block get weight 0 there.
// The drafted keys are one more block, with a mask of the path a row.
//
// More than 128 rows are two tiles that share each block (O0 and O1 take half of TMEM), fewer are
// one.  A step is half a block's keys: a tile has two S buffers of 64 columns, so that the next
// Q.K^T runs under the softmax, and the copies' ring has slots of half a block: Q takes 32 KiB a
// tile, which leaves 144 KiB (two tiles) or 176 KiB (one) for keys and values.
// Measured, ragged 8 x 128K, 16 drafts of 16 heads a KV head (206 MB, 128 CTAs): 67 us, of which 4.7
// set-up, 2.3 to the first S, 46 for 48 steps, 3.5 epilogue and 5 the join.  A step takes some 1,830
// cycles.  In 1,030 of them shared memory serves the products' operands, 128 bytes a cycle (Q again for
// every half block: 64 KiB; K and V once a tile: 64 KiB), and in 256 the copies land; HBM is busy 38 %
// of the time.  So a step waits for shared memory first, the rest is the chain of copy, product and
// softmax.  2 x 64K, 64 drafts (72 MB from HBM, read by four CTAs each): 79 us, 1.0 us a step, though it
// reads a third as much.
// Warps: 0-3 and 4-7 softmax and epilogue of a tile each, 8 TMA producer, 9 issues Q.K^T, 10 issues
// P.V.  P is written over S and read by the P.V product from TMEM, rounded to bf16 (by at most 2^-8 of
// each weight: the product takes V's type; its sum is not rounded).  Online softmax in the log2
// domain; the running base moves only when a step would push a row's weights past a bound, so O
// is rarely rescaled.  Every wait is bounded.
#include "launch.cuh"
#include "ptx.cuh"
#include "tma_host.cuh"
#include "tree.cuh"
#include "tree_decode_tc.cuh"

namespace msa {

namespace {

constexpr int kBk = 128;
constexpr int kTileRows = 128;
constexpr int kRowBytes = 128;
constexpr int kMaxItems = 512;         // blocks of a split
constexpr int kCols = 64;              // keys of a step
constexpr int kSteps = kBk / kCols;
constexpr int kMaxWords = kMaxBlocks / 32;
constexpr int kThreads = 352;
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;            // issues the Q.K^T products; warp 10 the P.V ones
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleThreshold = 8.0f;   // log2 units, on a block's maximum
constexpr float kSumThreshold = 512.0f;     // on a block's sum of weights
constexpr float kLn2 = 0.6931471805599453f;

template <int kD, int kTiles>
struct __align__(1024) Smem {
  static constexpr int kChunks = kD / 64;
  static constexpr int kTileBytes = kChunks * kTileRows * kRowBytes;   // [chunk][128 rows][128 B]
  static constexpr int kSlotBytes = kChunks * kCols * kRowBytes;       // [chunk][64 keys][128 B]
  // slots: K is copied a step ahead of V, which is used after the softmax
  static constexpr int kK = kD == 64 ? 10 : kTiles == 2 ? 5 : 6, kV = kK - 1;
  uint8_t q[kTiles][kTileBytes];
  uint8_t k[kK][kSlotBytes];
  uint8_t v[kV][kSlotBytes];
  TreeWord mask[kMaxItems];            // tokens of the CTA that selected the item
  TreeWord path[64];
  int blocks[kMaxItems];               // the item's block, and where its keys are (outer coordinate)
  int outer[kMaxItems];
  uint32_t bitmap[kMaxWords];
  uint16_t before[kMaxWords];          // blocks in the words before
  TreeWord sel[2];                     // tokens that selected the block of the first drafted position, the next
  TreeWord late;                       // tokens whose position is in that next block
  uint64_t k_full[kK], k_empty[kK], v_full[kV], v_empty[kV];
  uint64_t s_full[2 * kTiles], p_full[2 * kTiles], pv_done[2 * kTiles], o_full[2], drain[2];
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Packed pairs of fp32 (one 64-bit register) for the paired FMA / ADD instructions.
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 f32_pair(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.ftz.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.ftz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Sets bit t of a word in shared memory (32-bit halves: their atomics are single instructions).
__device__ __forceinline__ void set_bit(TreeWord& w, int t) {
  atomicOr(reinterpret_cast<uint32_t*>(&w) + (t >> 5), 1u << (t & 31));
}

// Rows of a token: the group's heads, padded to a power of two that divides the tile.
__host__ __device__ inline int padded_heads(int G) {
  int g = 1;
  while (g < G) g *= 2;
  return g;
}

template <typename S>
__device__ __forceinline__ void raise_abort(S& s, int* status, int code) {
  s.abort = 1;
  if (status) atomicExch(status, code);
}

template <int kD, int kTiles>
__global__ void __launch_bounds__(kThreads, 1)
tree_decode_tc_kernel(const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CUtensorMap tm_kd,
                      const __grid_constant__ CUtensorMap tm_vd,
                      const __nv_bfloat16* __restrict__ q, const int32_t* __restrict__ sel,
                      float* __restrict__ ws_o, float* __restrict__ ws_l, Dims p, int lg, int* status) {
  using S = Smem<kD, kTiles>;
  constexpr int kK = S::kK, kV = S::kV, kSlotBytes = S::kSlotBytes;
  constexpr uint32_t kIdescQK = ptx::idesc_bf16_f32(128, kCols, 0, 0);
  constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(128, kD, 0, 1);
  extern __shared__ uint8_t smem_raw[];
  S& s = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  ptx::grid_wait();
  ptx::launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int n_split = gridDim.x, split = blockIdx.x;
  const int bg = blockIdx.z, b = bg / p.Hkv, g = bg % p.Hkv, G = p.G;
  const int Gp = 1 << lg, per_cta = kTiles * kTileRows >> lg;   // rows of a token, tokens
  const int node0 = blockIdx.y * per_cta;
  const int n_nodes = min(per_cta, p.nR - node0);
  const int words = (p.nB + 31) / 32;
  const volatile int* abort = &s.abort;

  // The set-up works on all warps but the producer's, which starts its copies as soon as the union
  // is known.  What comes from memory is on its way first, all at once.
  constexpr int kOthers = kThreads - 32;
  const int me = warp == kProducerWarp ? -1 : warp < kProducerWarp ? tid : tid - 32;
  const int length = p.seq_lens[b];
  const TreeWord word = me >= 0 && me < p.nR ? p.tree_mask[(size_t)b * p.nR + me] : 0;
  constexpr int kQ = (kTiles * kTileRows * (kD / 8) + kOthers - 1) / kOthers, kSel = 4;
  const int32_t* srow = sel + ((size_t)bg * p.nR + node0) * p.k;
  const int entries = n_nodes * p.k;
  int sv0[kSel], st0[kSel];                                // block and token of this thread's first entries
#pragma unroll
  for (int i = 0; i < kSel; ++i)
    sv0[i] = me >= 0 && me + i * kOthers < entries ? srow[me + i * kOthers] : -1;
  uint4 qv[kQ];
#pragma unroll
  for (int i = 0; i < kQ; ++i) {
    const int e = me + i * kOthers, r = e / (kD / 8), u = e % (kD / 8), h = r & (Gp - 1);
    qv[i] = make_uint4(0, 0, 0, 0);
    if (me >= 0 && r >> lg < n_nodes && h < G)
      qv[i] = *reinterpret_cast<const uint4*>(
          q + (((size_t)b * p.nR + node0 + (r >> lg)) * p.Hq + g * G + h) * kD + u * 8);
  }
  if (tid == 0) {
    for (int i = 0; i < kK; ++i) {
      ptx::mbar_init(&s.k_full[i], 1);
      ptx::mbar_init(&s.k_empty[i], 1);
    }
    for (int i = 0; i < kV; ++i) {
      ptx::mbar_init(&s.v_full[i], 1);
      ptx::mbar_init(&s.v_empty[i], 1);
    }
    for (int i = 0; i < 2 * kTiles; ++i) {
      ptx::mbar_init(&s.s_full[i], 1);
      ptx::mbar_init(&s.p_full[i], 4);
      ptx::mbar_init(&s.pv_done[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&s.o_full[i], 1);
      ptx::mbar_init(&s.drain[i], 1);
    }
    s.abort = 0;
    s.late = s.sel[0] = s.sel[1] = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 2) {
    ptx::tmem_alloc(&s.tmem_base, kTmemCols);
    ptx::tmem_relinquish();
  }
  for (int w = tid; w < words; w += kThreads) s.bitmap[w] = 0;
  for (int i = tid; i < kMaxItems; i += kThreads) s.mask[i] = 0;
#pragma unroll
  for (int i = 0; i < kSel; ++i) st0[i] = (me + i * kOthers) / p.k;
  const int L = length < 0 ? 0 : length > p.Sk ? p.Sk : length;
  const int first = L / kBk;                               // block of the first drafted position
  if (me >= 0 && me < 64) s.path[me] = me < p.nR ? tree_path_of(p, word, me, L) : 0;
  ptx::tc_fence_before_sync();
  __syncthreads();
  ptx::tc_fence_after_sync();

  // ---- union of the tokens' selections, over blocks with cached keys
  // calls f(entry's block, token of the CTA) for every entry
  auto each_entry = [&](auto f) {
#pragma unroll
    for (int i = 0; i < kSel; ++i)
      if (sv0[i] >= 0) f(sv0[i], st0[i]);
    for (int e = me + kSel * kOthers; e < entries; e += kOthers) f(srow[e], e / p.k);
  };
  if (me >= 0) {
    if (me < 64 && s.path[me] && tree_pos(s.path[me], L) / kBk == first + 1) set_bit(s.late, me);
    each_entry([&](int blk, int t) {
      if (blk < 0 || blk >= p.nB || s.path[node0 + t] == 0) return;
      if (blk * kBk < L) atomicOr(&s.bitmap[blk >> 5], 1u << (blk & 31));
      if (blk == first || blk == first + 1) set_bit(s.sel[blk - first], node0 + t);
    });
  }
  __syncthreads();
  const uint32_t tmem = s.tmem_base;
  int n_union = 0;                                         // every warp counts for itself
  for (int w = lane; w < words; w += 32) n_union += __popc(s.bitmap[w]);
  n_union = __reduce_add_sync(0xffffffffu, n_union);
  // the drafted keys count as one more block, the last
  const bool any_draft = s.sel[0] != 0 || s.sel[1] != 0;
  const int total = n_union + (any_draft ? 1 : 0);
  const int p0 = (int)((long long)total * split / n_split);
  const int p1 = (int)((long long)total * (split + 1) / n_split);
  const int n_items = p1 - p0;                             // at most kMaxItems, by the launcher
  const int n_blk = min(p1, n_union) - p0;                 // items that are blocks (may be < 0: none)
  const bool draft_here = any_draft && p1 == total && n_items > 0;
  // calls f(word, its bits, blocks before it) for the bitmap's words, by one warp
  auto each_word = [&](auto f) {
    int base = 0;
    for (int w0 = 0; w0 < words; w0 += 32) {
      const uint32_t bits = w0 + lane < words ? s.bitmap[w0 + lane] : 0;
      int incl = __popc(bits);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (w0 + lane < words) f(w0 + lane, bits, base + incl - __popc(bits));
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
  };
  if (me < 0) {
    each_word([&](int w, uint32_t bits, int at) {          // the split's blocks, in order
      for (at -= p0; bits; bits &= bits - 1, ++at)
        if (at >= 0 && at < n_blk) s.blocks[at] = w * 32 + __ffs(bits) - 1;
    });
    __syncwarp();
    // contiguous cache: (64 dims, key, half of the dims, sequence x head); pools: (.., key in block, ..,
    // block x head), the table's entries read here, all at once
    for (int i = lane; i < n_blk; i += 32)
      s.outer[i] = p.block_table ? p.block_table[(size_t)b * p.nB + s.blocks[i]] * p.Hkv + g : bg;
    __syncwarp();
    asm volatile("bar.arrive 3, %0;" ::"n"(kThreads) : "memory");
  } else {
    if (warp == kMmaWarp)
      each_word([&](int w, uint32_t, int at) { s.before[w] = (uint16_t)at; });
    // Q as A operands: row r = token * Gp + head, K-major with the 128-byte swizzle (16-byte unit u of
    // row r at unit u ^ (r % 8)); zero for heads past the group and absent tokens
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
      const int e = me + i * kOthers, r = e / (kD / 8), u = e % (kD / 8);
      if (r >= kTiles * kTileRows) continue;
      if (r >> lg < n_nodes && s.path[node0 + (r >> lg)] == 0) qv[i] = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(s.q[r / kTileRows] + (u >> 3) * kTileRows * kRowBytes +
                                r % kTileRows * kRowBytes + (((u & 7) ^ (r & 7)) << 4)) = qv[i];
    }
    ptx::fence_proxy_async_smem();
    asm volatile("bar.sync 4, %0;" ::"n"(kOthers) : "memory");
    each_entry([&](int blk, int t) {
      if (blk < 0 || blk >= p.nB || blk * kBk >= L || s.path[node0 + t] == 0) return;
      const int at = (int)s.before[blk >> 5] +
                     __popc(s.bitmap[blk >> 5] & ((1u << (blk & 31)) - 1)) - p0;
      if (at >= 0 && at < n_blk) set_bit(s.mask[at], t);
    });
    asm volatile("bar.sync 3, %0;" ::"n"(kThreads) : "memory");
  }
  // steps, and the S buffer of tile i in step n (its use number n / 2); the drafts fill half a block
  const int n_steps = n_items * kSteps - (draft_here ? 1 : 0);
  auto buf_of = [](int i, int n) { return 2 * i + (n & 1); };

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------- TMA producer
    // K of step n goes out before V of step n - 1
    int k_issued = 0, v_issued = 0, ks = 0, vs = 0;
    uint32_t k_phase = 1, v_phase = 1;
    bool ok = true;
    if (lane == 0 && n_items > 0) {
      ptx::tma_prefetch_desc(&tm_k);
      ptx::tma_prefetch_desc(&tm_v);
    }
    for (int n = 0; n <= n_steps && n_steps > 0; ++n) {
      if (p.inject == 2 && split == 0 && n > 1) break;      // test hook: no copies any more
      // coordinates of a step's keys
      auto place = [&](int step, int& y, int& z) {
        const int j = step / kSteps;
        const bool draft = draft_here && j == n_items - 1;
        y = draft ? 0 : step % kSteps * kCols + (p.block_table ? 0 : s.blocks[j] * kBk);
        z = draft ? bg : s.outer[j];
        debug_check(draft || (s.blocks[j] >= 0 && s.blocks[j] < p.nB && z >= 0 &&
                              z < (p.block_table ? p.n_phys : p.B) * p.Hkv), status, kDbgCoord);
        return draft;
      };
      int y, z;
      if (n < n_steps) {
        const bool draft = place(n, y, z);
        if (!ptx::mbar_wait(&s.k_empty[ks], k_phase, abort)) { ok = false; break; }
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(&s.k_full[ks], kSlotBytes);
          ptx::tma_load_4d(s.k[ks], draft ? &tm_kd : &tm_k, &s.k_full[ks], 0, y, 0, z);
        }
        k_issued = n + 1;
        if (++ks == kK) ks = 0, k_phase ^= 1;
      }
      if (n > 0) {
        const bool draft = place(n - 1, y, z);
        if (!ptx::mbar_wait(&s.v_empty[vs], v_phase, abort)) { ok = false; break; }
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(&s.v_full[vs], kSlotBytes);
          ptx::tma_load_4d(s.v[vs], draft ? &tm_vd : &tm_v, &s.v_full[vs], 0, y, 0, z);
        }
        v_issued = n;
        if (++vs == kV) vs = 0, v_phase ^= 1;
      }
      __syncwarp();
    }
    if (!ok && lane == 0) raise_abort(s, status, 0x601);
    // copies in flight land before the CTA leaves (after a full run they have been used)
    if (lane == 0) {
      for (int j = k_issued > kK ? k_issued - kK : 0; j < k_issued; ++j)
        ptx::mbar_wait_timed(&s.k_full[j % kK], (j / kK) & 1);
      for (int j = v_issued > kV ? v_issued - kV : 0; j < v_issued; ++j)
        ptx::mbar_wait_timed(&s.v_full[j % kV], (j / kV) & 1);
    }
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------- Q.K^T issuer
    bool ok = true, issued_any = false;
    for (int n = 0; ok && n < n_steps; ++n) {
      const int st = n % kK;
      if (!ptx::mbar_wait(&s.k_full[st], (n / kK) & 1, abort)) { ok = false; break; }
      for (int i = 0; i < kTiles; ++i) {
        const int buf = buf_of(i, n), use = n >> 1;
        // overwrites the S / P buffer, which the P.V product of its use before reads
        if (use > 0 && !ptx::mbar_wait(&s.pv_done[buf], (use - 1) & 1, abort)) { ok = false; break; }
        ptx::tc_fence_after_sync();
        if (lane == 0) {
          const uint32_t qa = ptx::smem_u32(s.q[i]);
          const uint32_t kb = ptx::smem_u32(s.k[st]);
#pragma unroll
          for (int kk = 0; kk < kD / 16; ++kk) {
            const uint32_t off = (kk & 3) * 32;
            ptx::umma_bf16_ss(tmem + buf * kCols,
                              ptx::smem_desc_k_sw128(qa + (kk >> 2) * (kTileRows * kRowBytes) + off),
                              ptx::smem_desc_k_sw128(kb + (kk >> 2) * (kCols * kRowBytes) + off), kIdescQK,
                              kk > 0 ? 1u : 0u);
          }
          ptx::umma_commit(&s.s_full[buf]);
          if (i == kTiles - 1) ptx::umma_commit(&s.k_empty[st]);
        }
        issued_any = true;
        __syncwarp();
      }
    }
    if (!ok && lane == 0) raise_abort(s, status, 0x602);
    if (*abort && lane == 0 && issued_any) {               // one more commit covers all issued here
      ptx::umma_commit(&s.drain[0]);
      ptx::mbar_wait_timed(&s.drain[0], 0);
    }
  } else if (warp == kMmaWarp + 1) {
    // ------------------------------------------------------------ P.V issuer
    bool ok = true, issued_any = false;
    for (int n = 0; ok && n < n_steps; ++n) {
      const int j = n / kSteps, st = n % kV;
      const bool draft = draft_here && j == n_items - 1;
      if (!ptx::mbar_wait(&s.v_full[st], (n / kV) & 1, abort)) { ok = false; break; }
      // rows of V that no key of the sequence is in may hold anything, and 0 x NaN is NaN: zeros
      const int keys = draft ? 0 : L - s.blocks[j] * kBk - n % kSteps * kCols;
      if (keys < kCols) {
#pragma unroll 8
        for (int e = lane; e < kCols * (kD / 8); e += 32) {
          const int r = e / (kD / 8), u = e % (kD / 8);
          if (draft ? s.path[r] == 0 : r >= keys)
            *reinterpret_cast<uint4*>(s.v[st] + (u >> 3) * kCols * kRowBytes + r * kRowBytes + (u & 7) * 16) =
                make_uint4(0, 0, 0, 0);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
      }
      for (int i = 0; i < kTiles; ++i) {
        const int buf = buf_of(i, n);
        if (!ptx::mbar_wait(&s.p_full[buf], (n >> 1) & 1, abort)) { ok = false; break; }
        ptx::tc_fence_after_sync();
        if (lane == 0) {
          const uint32_t vb = ptx::smem_u32(s.v[st]);
#pragma unroll
          for (int kk = 0; kk < kCols / 16; ++kk)
            ptx::umma_bf16_ts(tmem + 256 + i * 128, tmem + buf * kCols + kk * 8,
                              ptx::smem_desc_mn_sw128(vb + kk * 16 * kRowBytes, kCols * kRowBytes, 1024),
                              kIdescPV, (n > 0 || kk > 0) ? 1u : 0u);
          ptx::umma_commit(&s.pv_done[buf]);
          if (i == kTiles - 1) ptx::umma_commit(&s.v_empty[st]);
          if (n + 1 == n_steps) ptx::umma_commit(&s.o_full[i]);
        }
        issued_any = true;
        __syncwarp();
      }
    }
    if (!ok && lane == 0) raise_abort(s, status, 0x603);
    if (*abort && lane == 0 && issued_any) {
      ptx::umma_commit(&s.drain[1]);
      ptx::mbar_wait_timed(&s.drain[1], 0);
    }
  } else if (warp < 4 * kTiles) {
    // ------------------------------------------------------ softmax and epilogue
    const int i = warp >> 2, quad = warp & 3;
    const int R = i * kTileRows + quad * 32 + lane;          // row of the CTA
    const int tl = R >> lg;                                  // its token
    const float c1 = p.sm_scale * 1.4426950408889634f;       // to log2 units
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t o_addr = tmem + lane_off + 256 + i * 128;
    float m_used = -INFINITY, l = 0.f;
    bool ok = true;
    constexpr int kChunk = kCols / 32;                       // 32 columns each
    for (int n = 0; n < n_steps; ++n) {
      const int j = n / kSteps, key0 = n % kSteps * kCols;   // the block, the step's first key in it
      const bool draft = draft_here && j == n_items - 1;
      const int buf = buf_of(i, n);
      const uint32_t s_addr = tmem + lane_off + buf * kCols;
      if (!ptx::mbar_wait(&s.s_full[buf], (n >> 1) & 1, abort)) { ok = false; break; }
      ptx::tc_fence_after_sync();
      // keys that the row sees: the first `lim` of the step, or for the drafts the bits of `in`
      TreeWord in = 0;
      int lim = 0;
      if (draft) {
        const int t = node0 + tl;
        const TreeWord bit = 1ull << (t & 63);
        if (tl < n_nodes && s.path[t])
          in = s.path[t] & ((s.sel[0] & bit ? ~s.late : 0) | (s.sel[1] & bit ? s.late : 0));
        for (TreeWord w = in; w; w &= w - 1) {               // path tokens that are not there
          const int a = __ffsll((long long)w) - 1;
          if (s.path[a] == 0) in &= ~(1ull << a);
        }
      } else if (tl < n_nodes && (s.mask[j] >> tl & 1)) {
        lim = max(0, min(kCols, L - s.blocks[j] * kBk - key0));
      }
      const bool some = draft ? in != 0 : lim > 0;
      uint32_t sv[kChunk][32];
      const uint64_t c1x2 = f32x2(c1, c1);
      auto sum_of = [](const uint64_t (&a)[kChunk]) {
        uint64_t x = add_f32x2(a[0], a[1]);
        if constexpr (kChunk == 4) x = add_f32x2(x, add_f32x2(a[2], a[3]));
        return x;
      };
      // P = 2^(s * c1 - base) from the S values in sv, written over S as bf16; returns the row sum.
      auto p_from_sv = [&](float base) {
        const uint64_t negm = f32x2(-base, -base);
        uint64_t acc[kChunk];
#pragma unroll
        for (int c = 0; c < kChunk; ++c) {
          uint32_t pk[16];
          acc[c] = f32x2(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 y = f32_pair(fma_f32x2(
                f32x2(__uint_as_float(sv[c][e]), __uint_as_float(sv[c][e + 1])), c1x2, negm));
            const float a0 = ex2(y.x), a1 = ex2(y.y);
            acc[c] = add_f32x2(acc[c], f32x2(a0, a1));
            pk[e >> 1] = pack_bf16x2(a0, a1);
          }
          ptx::tmem_st_x16(s_addr + c * 16, pk);
        }
        const float2 sum = f32_pair(sum_of(acc));
        return sum.x + sum.y;
      };
      // O *= alpha in every row of the warp (1 in rows that keep their base), once the P.V product
      // of the step before is complete (with two S buffers nothing else has waited for it)
      auto rescale_o = [&](float alpha) {
        if (n > 0) {
          if (!ptx::mbar_wait(&s.pv_done[buf_of(i, n - 1)], ((n - 1) >> 1) & 1, abort)) ok = false;
          ptx::tc_fence_after_sync();
        }
#pragma unroll 1
        for (int c = 0; c < kD / 32; ++c) {
          uint32_t ov[32];
          ptx::tmem_ld_x32(o_addr + c * 32, ov);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
          ptx::tmem_st_x32(o_addr + c * 32, ov);
        }
      };
      // tcgen05.ld/st are warp-collective, so every branch around them is warp-uniform.
      if (!__any_sync(0xffffffffu, some)) {
        // no row of the warp sees the block
        uint32_t zero[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) zero[e] = 0;
#pragma unroll
        for (int c = 0; c < kChunk; ++c) ptx::tmem_st_x16(s_addr + c * 16, zero);
      } else if (!draft && __all_sync(0xffffffffu, lim == 0 || (lim == kCols && m_used != -INFINITY))) {
        // whole blocks for rows that have a base: P is formed with it while S streams in from TMEM,
        // and the block's sum is checked afterwards; rows that do not see the block take an infinite
        // base, which makes their weights 0.
        const float base = lim == 0 ? INFINITY : m_used;
        const uint64_t negm = f32x2(-base, -base);
        uint64_t acc[kChunk];
        ptx::tmem_ld_x32(s_addr, sv[0]);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < kChunk; ++c) {
          if (c < kChunk - 1) ptx::tmem_ld_x32(s_addr + (c + 1) * 32, sv[c + 1]);
          uint32_t pk[16];
          acc[c] = f32x2(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 y = f32_pair(fma_f32x2(
                f32x2(__uint_as_float(sv[c][e]), __uint_as_float(sv[c][e + 1])), c1x2, negm));
            const float a0 = ex2(y.x), a1 = ex2(y.y);
            acc[c] = add_f32x2(acc[c], f32x2(a0, a1));
            pk[e >> 1] = pack_bf16x2(a0, a1);
          }
          ptx::tmem_st_x16(s_addr + c * 16, pk);
          if (c < kChunk - 1) ptx::tmem_ld_wait();
        }
        const float2 sum = f32_pair(sum_of(acc));
        const float lb = sum.x + sum.y;
        const bool redo = lim != 0 && !(lb <= kSumThreshold);
        if (__any_sync(0xffffffffu, redo)) {
          // rare: a row's weights grew past the bound; the warp redoes the block from its maximum
          float alpha = 1.f;
          if (redo) {
            float mx[kChunk], mb = -INFINITY;
#pragma unroll
            for (int c = 0; c < kChunk; ++c) {
              mx[c] = -INFINITY;
#pragma unroll
              for (int e = 0; e < 32; e += 2)
                mx[c] = max3(mx[c], __uint_as_float(sv[c][e]), __uint_as_float(sv[c][e + 1]));
              mb = fmaxf(mb, mx[c]);
            }
            mb *= c1;
            alpha = ex2(m_used - mb);
            m_used = mb;
          }
          l = l * alpha + p_from_sv(lim == 0 ? INFINITY : m_used);
          rescale_o(alpha);
        } else {
          l += lb;
        }
      } else {
        // a row's first block, or keys that a row does not see: the block's maximum first
#pragma unroll
        for (int c = 0; c < kChunk; ++c) ptx::tmem_ld_x32(s_addr + c * 32, sv[c]);
        ptx::tmem_ld_wait();
        float mc[kChunk], mb = -INFINITY;
#pragma unroll
        for (int c = 0; c < kChunk; ++c) {
          const int in_chunk = lim - 32 * c;
          const uint32_t word = draft ? (c < 2 ? (uint32_t)(in >> (32 * (c & 1))) : 0)
                                      : in_chunk >= 32 ? 0xffffffffu : in_chunk > 0 ? (1u << in_chunk) - 1 : 0;
          mc[c] = -INFINITY;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float x = word >> e & 1 ? __uint_as_float(sv[c][e]) : -INFINITY;
            sv[c][e] = __float_as_uint(x);
            mc[c] = fmaxf(mc[c], x);
          }
          mb = fmaxf(mb, mc[c]);
        }
        mb *= c1;
        float alpha = 1.f;
        bool rescale = false;
        if (mb > m_used + kRescaleThreshold) {
          if (m_used != -INFINITY) {
            alpha = ex2(m_used - mb);
            rescale = true;
            l *= alpha;
          }
          m_used = mb;
        }
        l += p_from_sv(m_used == -INFINITY ? 0.f : m_used);
        if (__any_sync(0xffffffffu, rescale)) rescale_o(alpha);
      }
      ptx::tmem_st_wait();
      ptx::tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&s.p_full[buf]);
      if (!ok) break;
    }
    if (!ok && lane == 0) raise_abort(s, status, 0x604);
    // the split's part of the row: O / l and its log-sum
    bool have_o = ok && n_items > 0;
    if (have_o) {
      if (!ptx::mbar_wait(&s.o_full[i], 0, abort)) {
        have_o = false;
        if (lane == 0) raise_abort(s, status, 0x605);
      }
    }
    if (have_o) ptx::tc_fence_after_sync();
    const bool some = have_o && l > 0.f;
    const float inv = some ? 1.f / l : 0.f;
    // Half of the dims at a time through shared memory, so that a row is written in runs: the tile's
    // own Q is no longer read (its last Q.K^T was before its last P.V), and its rows of 2 kD bytes
    // hold kD / 2 values, 16-byte unit u of row r at u ^ (r % units).
    constexpr int kPass = kD / 2, kUnits = kPass / 4;
    const int hl = R & (Gp - 1);
    const long long slot =                                   // of this thread's row; -1: none
        tl < n_nodes && hl < G
            ? (long long)((((size_t)b * p.nR + node0 + tl) * p.Hq + (size_t)g * G + hl) * n_split + split)
            : -1;
    debug_check(slot < 0 || node0 + tl < p.nR, status, kDbgStore);
    uint8_t* stage = s.q[i] + quad * 32 * kD * 2;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int c = 0; c < kPass / 32; ++c) {
        uint32_t ov[32];
        if (have_o) {
          ptx::tmem_ld_x32(o_addr + half * kPass + c * 32, ov);
          ptx::tmem_ld_wait();
        }
#pragma unroll
        for (int w = 0; w < 8; ++w)
          *reinterpret_cast<float4*>(stage + lane * kD * 2 + (((c * 8 + w) ^ (lane & (kUnits - 1))) << 4)) =
              some ? make_float4(__uint_as_float(ov[4 * w]) * inv, __uint_as_float(ov[4 * w + 1]) * inv,
                                 __uint_as_float(ov[4 * w + 2]) * inv, __uint_as_float(ov[4 * w + 3]) * inv)
                   : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      __syncwarp();
#pragma unroll 4
      for (int r0 = 0; r0 < 32; r0 += 32 / kUnits) {
        const int u = lane % kUnits, r = r0 + lane / kUnits;
        const long long at = __shfl_sync(0xffffffffu, slot, r);
        if (at < 0) continue;
        *reinterpret_cast<float4*>(ws_o + at * kD + half * kPass + u * 4) =
            *reinterpret_cast<const float4*>(stage + r * kD * 2 + ((u ^ (r & (kUnits - 1))) << 4));
      }
      __syncwarp();
    }
    if (slot >= 0) ws_l[slot] = some ? (m_used + __log2f(l)) * kLn2 : -INFINITY;
  }

  ptx::tc_fence_before_sync();
  __syncthreads();
  if (warp == 2) {
    ptx::tc_fence_after_sync();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

int tiles_of(const Dims& p) { return p.nR * padded_heads(p.G) > kTileRows ? 2 : 1; }

template <int kD, int kTiles>
cudaError_t launch(const Dims& p, const void* q, const void* k, const void* v, const void* kd,
                   const void* vd, const int32_t* sel, float* ws_o, float* ws_l, int n_split,
                   cudaStream_t st, int* status) {
  CUtensorMap tk, tv, tkd, tvd;
  // rows as (64 dims, key, half of the head, outer): one box {64, 64, halves, 1} lands half a block as
  // [half of the dims][64 keys][128 B], the swizzled chunks that the products read
  constexpr uint64_t kHalves = kD / 64;
  const uint64_t rows = p.block_table ? (uint64_t)kBk : (uint64_t)p.Sk;
  const uint64_t outer = (uint64_t)p.Hkv * (p.block_table ? (uint64_t)p.n_phys : (uint64_t)p.B);
  const uint64_t dims[4] = {64, rows, kHalves, outer};
  const uint64_t stride[3] = {kD * 2, 128, rows * kD * 2};
  const uint64_t ddims[4] = {64, (uint64_t)p.nR, kHalves, (uint64_t)p.B * p.Hkv};
  const uint64_t dstride[3] = {kD * 2, 128, (uint64_t)p.nR * kD * 2};
  const uint32_t box[4] = {64, (uint32_t)kCols, (uint32_t)kHalves, 1};
  cudaError_t e = make_tensor_map_bf16(&tk, k, 4, dims, stride, box);
  if (e == cudaSuccess) e = make_tensor_map_bf16(&tv, v, 4, dims, stride, box);
  if (e == cudaSuccess) e = make_tensor_map_bf16(&tkd, kd, 4, ddims, dstride, box);
  if (e == cudaSuccess) e = make_tensor_map_bf16(&tvd, vd, 4, ddims, dstride, box);
  if (e != cudaSuccess) return e;
  constexpr size_t smem = sizeof(Smem<kD, kTiles>) + 1024;
  static_assert(smem <= 232448, "shared memory of a CTA");
  e = cudaFuncSetAttribute(tree_decode_tc_kernel<kD, kTiles>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int Gp = padded_heads(p.G), per = kTiles * kTileRows / Gp;
  int lg = 0;
  while (1 << lg < Gp) ++lg;
  const dim3 grid((unsigned)n_split, (unsigned)((p.nR + per - 1) / per), (unsigned)(p.B * p.Hkv));
  return launch_after(tree_decode_tc_kernel<kD, kTiles>, grid, kThreads, smem, 0, st, tk, tv, tkd, tvd,
                      (const __nv_bfloat16*)q, sel, ws_o, ws_l, p, lg, status);
}

}  // namespace

bool tree_decode_tc_supported(const Dims& p) {
  return p.dtype == 1 && p.Bk == kBk && (p.d == 64 || p.d == 128) && p.G <= 64;
}

int tree_decode_tc_splits(const Dims& p) {
  const int tiles = tiles_of(p), per = tiles * kTileRows / padded_heads(p.G);
  const long long tokens = per < p.nR ? per : p.nR;
  const long long units = (long long)p.B * p.Hkv * ((p.nR + per - 1) / per);
  // one CTA a SM, no more than there can be blocks, and as many as keep a split's list in bounds
  long long most = tokens * p.k;
  if (most > p.nB) most = p.nB;
  most += 1;
  long long s = 152 / units;
  if (s > most) s = most;
  if (s < 1) s = 1;
  const long long least = (most + kMaxItems - 1) / kMaxItems;
  return (int)(s < least ? least : s);
}

cudaError_t launch_tree_decode_tc(const Dims& p, const void* q, const void* k, const void* v,
                                  const void* k_draft, const void* v_draft, const int32_t* sel,
                                  float* ws_o, float* ws_l, cudaStream_t st, int* status) {
  const int n_split = tree_decode_tc_splits(p);
  auto run = tiles_of(p) == 2 ? (p.d == 128 ? launch<128, 2> : launch<64, 2>)
                              : (p.d == 128 ? launch<128, 1> : launch<64, 1>);
  return run(p, q, k, v, k_draft, v_draft, sel, ws_o, ws_l, n_split, st, status);
}

}  // namespace msa
