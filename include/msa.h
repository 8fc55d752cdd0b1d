/*
 * msa.h -- C ABI of the MiniMax Sparse Attention (MSA) hot path for GB300 (sm_103a).
 *
 * The method (from the talk pages on MSA):
 *   - an index branch runs lightweight causal full attention with one index query head
 *     per KV head against ONE shared index key head, and its scores are reduced to
 *     per-key-block scores ("Sparse Attention Cannot Be Directly Ported Across
 *     Architectures", disconfirmai.com, paragraph introducing MSA; "How MiniMax M3 was
 *     built", aietalks.com, section "MSA uses a lightweight index branch before sparse
 *     attention");
 *   - every KV head takes its own top-k of blocks, never merged across heads (same
 *     article, paragraph "MSA addresses these issues"; aietalks.com, section
 *     "Block-level retrieval makes sparse attention easier to run on GPUs");
 *   - the main GQA branch computes exact softmax attention over the selected blocks only
 *     (Chinese topic page on MSA, summary paragraph).
 * The pages fix no block size, k, pooling or tie-break; this library uses: scores are the
 * MAX over a query tile's tokens and a block's causally visible keys of
 * index_scale * <q_I, k_I>; the block holding the tile's last query (the "current block")
 * is always selected and counts towards top_k; the other top_k-1 are the highest scores,
 * ties to the lower block index, -0 == +0; the list is written ascending, padded with -1.
 *
 * Layouts (row-major, contiguous, element type = shape->dtype unless stated):
 *   q, out        [batch, seq_q, n_heads_q, head_dim]
 *   k, v          [batch, n_heads_kv, seq_k, head_dim]    (head-major: a block of one
 *                                                          KV head is one contiguous run)
 *   idx_q         [batch, seq_q, n_heads_kv, index_dim]   (index query head g serves KV head g)
 *   idx_k         [batch, seq_k, index_dim]               (the single index key head)
 *   block_scores  float32 [batch, n_heads_kv, n_rows, n_blocks]
 *   sel           int32   [batch, n_heads_kv, n_rows, top_k]
 *   lse           float32 [batch, n_heads_q, seq_q], natural log
 * with n_blocks = ceil(seq_k / block_size) and n_rows = ceil(seq_q / q_tile).
 *
 * Two modes, told apart by the shape:
 *   prefill  seq_q == seq_k == T, query i at position i, rows are tiles of q_tile queries
 *            (block_size % q_tile == 0);
 *   decode   seq_q == 1, q_tile == 1, seq_k == L (the cache includes the new token), the
 *            query at position L-1, one row per sequence (selection per token).
 * Query head h uses KV head h / (n_heads_q / n_heads_kv).
 *
 * Conventions:
 *   - Ownership: the caller owns every buffer.  Only msa_sparse_decode needs scratch, and
 *     the caller passes it (msa_workspace_bytes); no entry point here allocates memory.
 *   - Pointers are device pointers (cudaMalloc or equivalent), 16-byte aligned.
 *   - Every call is asynchronous on `stream` (a cudaStream_t; NULL = legacy default
 *     stream) and returns after launching.  Argument checks happen before any launch; on
 *     failure nothing is launched and msa_last_error() describes the problem.
 *   - A kernel that gives up a bounded wait sets a device status word that
 *     msa_get_device_status() reports as MSA_ERR_TIMEOUT.
 *   - Inputs must be finite; NaN scores give an unspecified (but in-range) selection.
 *   - Calls on distinct streams may run concurrently; the device status word is shared.
 *   - The library looks up the device addresses of its own device variables (the status
 *     word, the static decode scratch) once per device and caches them.  cudaDeviceReset
 *     (or any other teardown of the primary context) leaves those addresses stale: using
 *     the library in the same process after a device reset is not supported.
 */
#ifndef MSA_H_
#define MSA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MSA_ABI_VERSION 2

typedef enum msa_status {
  MSA_OK = 0,
  MSA_ERR_INVALID_ARG = 1, /* null/misaligned pointer, inconsistent or out-of-range shape */
  MSA_ERR_UNSUPPORTED = 2, /* valid shape that no kernel here handles (e.g. head_dim 96) */
  MSA_ERR_CUDA = 3,        /* a CUDA call or kernel launch failed */
  MSA_ERR_TIMEOUT = 4,     /* a kernel gave up a bounded wait (device status word) */
  MSA_ERR_BOUNDS = 5       /* debug builds only: a device-side index check failed (device
                            * status word; see msa_debug_build) */
} msa_status;

typedef enum msa_dtype { MSA_F32 = 0, MSA_BF16 = 1 } msa_dtype;

typedef struct msa_shape {
  int32_t batch;       /* B >= 1 */
  int32_t seq_q;       /* prefill: T; decode: 1 */
  int32_t seq_k;       /* prefill: T; decode: cache length L >= 1 */
  int32_t n_heads_q;   /* Hq, a multiple of n_heads_kv */
  int32_t n_heads_kv;  /* Hkv = number of index query heads; batch * Hkv <= 65535 */
  int32_t head_dim;    /* d: 64 or 128 */
  int32_t index_dim;   /* dI: 64 or 128 */
  int32_t block_size;  /* keys per block, >= 1; at most 32768 blocks per sequence */
  int32_t top_k;       /* blocks per KV head, current block included, >= 1 */
  int32_t q_tile;      /* queries sharing one selection: prefill divides block_size (at most
                        * 65535 tiles per sequence); decode 1 */
  int32_t dtype;       /* msa_dtype of q, k, v, idx_q, idx_k, out */
  float sm_scale;      /* softmax scale; 0 means 1/sqrt(head_dim) */
  float index_scale;   /* index logit scale; 0 means 1/sqrt(index_dim) */
} msa_shape;

/* Index branch: block_scores[b, g, m, blk] = max over the queries t of row m and the keys
 * j <= t of block blk of index_scale * <idx_q[b, t, g, :], idx_k[b, j, :]>; -inf for blocks
 * with no visible key.  Accumulation is fp32.  Prefill uses tcgen05 tensor cores for
 * bf16 with index_dim 128; decode is a streaming scan of the index-key cache. */
msa_status msa_index_scores(const msa_shape* shape, const void* idx_q, const void* idx_k,
                            float* block_scores, void* stream);

/* Per-KV-head block top-k of block_scores (layout above) into sel: the current block plus
 * the best top_k-1 of the earlier blocks by (score desc, index asc), ascending, -1 padded.
 * Bit-exact and deterministic.  Rows may hold up to 32768 candidate blocks. */
msa_status msa_block_topk(const msa_shape* shape, const float* block_scores, int32_t* sel,
                          void* stream);

/* Ablation, not MSA: the aggregated selection the pages contrast MSA with (DSA-style, one
 * token set shared by every KV head).  For each (sequence, row) the candidates' scores are
 * the fp32 sums of the KV heads' block scores, added in head order 0, 1, ...; one selection
 * by the same rule as msa_block_topk is written to every head's row of sel.  Used to
 * measure the head-diversity loss of sharing ("Sparse Attention Cannot Be Directly Ported
 * Across Architectures", paragraph on applying DSA to GQA). */
msa_status msa_block_topk_shared(const msa_shape* shape, const float* block_scores,
                                 int32_t* sel, void* stream);

/* msa_index_scores followed by msa_block_topk in one launch, without the block-score round
 * trip through HBM: the index kernel keeps each KV head's running best top_k-1 blocks as
 * the scores of successive blocks come out of the tensor cores, and writes sel directly
 * (same selection rule, bit-identical to the two calls).  block_scores may be NULL; when
 * given, it is filled as by msa_index_scores.  bf16 prefill with index_dim 128,
 * block_size 128, q_tile 64, 4 KV heads and top_k <= 256; other shapes get
 * MSA_ERR_UNSUPPORTED. */
msa_status msa_index_topk_fused(const msa_shape* shape, const void* idx_q, const void* idx_k,
                                float* block_scores, int32_t* sel, void* stream);

/* Main branch, prefill (seq_q == seq_k): for query t and head h (KV head g), attend over the
 * keys j <= t of the blocks listed in sel[b, g, t / q_tile, :] (entries -1 are skipped;
 * entries must be distinct).  Writes out (dtype) and, if lse != NULL, lse.  A row whose key
 * set is empty gets out = 0 and lse = -inf.  workspace may be NULL (ws_bytes 0). */
msa_status msa_sparse_prefill(const msa_shape* shape, const void* q, const void* k,
                              const void* v, const int32_t* sel, void* out, float* lse,
                              void* workspace, size_t ws_bytes, void* stream);

/* Training: gradients of msa_sparse_prefill for a loss L with dL/dout = dout.  Inputs are
 * the forward's q, k, v, sel, its out (dtype) and lse (natural log), and dout (dtype, same
 * layout as out).  Outputs, float32: dq [batch, seq_q, n_heads_q, head_dim] (written),
 * dk and dv [batch, n_heads_kv, seq_k, head_dim] (cleared on the stream, then accumulated:
 * a key block selected by several tiles collects all their contributions).  With p the
 * attention weights, D = dout . out, ds = p (dout . v - D): dq = sm_scale sum ds k,
 * dk += sm_scale ds q, dv += p dout.  bf16 shapes with head_dim 128, block 128, q_tile 64
 * run on the tensor cores (a query-tile pass for dq, a key-block pass for dk / dv) and need
 * a device workspace of msa_workspace_bytes(shape, 2) bytes (per-row D and a bitmap of
 * which tiles selected which blocks); other shapes run on CUDA cores and need none
 * (workspace may then be null).  dk / dv sums over several CTAs use fp32 atomics, so their
 * last bits can vary from run to run. */
msa_status msa_sparse_prefill_backward(const msa_shape* shape, const void* q, const void* k,
                                       const void* v, const int32_t* sel, const void* out,
                                       const float* lse, const void* dout, float* dq, float* dk,
                                       float* dv, void* workspace, size_t ws_bytes,
                                       void* stream);

/* Training the index branch (the pages: the index branch is trained with a KL loss to match
 * the main branch's attention).  The pages give no formula; this library's reading: for
 * token t and KV head g, over the keys J the main branch attends (selected blocks, j <= t),
 * the target is the main branch's attention distribution averaged over the group's query
 * heads (held constant; computed from q, k and the forward's lse), the index distribution
 * is the softmax over J of index_scale <idx_q[t,g], idx_k[j]>, and
 *   loss = sum over (t, g) of KL(target || index)          (natural log).
 * Outputs, float32: loss (one device scalar, cleared then accumulated), d_idx_q [batch,
 * seq_q, n_heads_kv, index_dim] (written), d_idx_k [batch, seq_k, index_dim] (cleared, then
 * accumulated over every tile and head): the gradients of loss.  Prefill shapes, at most
 * 64 query heads per KV head.  bf16 shapes with head_dim = index_dim = 128, block 128,
 * q_tile 64 and 2, 4, 8, 16 or 32 query heads per KV head run on the tensor cores (a
 * query-tile pass for the loss and d_idx_q, a key-block pass for d_idx_k) and need a
 * device workspace of msa_workspace_bytes(shape, 3) bytes; other shapes run on CUDA cores
 * in fp32 and need none.  d_idx_k and the loss are sums with fp32 atomics, so their last
 * bits can vary from run to run. */
msa_status msa_index_kl_loss(const msa_shape* shape, const void* q, const void* k,
                             const float* lse, const void* idx_q, const void* idx_k,
                             const int32_t* sel, float* loss, float* d_idx_q, float* d_idx_k,
                             void* workspace, size_t ws_bytes, void* stream);

/* Main branch, decode (seq_q == 1, q_tile == 1): the new token of every sequence attends
 * over the selected blocks of the cache (split over the blocks, partial results merged by
 * log-sum-exp).  workspace: device scratch of at least msa_workspace_bytes(shape, 1)
 * bytes, 16-byte aligned, owned by the caller; its contents on entry do not matter. */
msa_status msa_sparse_decode(const msa_shape* shape, const void* q, const void* k_cache,
                             const void* v_cache, const int32_t* sel, void* out, float* lse,
                             void* workspace, size_t ws_bytes, void* stream);

/* Decode for callers that cannot allocate device memory.  Some callers have no way to
 * call cudaMalloc where decode runs: a plugin whose host framework owns every device
 * allocation and hands it no allocator, or a serving loop that must not allocate after
 * start-up because cudaMalloc can stall the device and can fail under memory pressure.
 * This entry point computes exactly what msa_sparse_decode computes, with the same
 * arguments minus the workspace: the split-KV partial results go to a scratch array the
 * library keeps in device memory (MSA_STATIC_DECODE_SCRATCH_BYTES, held on every GPU that
 * loads the library until the process exits).  The talk pages have no counterpart to it.
 *   - A shape whose scratch (msa_workspace_bytes(shape, 1)) exceeds the array is rejected
 *     with MSA_ERR_UNSUPPORTED before anything runs; msa_last_error() names both sizes.
 *   - The first call on each device looks up the array's device address with that device
 *     current (cudaGetSymbolAddress) and caches it; make that first call before any stream
 *     capture.
 *   - Every call on a device uses the same array.  Calls that overlap on the GPU (other
 *     streams, other host threads) race on it and corrupt each other's results: serialise
 *     them.  Each call writes every scratch entry it reads, so leftovers of earlier calls do
 *     not matter and nothing needs clearing.
 *   - It calls no cudaMalloc, cudaFree or allocating library routine. */
#define MSA_STATIC_DECODE_SCRATCH_BYTES (8u << 20)
msa_status msa_sparse_decode_static(const msa_shape* shape, const void* q, const void* k_cache,
                                    const void* v_cache, const int32_t* sel, void* out,
                                    float* lse, void* stream);

/* Decode over a paged cache with a length per sequence (the serving form of decode).
 * shape: a decode shape (seq_q = q_tile = 1) whose seq_k is the capacity of the block table
 * (n_blocks = ceil(seq_k / block_size) entries per sequence); bf16, head_dim = index_dim =
 * 128, block_size 128, 4 KV heads, at most 16 query heads per KV head.
 *   seq_lens     int32 [batch], device: cache length L_b of sequence b, 1 <= L_b <= seq_k
 *                (the new token, at position L_b - 1, is already in the cache; 0 means an
 *                empty sequence: scores -inf, sel -1, out 0, lse -inf).
 *   block_table  int32 [batch, n_blocks], device: physical block holding logical block j of
 *                sequence b (entries past the sequence's last block are not read).
 *   n_phys       number of physical blocks in the pools.
 *   idx_k_pool   [n_phys, block_size, index_dim];  k_pool, v_pool [n_phys, n_heads_kv,
 *                block_size, head_dim]: one physical block holds all KV heads' keys of 128
 *                consecutive positions, each head's block contiguous.
 * Semantics are those of the contiguous decode on each sequence's logical cache.  Entries
 * of block_table outside [0, n_phys) read as zeros (no fault) and give meaningless output.
 * The three calls chain like the contiguous ones; msa_sparse_decode_paged takes the same
 * workspace as msa_sparse_decode (msa_workspace_bytes(shape, 1)). */
msa_status msa_index_scores_paged(const msa_shape* shape, const int32_t* seq_lens,
                                  const int32_t* block_table, int32_t n_phys, const void* idx_q,
                                  const void* idx_k_pool, float* block_scores, void* stream);
msa_status msa_block_topk_ragged(const msa_shape* shape, const int32_t* seq_lens,
                                 const float* block_scores, int32_t* sel, void* stream);
msa_status msa_sparse_decode_paged(const msa_shape* shape, const int32_t* seq_lens,
                                   const int32_t* block_table, int32_t n_phys, const void* q,
                                   const void* k_pool, const void* v_pool, const int32_t* sel,
                                   void* out, float* lse, void* workspace, size_t ws_bytes,
                                   void* stream);

/* ------------------------------------------------------------------ rotary positions
 * Rotates (q, k, idx_q, idx_k before the calls above) or, with inverse = 1, rotates back
 * (their gradients) by position-dependent angles: with p = positions[b, t] + pos_offset (or
 * t + pos_offset without positions) and the turn a = p * freqs[i] / 2^64 of pair i,
 *   (x0, x1) -> scale * (x0 cos - x1 sin, x0 sin + x1 cos)  of the angle 2 pi a  (-2 pi a
 *   with inverse: scale and inverse together are the gradient of scale without inverse).
 * Pair i of a head is dims (i, i + rotary_dim / 2), or (2 i, 2 i + 1) with interleaved = 1;
 * dims from rotary_dim on are copied.  freqs holds turns per position in units of 2^-64
 * turns, so the product wraps at whole turns exactly and far positions lose nothing; any
 * scheme for long contexts (positions divided, base raised, ramped frequencies) is a choice
 * of freqs and scale.  The sine takes the angle in fp32, reduced to an eighth of a turn: it is off
 * by at most 2^-28 + 2^-34 turns (2^-25 radians); products are fp32, the result is rounded once to
 * the dtype.
 *   positions   int32 [batch, seq], device; NULL: 0, 1, ..., seq - 1 in every sequence.
 *               With the cache lengths of a decode batch (seq = 1) and pos_offset = -1 the
 *               new tokens sit at the end of their caches, as long as nothing was evicted
 *               (msa_cache_evict shortens the lengths, but not the positions).  Sums wrap as
 *               32-bit integers.
 * Up to MSA_ROPE_MAX_TENSORS tensors sharing these positions go in one launch; each is
 * [batch, seq, n_heads, head_dim], or [batch, n_heads, seq, head_dim] with head_major = 1.
 * y may be x itself (in place); otherwise no y may overlap another tensor.
 * head_dim: a multiple of 16, at most 1024; rotary_dim: a multiple of 16 of at most head_dim.
 * desc and tensors are host structs, read before the call returns. */
#define MSA_ROPE_MAX_TENSORS 8
typedef struct msa_rope_desc {
  int32_t batch, seq;
  int32_t dtype;       /* msa_dtype of every tensor of the call */
  int32_t pos_offset;
  int32_t interleaved; /* 0 or 1 */
  int32_t inverse;     /* 0 or 1 */
  float scale;         /* factor on the rotated dims; finite; 0 means 1 */
} msa_rope_desc;
typedef struct msa_rope_tensor {
  const void* x;
  void* y;
  const uint64_t* freqs; /* device, [rotary_dim / 2] */
  int32_t n_heads, head_dim, rotary_dim;
  int32_t head_major;    /* 0 or 1 */
} msa_rope_tensor;
msa_status msa_rope(const msa_rope_desc* desc, const msa_rope_tensor* tensors, int32_t n_tensors,
                    const int32_t* positions, void* stream);

/* ---------------------------------------------------------------- the 4-bit KV cache
 * K and V in 4 bits: 5 bits a value with their scales, 160 * head_dim bytes for the 128 keys
 * of one KV head's block against 512 * head_dim in bf16.  A group is 32 consecutive dims of one
 * token and head.  With hi, lo its largest and smallest value (fp32 arithmetic, each operation
 * rounded to nearest even):
 *   step = bf16(hi * f - lo * f), f = fp32(1 / 15)    (steps below 2^-100 become 0)
 *   mid  = bf16(lo + 8 * step)
 *   code = clamp(rint((x - mid) * fp32(1 / step)) + 8, 0, 15), 8 when step is 0
 *   value = mid + (code - 8) * step                   (what the cache holds)
 * |value - x| <= step / 2 + 2^-8 |mid| + 2^-8 * 8 step (for |x| within bf16's range); a group
 * holding a NaN or an infinity is stored as NaN values.
 *
 * cache   uint8 [n_phys, n_heads_kv, 160 * head_dim], 16-byte aligned: K's record of the
 *         block, then V's.  With a block_table (int32 [batch, n_blocks]) logical block j of
 *         sequence b is physical block block_table[b, j], as in the paged calls above;
 *         without one (NULL) it is b * n_blocks + j, and n_phys must be batch * n_blocks.
 * One record (d = head_dim, ng = d / 32 groups; byte offsets):
 *   [0, 64 d)       codes, two a byte, the lower dim in the low half;
 *     K: key j, dim 32 g + 8 c + i (c < 4, i < 8):  j * d / 2 + c * 4 ng + g * 4 + i / 2
 *     V: key j, dim 32 g + 4 r + i (r < 8, i < 4):
 *        (r * 128 + 2 * P + j % 2) * 2 ng + g * 2 + i / 2,
 *        P = (j / 2) ^ (4 * (r % 2)) for d = 128, (j / 2) ^ (4 * (r % 4)) for d = 64
 *   [64 d, 72 d)    step, bf16, group g of key j at element g * 128 + j
 *   [72 d, 80 d)    mid, likewise
 * so that a thread's share of a tensor-core operand is one aligned load.
 *
 * shape: a decode shape (seq_q = q_tile = 1) with block_size 128 whose seq_k is the capacity
 * (n_blocks = ceil(seq_k / 128)); n_heads_q, index_dim and top_k matter to the attention
 * call only.  seq_lens int32 [batch], device (NULL: every length is seq_k; lengths are
 * clamped to [0, seq_k]).  Table entries outside [0, n_phys) are skipped (nothing is read
 * or written there). */

/* Quantises tokens into the cache.  k, v: [batch, n_heads_kv, n_new, head_dim] of the
 * shape's dtype.  Token i of sequence b goes to position starts[b] + i, or, with starts
 * NULL, to seq_lens[b] - n_new + i (the last n_new positions); positions outside
 * [0, seq_lens[b]) are not stored, so a batch padded on the right is passed as it is.  Only
 * the stored tokens' bytes change.  A decode step is n_new = 1. */
msa_status msa_cache_pack(const msa_shape* shape, int32_t n_new, const int32_t* starts,
                          const int32_t* seq_lens, const int32_t* block_table, int32_t n_phys,
                          const void* k, const void* v, void* cache, void* stream);

/* The values of the same positions (rounded once to the dtype) into k, v
 * [batch, n_heads_kv, n_out, head_dim]; rows of positions outside [0, seq_lens[b]) are left
 * as they are. */
msa_status msa_cache_unpack(const msa_shape* shape, int32_t n_out, const int32_t* starts,
                            const int32_t* seq_lens, const int32_t* block_table, int32_t n_phys,
                            const void* cache, void* k, void* v, void* stream);

/* msa_sparse_decode over the 4-bit cache: attention of q [batch, 1, n_heads_q, head_dim] over
 * the values that the selected blocks hold (below 2^118 in magnitude; V's steps within 2^24 of
 * the largest of their group of dims keep all their digits).  out, lse as there (lse may be
 * NULL); bytes of the last block past the sequence's length are never used, whatever they hold.
 * No workspace.  At most 64 query heads per KV head.
 * mass: NULL, or the accumulated attention weights below (then top_k is at most 1024). */
msa_status msa_sparse_decode_packed(const msa_shape* shape, const int32_t* seq_lens,
                                    const int32_t* block_table, int32_t n_phys, const void* q,
                                    const void* cache, const int32_t* sel, void* out, float* lse,
                                    float* mass, void* stream);

/* -------------------------------------------- eviction by accumulated attention weight
 * Decode with the attention weight that every block receives added up:
 *   mass[b, g, sel[b, g, i]] += sum over the group's query heads h and the keys j of that
 *   block of exp(z_hj - lse_h)                   (the weights of one head sum to 1)
 * mass: float32 [batch, n_heads_kv, n_blocks], the caller's, zeroed when a sequence starts.
 * out and lse (may be NULL) are bit for bit those of msa_sparse_decode where that runs on the
 * tensor cores (bf16, head_dim 128, block 128, at most 16 query heads per KV head), or, with
 * seq_lens and block_table (both given), of msa_sparse_decode_paged on its shapes; on other
 * shapes the sums run in another order.  A selected block's entry gets one addition a call, so
 * results repeat bit for bit.  (A block listed twice is counted twice, in either order.)
 * Where a kernel gives up a bounded wait (MSA_ERR_TIMEOUT), nothing is added for that sequence
 * and KV head, and the heads concerned have out 0 and lse -inf.
 * top_k is at most 2^20.  workspace: msa_workspace_bytes(shape, 4) bytes, as for
 * msa_sparse_decode. */
msa_status msa_sparse_decode_mass(const msa_shape* shape, const int32_t* seq_lens,
                                  const int32_t* block_table, int32_t n_phys, const void* q,
                                  const void* k, const void* v, const int32_t* sel, void* out,
                                  float* lse, float* mass, void* workspace, size_t ws_bytes,
                                  void* stream);

/* Chooses, for every sequence of more than `keep` blocks, the blocks that stay: the first
 * n_first, the last n_recent (the one that is being filled among them), and of the others
 * those of the largest score, ties to the lower block index; a block's score is the fp32 sum
 * of its mass over the KV heads in head order (NaN counts as the lowest).  Whole blocks go
 * and the rest keep their keys together, so the index scores of those that stay do not
 * change; all heads of a sequence drop the same ones, as they share index keys and table.
 * Keys that were rotated stay rotated to the positions they had, so the new tokens' positions
 * (msa_rope) go on counting past the shortened lengths.
 *   kept      int32 [batch, keep]: the old indices of the blocks that stay, ascending, -1 padded
 *   new_lens  int32 [batch]: the lengths without the dropped blocks
 *   mass_out  [batch, n_heads_kv, n_blocks]: mass of the kept blocks, in their order, then 0
 *   table_out int32 [batch, n_blocks] (NULL without a block_table): the sequence's entries
 *             with the kept blocks first and the dropped ones after them (both ascending),
 *             entries past the sequence's last block as they were.  A sequence grows into
 *             the blocks it dropped, or the caller takes them back.
 * new_lens, mass_out and table_out may be the inputs themselves (in place), but may not
 * overlap them otherwise, nor one another or kept.  shape: a decode shape (n_blocks at most
 * 32768); seq_lens NULL: every length is seq_k.
 * n_first + n_recent <= keep <= 2^20, n_first >= 0, n_recent >= 1. */
msa_status msa_cache_evict(const msa_shape* shape, int32_t keep, int32_t n_first, int32_t n_recent,
                           const int32_t* seq_lens, const float* mass, const int32_t* block_table,
                           int32_t* kept, int32_t* new_lens, float* mass_out, int32_t* table_out,
                           void* stream);

/* Contiguous caches: copies block kept[b, i] of every source to block i of its destination
 * (entries outside the source are skipped).  Up to MSA_GATHER_MAX_TENSORS caches
 * [batch, n_heads, rows, row_bytes] a launch (K, V, index keys; the 4-bit cache without a
 * table is n_heads = 1, rows = 128 * n_blocks, row_bytes = n_heads_kv * 160 * head_dim / 128).
 * Rows past src_rows are not read, rows past dst_rows not written; rows of the destination
 * that no kept block covers stay as they are.  Sources and destinations must not overlap. */
#define MSA_GATHER_MAX_TENSORS 8
typedef struct msa_gather_tensor {
  const void* src;
  void* dst;
  int64_t src_rows, dst_rows; /* rows per (sequence, head) */
  int32_t n_heads;
  int32_t row_bytes;          /* a multiple of 16, at most 65536 */
} msa_gather_tensor;
msa_status msa_cache_gather(int32_t batch, const msa_gather_tensor* tensors, int32_t n_tensors,
                            const int32_t* kept, int32_t keep, int32_t block_size, void* stream);

/* ---------------------------------------------------- decode over a tree of drafted tokens
 * Checks several drafted tokens of every sequence in one step: the caches are read once for all
 * of them.  The drafts of a sequence form a forest of up to MSA_TREE_MAX_TOKENS tokens; token i's
 * parent is an earlier token or, for -1, the last cached token.  mask [batch, n_tokens] is the
 * tree in bits: bit a of mask[b, i] is set when token a is on the path from the root to i, i
 * among them; 0 (or any word without bit i) means that the sequence has no token i.  With the
 * cache length L_b (drafts not counted) and depth = bits of mask[b, i] - 1, token i is at position
 * L_b + depth.  It sees the cached keys j < L_b and the keys of its path, each in the block of
 * its position: what a decode step would give it with its path appended to the cache.
 *
 * shape: seq_q = n_tokens (1 .. 64), q_tile = 1, seq_k the capacity of the caches (with a block
 * table: n_blocks = ceil(seq_k / block_size) entries a sequence); a token at a position of seq_k
 * or more counts as absent.  Arrays over tokens have them as the shape's seq_q:
 *   q, out [batch, n_tokens, n_heads_q, head_dim], idx_q [batch, n_tokens, n_heads_kv, index_dim],
 *   k_draft, v_draft [batch, n_heads_kv, n_tokens, head_dim], lse [batch, n_heads_q, n_tokens],
 *   block_scores [batch, n_heads_kv, n_tokens, n_blocks], sel [batch, n_heads_kv, n_tokens, top_k].
 * Absent tokens get scores -inf, sel -1, out 0, lse -inf, and nothing of theirs is used, whatever
 * it holds.  seq_lens int32 [batch] (device) is needed; lengths are clamped to [0, seq_k].
 * block_table NULL: the caches are contiguous (n_phys is read for 8-bit index keys only); else
 * pools of n_phys blocks, as in the paged calls.  Table entries outside [0, n_phys) cause no fault
 * and meaningless output.  Cached keys and values, and those of the tree's tokens, must be finite;
 * rows past the lengths may hold anything. */
#define MSA_TREE_MAX_TOKENS 64

/* The tree's masks from parents int32 [batch, n_tokens], and (positions may be NULL) the tokens'
 * positions int32 [batch, n_tokens], -1 for absent ones.  A token is absent when its parent is not
 * in [-1, i), or is absent. */
msa_status msa_tree_mask(const msa_shape* shape, const int32_t* seq_lens, const int32_t* parents,
                         uint64_t* mask, int32_t* positions, void* stream);

/* Index keys in 8 bits: 128 * (index_dim + 1) bytes for a block of 128 keys against 256 * index_dim
 * in bf16.  Every key (row) has a power of two of its own: with amax its largest magnitude
 *   e = the least integer >= -126 with amax <= 448 * 2^e
 *   code = x * 2^-e rounded to nearest even to the 8-bit float of 4 exponent and 3 fraction bits
 *   value = code * 2^e                                (what the cache holds; exact in bf16)
 * |value - x| <= max(2^-4 |x|, 2^(e - 10)).  A row with a NaN or an infinity is stored as NaN; it
 * gives its block an unspecified score.  Values of 2^128 or more (amax above 1.9375 * 2^127) read
 * back as infinity.
 * cache   uint8 [n_phys, 128 * (index_dim + 1)], 16-byte aligned.  One record:
 *   [0, 128 d)        codes of key j, dim i at j * d + i            (d = index_dim)
 *   [128 d, 128 d + 128)  e + 127 of key j (255: the NaN row)
 * With a block_table logical block j of sequence b is physical block block_table[b, j]; without
 * one it is b * n_blocks + j, and n_phys must be batch * n_blocks.
 * shape: of any step over this cache (batch, seq_k, index_dim, block_size = 128 and dtype matter).
 * x, y: [batch, n, index_dim] of the shape's dtype.  Token i of sequence b is at position
 * starts[b] + i, or, with starts NULL, at seq_lens[b] - n + i; positions outside [0, seq_lens[b])
 * are not stored, and their rows of y are left as they are.  seq_lens NULL: every length is
 * seq_k.  Only the stored tokens' bytes change. */
msa_status msa_index_pack(const msa_shape* shape, int32_t n_new, const int32_t* starts,
                          const int32_t* seq_lens, const int32_t* block_table, int32_t n_phys,
                          const void* x, void* cache, void* stream);
msa_status msa_index_unpack(const msa_shape* shape, int32_t n_out, const int32_t* starts,
                            const int32_t* seq_lens, const int32_t* block_table, int32_t n_phys,
                            const void* cache, void* y, void* stream);

/* msa_index_scores for the tokens of a tree, each for itself: the maximum over the keys it sees
 * of every block, -inf for a block without one.  At most 64 KV heads.
 *   packed = 1: idx_k is the 8-bit cache above, idx_draft uint8 [batch, 128 * (index_dim + 1)] the
 *               drafts' keys in one record a sequence, token i its row i (msa_index_pack with
 *               seq_k = n_tokens, starts and seq_lens NULL); block_size 128;
 *   packed = 0: idx_k of the shape's dtype, [batch, seq_k, index_dim] or pools [n_phys, block_size,
 *               index_dim]; idx_draft [batch, n_tokens, index_dim].
 * Products are exact and accumulated in fp32 (bf16 queries of 128 dims against 8-bit keys take
 * three 8-bit parts that hold all of a dim's digits if it is 2^-23 of the query's largest or more;
 * smaller ones are off by at most 2^-31 of the largest, which is 2^-110 or more; 8-bit keys are below
 * 2^100 in magnitude). */
msa_status msa_index_scores_tree(const msa_shape* shape, const int32_t* seq_lens,
                                 const int32_t* block_table, int32_t n_phys, const uint64_t* mask,
                                 const void* idx_q, const void* idx_k, const void* idx_draft,
                                 int32_t packed, float* block_scores, void* stream);

/* msa_block_topk for the tokens of a tree: the block of the token's position, and the best
 * top_k - 1 of those before it. */
msa_status msa_block_topk_tree(const msa_shape* shape, const int32_t* seq_lens,
                               const uint64_t* mask, const float* block_scores, int32_t* sel,
                               void* stream);

/* Attention of the tree's tokens: msa_sparse_decode for each, over the keys it sees in its selected
 * blocks.  k, v: [batch, n_heads_kv, seq_k, head_dim], or pools [n_phys, n_heads_kv, block_size,
 * head_dim].  lse may be NULL.  Entries of sel outside [0, the token's own block] are skipped;
 * entries must be distinct.  At most 64 query heads per KV head, top_k at most 2^20.  bf16 in blocks of 128 runs on
 * the tensor cores, which read a block once for the tokens (256 query heads of a KV head at a
 * time) that selected it.  workspace: msa_workspace_bytes(shape, 5) bytes, 16-byte aligned. */
msa_status msa_sparse_decode_tree(const msa_shape* shape, const int32_t* seq_lens,
                                  const int32_t* block_table, int32_t n_phys, const uint64_t* mask,
                                  const void* q, const void* k, const void* v, const void* k_draft,
                                  const void* v_draft, const int32_t* sel, void* out, float* lse,
                                  void* workspace, size_t ws_bytes, void* stream);

/* Moves the accepted tokens' rows into the caches: row accepted[b, i] of every source goes to
 * position seq_lens[b] + i, and new_lens[b] = seq_lens[b] + the number of them.  accepted int32
 * [batch, n_accept] (n_accept at most 64): a sequence's list ends at its first entry outside [0,
 * n_tokens), or where the cache is full.  Nothing else in the caches changes.  new_lens may be
 * seq_lens itself.  The rows are stored as they are, so the tokens must be ones that the tree has: an
 * absent token's may hold anything, and cached rows must be finite.  msa_tree_commit_masked, given
 * the tree's mask [batch, n_tokens] and the step's seq_lens, ends a list at an absent token too (mask
 * NULL: it is msa_tree_commit).  Up to MSA_COMMIT_MAX_TENSORS caches a call:
 *   packed = 0: src [batch, n_heads, n_tokens, row_bytes]; dst [batch, n_heads, seq_k, row_bytes],
 *               or with a block_table pools [n_phys, n_heads, block_size, row_bytes];
 *   packed = 1: 8-bit index keys (n_heads 1, row_bytes = index_dim 64 or 128, block_size 128):
 *               src one record a sequence, dst the cache.
 * row_bytes: a multiple of 16; n_heads * row_bytes at most 2^24.  Without a block_table n_phys must
 * be batch * n_blocks.  A position whose table entry is outside [0, n_phys) is not stored.  No dst
 * may overlap another buffer of the call.  tensors is a host array, read before the call returns. */
#define MSA_COMMIT_MAX_TENSORS 8
typedef struct msa_commit_tensor {
  const void* src;
  void* dst;
  int32_t n_heads;
  int32_t row_bytes;
  int32_t packed;
} msa_commit_tensor;
msa_status msa_tree_commit(const msa_shape* shape, const int32_t* seq_lens,
                           const int32_t* block_table, int32_t n_phys, const int32_t* accepted,
                           int32_t n_accept, const msa_commit_tensor* tensors, int32_t n_tensors,
                           int32_t* new_lens, void* stream);
msa_status msa_tree_commit_masked(const msa_shape* shape, const int32_t* seq_lens,
                                  const int32_t* block_table, int32_t n_phys, const uint64_t* mask,
                                  const int32_t* accepted, int32_t n_accept,
                                  const msa_commit_tensor* tensors, int32_t n_tensors,
                                  int32_t* new_lens, void* stream);

/* Scratch bytes msa_sparse_prefill (which = 0), msa_sparse_decode (which = 1),
 * msa_sparse_prefill_backward (which = 2), msa_index_kl_loss (which = 3),
 * msa_sparse_decode_mass (which = 4) or msa_sparse_decode_tree (which = 5, a tree's shape) needs
 * for this shape; 0 when none.  Returns 0 for an
 * invalid shape. */
size_t msa_workspace_bytes(const msa_shape* shape, int which);

/* Synchronises `stream`, then reports (and clears) the device status word and any pending
 * CUDA error: MSA_OK, MSA_ERR_TIMEOUT or MSA_ERR_CUDA. */
msa_status msa_get_device_status(void* stream);

/* Static description of a status code. */
const char* msa_status_string(msa_status status);

/* Human-readable detail of the last failure on the calling thread ("" if none). */
const char* msa_last_error(void);

/* Test hook for the failure path.  mode 1: every tensor-core sparse-prefill launch made
 * afterwards (from any thread) has its copy-issuing warp issue nothing, so the warps that
 * wait for the copies give up after their one-second bound, the kernel writes zeros and
 * -inf, and the next msa_get_device_status() reports MSA_ERR_TIMEOUT.  No copy or MMA is
 * ever in flight in this mode, and the CUDA context stays usable.  mode 2: in every tensor-core
 * decode launch, the CTA of a row's first split issues only the copy of its first block, so it
 * gives up in the same way if it has another.  Over drafted tokens: attention issues K of its first
 * block and V of half of it, and gives up on that block too; index scores issue the first tile of a
 * sequence's first range (the drafts, where the range is the sequence's last) and write -inf for
 * the blocks they have not reached.  mode 0 (default): normal operation.  Any other mode:
 * MSA_ERR_INVALID_ARG. */
msa_status msa_debug_set_fault(int32_t mode);

/* MSA_ABI_VERSION of the loaded library. */
int32_t msa_abi_version(void);

/* 1 when the library was built with -DMSA_DEBUG, else 0.  A debug build checks on the
 * device, before the kernels of each call run, every selection entry it is given (-1 or a
 * block of the sequence: below ceil(seq_k / block_size), or below ceil(seq_lens[b] /
 * block_size) for a paged cache; no block twice in a row), every block-table entry of the
 * sequence's blocks (within [0, n_phys)) and every cache length (within [0, seq_k]); and,
 * inside the tensor-core kernels, the coordinates of their tensor copies and the indices of
 * their output stores.  A failed check records a code in the device status word, which
 * msa_get_device_status() reports as MSA_ERR_BOUNDS; no check traps, and an out-of-range
 * store is skipped.  Release builds carry none of these checks (they skip selection entries
 * outside [0, n_blocks) without reporting them). */
int32_t msa_debug_build(void);

#ifdef __cplusplus
}
#endif

#endif /* MSA_H_ */
