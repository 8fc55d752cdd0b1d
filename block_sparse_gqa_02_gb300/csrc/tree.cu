// Around a decode step over drafted tokens: the paths of a tree from its parents, and the rows of
// the accepted tokens into the caches.  Both are small and bound by latency: one launch each (cold, 8
// sequences: 2.8 us for the paths, 8.5 for the rows, a chain of length, list, (mask,) table and row).
#include <cooperative_groups.h>

#include "index_cache.cuh"
#include "launch.cuh"
#include "ptx.cuh"
#include "tree.cuh"

namespace msa {

namespace {

namespace cg = cooperative_groups;

// One warp a sequence, tokens lane and lane + 32.  Paths by doubling: after round r a token's bits
// are those of its nearest 2^r ancestors and `up` is the next one, so six rounds reach all 64.
__global__ void __launch_bounds__(32)
tree_mask_kernel(const int32_t* __restrict__ parents, TreeWord* __restrict__ mask,
                 int32_t* __restrict__ positions, Dims p) {
  constexpr int kRoot = -1, kNone = -2;
  __shared__ TreeWord path[64];
  __shared__ int up[64];
  ptx::grid_wait();
  ptx::launch_dependents();
  const int b = blockIdx.x, lane = threadIdx.x, n = p.nR;
  const int L = seq_len_of(p, b);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = lane + 32 * h;
    path[i] = 1ull << i;
    const int up_i = i < n ? parents[(size_t)b * n + i] : kNone;
    up[i] = up_i >= kRoot && up_i < i ? up_i : kNone;
  }
  __syncwarp();
#pragma unroll
  for (int r = 0; r < 6; ++r) {
    TreeWord w[2];
    int u[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = lane + 32 * h;
      u[h] = up[i];
      w[h] = path[i];
      if (u[h] >= 0) {
        w[h] |= path[u[h]];
        u[h] = up[u[h]];
      }
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      up[lane + 32 * h] = u[h];
      path[lane + 32 * h] = w[h];
    }
    __syncwarp();
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = lane + 32 * h;
    if (i >= n) continue;
    const bool there = up[i] == kRoot && __popcll(path[i]) - 1 < p.Sk - L;
    mask[(size_t)b * n + i] = there ? path[i] : 0;
    if (positions) positions[(size_t)b * n + i] = there ? tree_pos(path[i], L) : -1;
  }
}

constexpr int kCommitThreads = 256;

struct CommitArgs {
  msa_commit_tensor t[MSA_COMMIT_MAX_TENSORS];
  int n, n_accept;
};

// A cluster a sequence (its CTAs along x): they share out the 16-byte units of the rows, and one
// of them writes the new length when all have read the old one (which may be the same word).
__global__ void __launch_bounds__(kCommitThreads)
tree_commit_kernel(const __grid_constant__ CommitArgs a, const int32_t* __restrict__ accepted,
                   int32_t* new_lens, Dims p) {
  __shared__ int node[64];
  __shared__ long long row[64];       // block_row() of the position
  __shared__ int s_count;
  cg::cluster_group cluster = cg::this_cluster();
  ptx::grid_wait();
  ptx::launch_dependents();
  const int parts = (int)cluster.num_blocks(), part = (int)cluster.block_rank();
  const int b = blockIdx.x / parts, tid = threadIdx.x;
  const int L = seq_len_of(p, b);
  if (tid < 32) {                                          // the list ends at its first non-token
    int count = 0;
    for (int i0 = 0; i0 < a.n_accept; i0 += 32) {
      const int i = i0 + tid;
      const int x = i < a.n_accept ? accepted[(size_t)b * a.n_accept + i] : -1;
      // with the masks: a token that the tree has
      const bool ok = x >= 0 && x < p.nR && i < p.Sk - L && (!p.tree_mask || tree_path(p, b, x, L));
      const unsigned bad = ~__ballot_sync(0xffffffffu, ok);
      const int good = bad ? __ffs(bad) - 1 : 32;
      if (ok && tid < good) {
        node[i] = x;
        // the physical block of the position and the row in it, or -1 where the table names none
        const int pos = L + i, blk = pos / p.Bk;
        const int phys = physical_index_block(p, b, blk);
        row[i] = phys < 0 ? -1 : (long long)phys * p.Bk + (pos - blk * p.Bk);
      }
      count += good;
      if (good < 32) break;
    }
    if (tid == 0) s_count = count;
  }
  __syncthreads();
  const int count = s_count;
  constexpr int kFlight = 4;
  for (int ti = 0; ti < a.n; ++ti) {
    const msa_commit_tensor& t = a.t[ti];
    const int per = t.row_bytes / 16;
    const int units = t.n_heads * count * per;
    const size_t src_head = t.packed ? 0 : (size_t)p.nR * t.row_bytes;
    const uint8_t* src = static_cast<const uint8_t*>(t.src) +
                         (t.packed ? (size_t)b * kIndexBlock * (t.row_bytes + 1)
                                   : (size_t)b * t.n_heads * src_head);
    uint8_t* dst = static_cast<uint8_t*>(t.dst);
    auto dst_row = [&](int h, int i) -> uint8_t* {
      if (t.packed) {                                      // a record's codes
        const long long phys = row[i] / kIndexBlock;
        return row[i] < 0 ? nullptr : dst + phys * kIndexBlock * (t.row_bytes + 1) +
                                          (row[i] - phys * kIndexBlock) * t.row_bytes;
      }
      if (!p.block_table)
        return dst + (((size_t)b * t.n_heads + h) * p.Sk + L + i) * t.row_bytes;
      const long long phys = row[i] / p.Bk;
      return row[i] < 0 ? nullptr
                        : dst + ((phys * t.n_heads + h) * p.Bk + (row[i] - phys * p.Bk)) * t.row_bytes;
    };
    for (int u0 = part * kCommitThreads + tid; u0 < units; u0 += kFlight * parts * kCommitThreads) {
      uint4 x[kFlight];
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        const int u = u0 + f * parts * kCommitThreads;
        if (u < units) {
          const int i = u / per % count, h = u / per / count;
          x[f] = *reinterpret_cast<const uint4*>(src + h * src_head +
                                                 (size_t)node[i] * t.row_bytes + u % per * 16);
        }
      }
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        const int u = u0 + f * parts * kCommitThreads;
        if (u < units) {
          const int i = u / per % count, h = u / per / count;
          uint8_t* to = dst_row(h, i);
          if (to) *reinterpret_cast<uint4*>(to + u % per * 16) = x[f];
        }
      }
    }
    if (t.packed && part == 0 && tid < count && row[tid] >= 0) {   // the rows' exponents
      const long long phys = row[tid] / kIndexBlock;
      const size_t record = (size_t)kIndexBlock * (t.row_bytes + 1);
      dst[phys * record + (size_t)kIndexBlock * t.row_bytes + (row[tid] - phys * kIndexBlock)] =
          src[(size_t)kIndexBlock * t.row_bytes + node[tid]];
    }
  }
  cluster.sync();
  if (part == 0 && tid == 0) new_lens[b] = L + count;
}

}  // namespace

cudaError_t launch_tree_mask(const Dims& p, const int32_t* parents, unsigned long long* mask,
                             int32_t* positions, cudaStream_t st) {
  return launch_after(tree_mask_kernel, dim3((unsigned)p.B), 32, 0, 0, st, parents, mask, positions,
                      p);
}

cudaError_t launch_tree_commit(const Dims& p, const int32_t* accepted, int n_accept,
                               const msa_commit_tensor* tensors, int n, int32_t* new_lens,
                               cudaStream_t st) {
  CommitArgs a;
  a.n = n;
  a.n_accept = n_accept;
  long long units = 0;
  for (int i = 0; i < n; ++i) {
    a.t[i] = tensors[i];
    units += (long long)tensors[i].n_heads * n_accept * (tensors[i].row_bytes / 16);
  }
  // CTAs of a sequence: four units a thread, at most the portable cluster
  int parts = 1;
  while (parts < 8 && units > (long long)parts * kCommitThreads * 4) parts *= 2;
  return launch_after(tree_commit_kernel, dim3((unsigned)p.B * parts), kCommitThreads, 0, parts, st, a,
                      accepted, new_lens, p);
}

}  // namespace msa
