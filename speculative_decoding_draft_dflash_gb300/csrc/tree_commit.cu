// Commits an accepted path: cache row ctx + path[i] of a sequence becomes its row ctx + i, K and V of
// every layer, and the sequence's length ctx + a + 1.
//
// The path ascends, so path[i] >= i: in this order a row is read before anything is written over
// it. A thread holds one 16-byte (or 8-byte) column of all the path's rows and moves them in that
// order, up to eight rows loaded before the first is stored; no other thread touches its column,
// so nothing has to be waited for. A CTA per sequence, layer and K or V.
//
// Bound by loads in flight. 16 layers of 64 sequences, paths of 4 to 16 nodes, 8 heads of 128 in bf16:
// 64 MB read and written, 14.5 us in a replayed graph (4.4 TB/s; the copy rate allows 9.4 us): each CTA moves
// a few KB in runs of 256 bytes, behind three dependent loads (lengths, path, pages). Eight CTAs on an SM, by 64
// registers: 16.0 us with as many registers as the loads would like, 14.7 with nine, 15.9 and 18.1 with ten and
// twelve, which spill; four rows in flight instead of eight 15.5. Two layers of 32 sequences, 1.3 MB: 3.2 us.
#include "tree.cuh"

namespace dflash {
namespace {

constexpr int kRows = 64;  // rows whose addresses are in shared memory at a time
constexpr int kAhead = 8;  // rows in flight per thread

template <typename T>
__global__ void __launch_bounds__(128, 8) tree_commit_kernel(const TreeCommitParams p) {
  __shared__ long long src[kRows], dst[kRows];  // row of KV head 0 in the layer, -1: not moved
  grid_wait();
  const int b = blockIdx.x, l = blockIdx.y >> 1, which = blockIdx.y & 1;
  const int a = p.accept_len[b], ctx = p.ctx_len[b], nodes = p.nodes[b];
  if (a == -1) return;
  const bool first = blockIdx.y == 0 && threadIdx.x == 0;
  bool bad = a < 0 || a >= p.max_path || nodes < 0 || nodes > p.max_nodes || ctx < 0 || nodes > p.capacity - ctx;
  const int32_t* path = p.path + (size_t)b * p.max_path;
  if (!bad) {
    bool mine = false;
    for (int i = threadIdx.x; i <= a; i += blockDim.x) {
      const int u = path[i];
      mine |= u < 0 || u >= nodes || (i > 0 && path[i - 1] >= u);
    }
    bad = __syncthreads_or(mine);
  }
  if (bad) {
    if (first) atomicOr(p.status, DFLASH_DEV_TREE);
    return;
  }
  if (which == 0 && threadIdx.x == 0) p.lens[(size_t)l * p.batch + b] = ctx + a + 1;
  char* base = (which ? p.cache_v : p.cache_k) + l * p.layer_bytes;
  const int per_row = p.row_bytes / (int)sizeof(T), cols = p.n_kv * per_row;
  auto row_of = [&](int slot) -> long long {
    if (!p.block_table) return (long long)b * p.n_kv * p.unit_rows + slot;
    const int page = p.block_table[(size_t)b * p.pages_per_seq + (slot >> 7)];
    if (page < 0 || page >= p.n_pages) {
      atomicOr(p.status, DFLASH_DEV_PAGE);
      return -1;
    }
    return (long long)page * p.n_kv * p.unit_rows + (slot & 127);
  };
  for (int i0 = 0; i0 <= a; i0 += kRows) {
    const int m = min(kRows, a + 1 - i0);
    if (i0 > 0) __syncthreads();
    for (int i = threadIdx.x; i < m; i += blockDim.x) {
      const int u = path[i0 + i];
      const long long to = u == i0 + i ? -1 : row_of(ctx + i0 + i), from = to < 0 ? -1 : row_of(ctx + u);
      src[i] = from;
      dst[i] = from < 0 ? -1 : to;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += blockDim.x) {
      const int h = c / per_row, e = c - h * per_row;
      char* col = base + (size_t)h * p.unit_rows * p.row_bytes + (size_t)e * sizeof(T);
      for (int i = 0; i < m; i += kAhead) {
        T v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (i + k < m && src[i + k] >= 0) v[k] = *reinterpret_cast<const T*>(col + src[i + k] * p.row_bytes);
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (i + k < m && src[i + k] >= 0) *reinterpret_cast<T*>(col + dst[i + k] * p.row_bytes) = v[k];
      }
    }
  }
}

}  // namespace

cudaError_t tree_commit(const TreeCommitParams& p, cudaStream_t s) {
  LaunchScope ls_(DFLASH_KERNEL_TREE_COMMIT, s);
  const dim3 grid(p.batch, 2 * p.n_layers);
  return launch_overlapped(p.row_bytes % 16 == 0 ? tree_commit_kernel<uint4> : tree_commit_kernel<uint2>, grid, 128, 0, s, p);
}

}  // namespace dflash
