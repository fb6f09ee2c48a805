// Positions, depths and ancestor masks of a step's rows, the newest nodes of their sequences' trees:
//
//   node = nodes before the step + place among the sequence's rows
//   depth(node) = depth(parent) + 1 (no parent: 0), position = committed rows + depth,
//   mask(node) = mask(parent) | bit(node)
//
// A CTA per sequence, a warp per row: the warp follows the parents through shared memory and sets
// a bit per step, each lane holding words of the mask, up to the first node whose mask is complete
// (one of an earlier step, or of an earlier block of kBlock rows), which it takes over. So a row
// costs its depth in shared-memory latencies, and a chain of thousands of rows stays linear.
//
// Bound by latency: 58 to 220 KB of masks are a few hundredths of a microsecond at the copy rate. 32 trees of
// 64 nodes 2.9 us in a replayed graph, 16 new rows behind 200 to 900 nodes of 64 sequences 2.5 (5.0 and 4.7
// call by call, which is the host's time): the launch, then three dependent loads (lengths, parents, the
// masks taken over) and the walk.
#include "tree.cuh"

namespace dflash {
namespace {

constexpr int kBlock = 128;  // rows between two barriers

// NW: mask words of a lane.
template <int NW>
__global__ void __launch_bounds__(1024) tree_map_kernel(const TreeMapParams p) {
  __shared__ int up[kTreeMaxNodes];
  grid_wait();
  const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int lo = p.cu_rows[b], hi = p.cu_rows[b + 1], kv = p.kv_lens[b];
  const int t0 = p.nodes_before ? p.nodes_before[b] : 0;
  if (lo < 0 || hi < lo || hi > p.rows) {
    if (threadIdx.x == 0) {
      atomicOr(p.status, DFLASH_DEV_ROWS);
      p.nodes[b] = t0;
      p.kv_lens[b] = 0;
    }
    return;
  }
  const int n = hi - lo;
  if (n == 0) {
    if (threadIdx.x == 0) p.nodes[b] = t0;
    return;
  }
  // kv 0: the step refused the sequence already
  bool bad = kv != 0 && (t0 < 0 || n > p.max_nodes - t0 || kv < t0 + n);
  if (!bad && kv != 0) {
    bool mine = false;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const int u = p.parents[lo + i];
      up[i] = u;
      mine |= u < -1 || u >= t0 + i;
    }
    bad = __syncthreads_or(mine);
  }
  if (bad || kv == 0) {
    for (int i = threadIdx.x; i < n; i += blockDim.x) p.slots[lo + i] = p.positions[lo + i] = -1;
    if (threadIdx.x == 0) {
      if (bad) atomicOr(p.status, DFLASH_DEV_TREE);
      p.nodes[b] = t0;
      p.kv_lens[b] = 0;
    }
    return;
  }
  if (threadIdx.x == 0) p.nodes[b] = t0 + n;
  const int ctx = kv - n - t0, words = p.max_nodes >> 5;
  const size_t row0 = (size_t)b * p.max_nodes;
  for (int base = 0; base < n; base += kBlock) {
    const int end = min(n, base + kBlock), known = t0 + base;  // nodes below `known` are complete
    for (int i = base + warp; i < end; i += nw) {
      uint32_t m[NW] = {};
      int node = t0 + i, depth = 0;
      while (node >= known) {
#pragma unroll
        for (int k = 0; k < NW; ++k)
          if ((node >> 5) == lane + 32 * k) m[k] |= 1u << (node & 31);
        node = up[node - t0];
        depth += node >= 0;
      }
      if (node >= 0) {
        depth += p.depths[row0 + node];
#pragma unroll
        for (int k = 0; k < NW; ++k)
          if (lane + 32 * k < words) m[k] |= p.masks[(row0 + node) * words + lane + 32 * k];
      }
#pragma unroll
      for (int k = 0; k < NW; ++k)
        if (lane + 32 * k < words) p.masks[(row0 + t0 + i) * words + lane + 32 * k] = m[k];
      if (lane == 0) {
        p.depths[row0 + t0 + i] = depth;
        p.positions[lo + i] = ctx + depth;
      }
    }
    if (end < n) __syncthreads();
  }
}

}  // namespace

cudaError_t tree_map(const TreeMapParams& p, cudaStream_t s) {
  LaunchScope ls_(DFLASH_KERNEL_TREE_MAP, s);
  // a warp for each of a sequence's rows, on average
  const int per = p.rows / p.batch + 1, warps = per < 4 ? 4 : per > 32 ? 32 : per;
  const int words = p.max_nodes / 32;
  return launch_overlapped(words <= 32 ? tree_map_kernel<1> : words <= 64 ? tree_map_kernel<2> : tree_map_kernel<4>,
                           dim3(p.batch), 32 * warps, 0, s, p);
}

}  // namespace dflash
