// Acceptance of a verified tree, on the device: from node 0 (the anchor) to the child whose token
// is the target's next token at the node, the lowest such child, as long as there is one. (The
// chain of dflash_accept is the tree in which every node has one child.)
//
// next(p) = min {i > p : parent(i) = p, token(i) = posterior(p)} is found for all nodes at once,
// a lane per row with a minimum in shared memory; the path is then one load a step. A warp per
// sequence; the CTAs are one cluster of at most sixteen, which the prefix sum of the accepted
// rows needs (totals exchanged through distributed shared memory).
//
// Bound by latency: a load of the lengths, of the rows, of the posterior at their parents, the minima,
// the walk, a cluster barrier. 32 trees of 64 nodes 3.4 us in a replayed graph, 512 trees of 17 to 200
// nodes 7.1 (a warp there has a sequence, and an SM 32 of them). Eight CTAs, two sequences a warp: 9.4;
// a second launch for the prefix sum would cost about 2. Trees of more than kNext rows, which a warp's
// shared memory does not hold, are walked node by node with a vote over 32 rows at a time.
#include <cooperative_groups.h>
#include <limits.h>

#include "tree.cuh"

namespace dflash {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kNext = 512;  // rows of a tree whose successors fit a warp's share of shared memory
constexpr int kCtas = 16;                     // more than eight is not portable, but fits a GPC here
constexpr int kPer = kChunkMaxBatch / kCtas;  // sequences of a CTA, at most

struct Smem {
  int next[kWarps][kNext];
  int rows[kPer];  // accepted rows
  int warp_tot[kWarps];
  int total;
};

__global__ void __launch_bounds__(kThreads) tree_accept_kernel(const TreeAcceptParams p, int per) {
  extern __shared__ int4 smem4[];
  Smem& sh = *reinterpret_cast<Smem*>(smem4);
  grid_wait();
  grid_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s0 = (int)blockIdx.x * per, s1 = min(p.batch, s0 + per);
  int* next = sh.next[warp];
  for (int b = s0 + warp; b < s1; b += kWarps) {
    const int lo = p.cu_rows[b], hi = p.cu_rows[b + 1];
    int n = hi - lo, len = 0, cur = 0, anchor = -1;
    if (lo < 0 || hi < lo || hi > p.rows) {
      if (lane == 0) atomicOr(p.status, DFLASH_DEV_ROWS);
      n = 0;
    }
    if (p.kv_lens[b] <= 0) n = 0;
    const int32_t* par = p.parents + lo;
    const int32_t* tok = p.tokens + lo;
    const int32_t* post = p.posterior + lo;
    int32_t* path = p.path + (size_t)b * p.max_path;
    if (n > 0 && n <= kNext) {
      for (int i = lane; i < n; i += 32) next[i] = INT_MAX;
      __syncwarp();
      for (int i = lane; i < n; i += 32) {
        const int u = par[i];
        if (u >= 0 && u < i && tok[i] == post[u]) atomicMin(next + u, i);
      }
      __syncwarp();
      for (;;) {
        if (lane == 0) path[len] = cur;
        ++len;
        const int to = next[cur];
        if (to == INT_MAX || len == p.max_path) break;
        cur = to;
      }
      __syncwarp();  // the next sequence writes these
    } else if (n > 0) {
      for (;;) {
        if (lane == 0) path[len] = cur;
        ++len;
        const int want = post[cur];
        unsigned hit = 0;
        int base = cur & ~31;
        for (; base < n && !hit; base += 32) {
          const int i = base + lane;
          hit = __ballot_sync(0xffffffffu, i < n && i > cur && par[i] == cur && tok[i] == want);
        }
        if (!hit || len == p.max_path) break;
        cur = base - 32 + __ffs(hit) - 1;
      }
    }
    if (n > 0) anchor = post[cur];
    for (int i = len + lane; i < p.max_path; i += 32) path[i] = -1;
    if (lane == 0) {
      p.accept_len[b] = len - 1;
      p.next_anchor[b] = anchor;
      p.ctx_next[b] = p.ctx_len[b] + len;
      sh.rows[b - s0] = len;
    }
  }
  __syncthreads();
  // inclusive prefix sum over this CTA's sequences (at most one per thread)
  const int mine = s0 + (int)threadIdx.x;
  int v = mine < s1 ? sh.rows[threadIdx.x] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) sh.warp_tot[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int t = sh.warp_tot[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += u;
    }
    sh.warp_tot[lane] = t;
    if (lane == 31) sh.total = t;
  }
  __syncthreads();
  if (warp > 0) v += sh.warp_tot[warp - 1];
  if (gridDim.x > 1) {
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    for (unsigned c = 0; c < blockIdx.x; ++c) v += *cl.map_shared_rank(&sh.total, c);
    cl.sync();  // no CTA leaves while another reads its total
  }
  if (mine < s1) p.next_cu_rows[mine + 1] = v;
  if (blockIdx.x == 0 && threadIdx.x == 0) p.next_cu_rows[0] = 0;
}

}  // namespace

cudaError_t tree_accept(const TreeAcceptParams& p, cudaStream_t s) {
  static SmemLimit limit;
  cudaError_t e = limit.raise(tree_accept_kernel, (int)sizeof(Smem), true);
  if (e != cudaSuccess) return e;
  LaunchScope ls_(DFLASH_KERNEL_TREE_ACCEPT, s);
  const int want = (p.batch + kWarps - 1) / kWarps, ctas = want > kCtas ? kCtas : want;
  const int per = (p.batch + ctas - 1) / ctas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Smem);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, tree_accept_kernel, p, per);
}

}  // namespace dflash
