// Plan of a chunk step: pages from the free list, slots and positions of the new rows, and
// the lengths after the step (KV Cache + Speculative Decoding Interview Cheat Sheet, section
// 5: logical rows in fixed-size pages behind a block table).
//
//   total_b = len_b + n_b,  need_b = max(0, ceil(total_b / 128) - held_b),
//   end_b = need_0 + .. + need_b (sequences that fit the capacity),
//   page i of need_b = free[taken + end_b - need_b + i],
//   slot of a row at position p = table[b][p / 128] * 128 + p % 128.
//
// A few KB of integers: the launch and its chain of dependent loads are the cost. Every CTA
// makes the whole plan of the sequences for itself (a prefix sum over their needs) and then
// gives 1024 rows their slots, a page beyond those held coming straight from the free list; the
// first CTA writes what belongs to the sequences. So no CTA waits for another, unless the
// caller's outputs are the inputs (pages held, pages taken): then the CTAs are one cluster, and
// the first writes once all have read. (One cluster whose first CTA plans for the others took
// 13 us for 69687 rows of 256 sequences: two more dependent loads and a cluster barrier.)
// Measured (replayed in a graph): 512 rows of 32 sequences 3.5 to 3.8 us, 69687 rows of 256 4.5 to
// 4.8 us; in place 3.8 and 12.0 us (a cluster has eight CTAs at most).
#include "chunk.cuh"
#include "sm100_ptx.cuh"

namespace dflash {
namespace {

constexpr int kThreads = 1024;
constexpr int kPage = 128;
constexpr int kRefused = -2147483647;  // no shift is that small: lengths and row numbers are >= 0

__global__ void __launch_bounds__(kThreads) chunk_map_kernel(const ChunkMapParams p) {
  extern __shared__ int smem[];
  int* cu_s = smem;                     // [batch + 1]
  int* shift_s = cu_s + p.batch + 1;    // [batch] position = row + shift, or refused
  int* held_s = shift_s + p.batch;      // [batch] pages held before
  int* from_s = held_s + p.batch;       // [batch] place of its first new page in the free list
  __shared__ long long warp_tot[kThreads / 32];
  __shared__ long long carry;
  __shared__ int taken_sum;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool first_cta = blockIdx.x == 0;
  if (threadIdx.x == 0) {
    carry = 0;
    taken_sum = 0;
    cu_s[p.batch] = p.cu_rows[p.batch];
  }
  const int head = p.paged ? *p.taken : 0;
  const long long avail = (long long)p.n_free - head;
  unsigned bad = p.paged && head < 0 ? DFLASH_DEV_CAPACITY : 0u;
  for (int base = 0; base < p.batch; base += kThreads) {
    const int b = base + threadIdx.x;
    bool fits = false;
    int held = 0, need = 0, lo = 0, len = 0;
    long long total = 0;
    if (b < p.batch) {
      lo = p.cu_rows[b];
      const int hi = p.cu_rows[b + 1];
      len = p.lens[b];
      held = p.paged ? p.held[b] : 0;
      cu_s[b] = lo;
      total = (long long)len + hi - lo;
      if (lo < 0 || hi < lo || hi > p.rows) {
        bad |= DFLASH_DEV_ROWS;
      } else if (len < 0 || total > p.capacity || held < 0 || held > p.pages_per_seq || head < 0) {
        bad |= DFLASH_DEV_CAPACITY;
      } else {
        fits = true;
        if (p.paged) need = max(0, (int)((total + kPage - 1) / kPage) - held);
      }
    }
    // inclusive prefix sum of the pages asked for
    long long v = need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) warp_tot[warp] = v;
    __syncthreads();
    if (warp == 0) {
      long long t = warp_tot[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) t += u;
      }
      warp_tot[lane] = t;
    }
    __syncthreads();
    const long long end = carry + (warp > 0 ? warp_tot[warp - 1] : 0) + v;
    const bool ok = fits && (need == 0 || end <= avail);
    if (fits && !ok) bad |= DFLASH_DEV_CAPACITY;
    const int got = ok ? need : 0;
    if (b < p.batch) {
      shift_s[b] = ok ? len - lo : kRefused;
      held_s[b] = held;
      from_s[b] = (int)(head + end - need);
    }
    if (p.alias) ptx::cluster_sync();  // every CTA has read this part of the inputs
    if (first_cta) {
      if (b < p.batch) {
        p.kv_lens[b] = ok ? (int)total : 0;
        if (p.paged) p.held_out[b] = held + got;
      }
      // the new pages of this warp's sequences, one per lane: the sequence of the k-th page is
      // the first whose running count exceeds k
      int upto = got;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += u;
      }
      const int pages = __shfl_sync(0xffffffffu, upto, 31);
      for (int k0 = 0; k0 < pages; k0 += 32) {
        const int k = k0 + lane;
        int l = 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          if (__shfl_sync(0xffffffffu, upto, l + o - 1) <= k) l += o;
        l = min(l, 31);
        const int n = __shfl_sync(0xffffffffu, got, l), h = __shfl_sync(0xffffffffu, held, l);
        const int i = k - (__shfl_sync(0xffffffffu, upto, l) - n);
        const long long at = head + __shfl_sync(0xffffffffu, end, l) - n + i;
        if (k < pages) {
          const int id = p.free_pages[at];
          p.table[(size_t)(base + warp * 32 + l) * p.pages_per_seq + h + i] = id;
          if (id < 0 || id >= p.n_pages) bad |= DFLASH_DEV_PAGE;
        }
      }
      const int warp_got = __reduce_add_sync(0xffffffffu, got);
      if (lane == 0 && warp_got) atomicAdd(&taken_sum, warp_got);
    }
    __syncthreads();
    if (threadIdx.x == 0) carry += warp_tot[kThreads / 32 - 1];
    __syncthreads();
  }
  if (first_cta) {
    if (p.paged && threadIdx.x == 0) *p.taken_out = head + taken_sum;
    bad = __reduce_or_sync(0xffffffffu, bad);
    if (lane == 0 && bad) atomicOr(p.status, bad);
  }
  // rows: the sequence by binary search (the last b with cu[b] <= r)
  for (long long r = (long long)blockIdx.x * kThreads + threadIdx.x; r < p.rows; r += (long long)gridDim.x * kThreads) {
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cu_s[mid] <= r) lo = mid; else hi = mid;
    }
    int slot = -1, pos = -1;
    if (r >= cu_s[lo] && r < cu_s[lo + 1] && shift_s[lo] != kRefused) {
      pos = (int)r + shift_s[lo];
      if (p.paged) {
        const int i = pos / kPage, mine = held_s[lo];
        const int page = i < mine ? p.table[(size_t)lo * p.pages_per_seq + i] : p.free_pages[from_s[lo] + i - mine];
        if (page >= 0 && page < p.n_pages) {
          slot = page * kPage + pos % kPage;
        } else {
          pos = -1;
          atomicOr(p.status, DFLASH_DEV_PAGE);
        }
      } else {
        slot = lo * p.capacity + pos;
      }
    }
    p.slots[r] = slot;
    p.positions[r] = pos;
  }
}

}  // namespace

cudaError_t chunk_map(const ChunkMapParams& p, cudaStream_t s) {
  static SmemLimit limit;
  cudaError_t e = limit.raise(chunk_map_kernel, (4 * kChunkMaxBatch + 1) * (int)sizeof(int));
  if (e != cudaSuccess) return e;
  LaunchScope ls_(DFLASH_KERNEL_CHUNK_MAP, s);
  // a row per thread; a cluster is eight CTAs at most
  const long long full = ((long long)p.rows + kThreads - 1) / kThreads, most = p.alias ? 8 : chunk_sms();
  const int ctas = (int)(full < 1 ? 1 : full > most ? most : full);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)(4 * p.batch + 1) * sizeof(int);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = p.alias ? ctas : 1;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_map_kernel, p);
}

}  // namespace dflash
