// The chunk step (map, append, causal attention): parameters of its kernels, and the work
// split that both attention kernels and their merge share.
#pragma once

#include "dflash_internal.cuh"

namespace dflash {

constexpr int kChunkMaxBatch = 8192;  // sequences of a step (prefix sums live in shared memory)

struct ChunkMapParams {
  const int32_t* cu_rows;
  const int32_t* lens;
  int32_t* kv_lens;
  int32_t* slots;
  int32_t* positions;
  // paged: the pool (null otherwise)
  int32_t* table;
  const int32_t* held;
  int32_t* held_out;
  const int32_t* free_pages;
  const int32_t* taken;
  int32_t* taken_out;
  unsigned* status;
  int batch, rows, capacity, pages_per_seq, n_pages, n_free;
  bool paged;
  bool alias;  // held_out is held, or taken_out is taken
};
int chunk_sms();  // SMs of the current device

cudaError_t chunk_map(const ChunkMapParams& p, cudaStream_t s);

struct ChunkAppendParams {
  const int32_t* slots;
  const int32_t* positions;
  const int32_t* kv_lens;
  int32_t* lens;          // this layer's
  const void* q;          // or null
  const void* k;
  const void* v;
  long long ld_q, ld_k, ld_v;
  const void* gamma_q;    // or null: no norm
  const void* gamma_k;
  const float2* rope;     // or null: no rotation
  void* q_out;
  void* cache_k;          // layer base: units of [n_kv][unit_rows][d_h] (a page, or a sequence)
  void* cache_v;
  unsigned* status;
  long long n_slots;      // units * unit_rows
  int unit_rows;
  int batch, rows, capacity, n_h, n_kv, d_h, table_len;
  float eps, k_inv, v_inv;  // E4M3: codes of x * inv, inv = 1 / scale
  bool fp8;
};
cudaError_t chunk_append(int dtype, const ChunkAppendParams& p, cudaStream_t s);

struct ChunkAttnParams {
  const int32_t* cu_rows;
  const int32_t* kv_lens;
  const void* q;
  long long ld_q;
  const void* cache_k;        // layer base
  const void* cache_v;
  const int32_t* block_table; // paged, or null
  void* out;                  // [rows][n_h * d_h]
  float* part;                // [2 * CTAs] partial items (rows x d_h), not normalised
  float2* part_ml;            // [2 * CTAs][rows of an item]: (maximum, sum) of each partial row
  int4* merge;                // [CTAs]: {sequence, KV head, item, pieces} of the range cut in CTA c
  unsigned* status;
  int batch, rows, n_h, n_kv, d_h, G, capacity, pages_per_seq, n_pages, window;
  float scaling, k_scale, v_scale;
  bool fp8;
};

size_t chunk_attn_workspace(int dtype, int d_h);
// Carves part, part_ml and merge out of the workspace; false when it is too small.
bool chunk_attn_carve(int dtype, int d_h, ChunkAttnParams& p, void* workspace, size_t bytes);
cudaError_t chunk_attn(int dtype, const ChunkAttnParams& p, cudaStream_t s);
int chunk_attn_simt_item_rows(int d_h);
int chunk_attn_simt_ctas(int d_h);
cudaError_t chunk_attn_simt(const ChunkAttnParams& p, cudaStream_t s);  // f32
cudaError_t chunk_attn_tc(const ChunkAttnParams& p, cudaStream_t s);    // bf16
int chunk_attn_tc_item_rows(int G);

// ---------------------------------------------------------------------------
// The work split. The query rows of (sequence b, KV head) are its n new rows times the G
// query heads that share the KV head, stacked row-major (row = token * G + head). An item
// is `item_rows` consecutive stacked rows with all their key tiles; all items lie end to end as
// one line of costs (a fixed cost each, plus one per key tile) and CTA c works on
// [total * c / n, total * (c + 1) / n) of it, cutting items where its share begins or ends.
// A piece of a cut item leaves an fp32 partial in the workspace (at most two per CTA: the
// end of an item begun before, and the start of one continued after), so the workspace
// depends on the number of CTAs alone. Every CTA derives its share from the lengths by
// itself: no list, no launch of its own, nothing read back to the host.
// ---------------------------------------------------------------------------
namespace chunk {

// TOKENS: an item is item_tokens whole tokens; else item_rows stacked rows wherever they end.
// (The functions here are compiled into a kernel whose code has to stay small: what does not
// fit the instruction cache is fetched again and again by warps that do different things.)
template <bool TOKENS>
struct Split {
  const int32_t* cu_rows;
  const int32_t* kv_lens;
  int batch, rows, n_kv, G, capacity, window;
  int item_rows;   // stacked rows of an item
  int item_tokens; // TOKENS: tokens of an item
  int half_rows;   // an item of at most so many rows has the smaller tile cost
  int tile_shift;  // log2 of a tile's keys
  // Cost units: an item, a key tile of an item, and of one of at most half_rows rows.
  int item_cost, tile_cost, half_cost;
};

struct Seq {
  int row0, n, kv;  // first row, new rows, rows held (0: refused)
};

template <bool TOKENS>
__device__ __forceinline__ Seq load_seq(const Split<TOKENS>& p, int b, unsigned* bad) {
  Seq s;
  s.row0 = p.cu_rows[b];
  s.n = p.cu_rows[b + 1] - s.row0;
  s.kv = p.kv_lens[b];
  if (s.row0 < 0 || s.n < 0 || s.n > p.rows - s.row0) {
    *bad |= DFLASH_DEV_ROWS;
    s.n = 0;
  }
  if (s.kv < 0 || s.kv > p.capacity) {
    *bad |= DFLASH_DEV_CAPACITY;
    s.kv = 0;
  }
  return s;
}

// (rows * G fits 31 bits)
template <bool TOKENS>
__device__ __forceinline__ int n_items(const Split<TOKENS>& p, const Seq& s) {
  if (TOKENS) return (int)((unsigned)(s.n + p.item_tokens - 1) / (unsigned)p.item_tokens);
  return (int)((unsigned)(s.n * p.G + p.item_rows - 1) / (unsigned)p.item_rows);
}

// Positions of the first and the last row of item t.
template <bool TOKENS>
__device__ __forceinline__ int2 item_span(const Split<TOKENS>& p, const Seq& s, int t) {
  const int p0 = s.kv - s.n;
  if (TOKENS) return make_int2(p0 + t * p.item_tokens, p0 + min((t + 1) * p.item_tokens, s.n) - 1);
  const unsigned r0 = t * p.item_rows, r1 = min(r0 + p.item_rows, (unsigned)(s.n * p.G));
  return make_int2(p0 + (int)(r0 / (unsigned)p.G), p0 + (int)((r1 - 1) / (unsigned)p.G));
}

// First key (a multiple of the tile) and key tiles of item t.
template <bool TOKENS>
__device__ __forceinline__ int2 item_keys(const Split<TOKENS>& p, const Seq& s, int t) {
  const int2 span = item_span(p, s, t);
  if (span.y < 0) return make_int2(0, 0);
  int k0 = 0;
  if (p.window > 0 && span.x >= p.window) k0 = (span.x - p.window + 1) >> p.tile_shift << p.tile_shift;
  return make_int2(k0, ((span.y - k0) >> p.tile_shift) + 1);
}

// Cost units of a key tile of item t, and of the whole item.
template <bool TOKENS>
__device__ __forceinline__ int tile_units(const Split<TOKENS>& p, const Seq& s, int t) {
  return s.n * p.G - t * p.item_rows > p.half_rows ? p.tile_cost : p.half_cost;
}
template <bool TOKENS>
__device__ __forceinline__ int item_units(const Split<TOKENS>& p, const Seq& s, int t) {
  return p.item_cost + tile_units(p, s, t) * item_keys(p, s, t).y;
}

// A CTA's share and where it starts.
struct Start {
  long long begin, end;  // on the cost line
  long long total;
  int ctas;              // CTAs with a share
  int b, kvh, t;         // the item that holds `begin`
  int off;               // cost units of it before `begin`
  Seq s;                 // its sequence
};

// CTAs that get a share: large enough for a key tile, so that every CTA inside a cut item has
// at least one.
template <bool TOKENS>
__device__ __forceinline__ int active_ctas(const Split<TOKENS>& p, long long total, int ctas) {
  const int least = max(p.tile_cost, p.half_cost);
  return total >= (long long)ctas * least ? ctas : max(1, (int)(total / least));
}
static __device__ __noinline__ long long bound(long long total, int active, int c) {
  return total * c / active;
}

// Shared scratch of locate: every sequence and its cost.
constexpr size_t kLocateBytes = sizeof(Seq) + sizeof(long long);  // per sequence

// Run by all threads of the CTA; `scratch` is 16-byte aligned shared memory of kLocateBytes per
// sequence (free again after the call and a __syncthreads), `st` shared. A thread per sequence
// reads the lengths; then eight lanes per sequence add up its items.
template <bool TOKENS>
__device__ __noinline__ void locate(const Split<TOKENS>& p, void* scratch, Start* st, unsigned* status) {
  long long* cost = reinterpret_cast<long long*>(scratch);
  Seq* seq = reinterpret_cast<Seq*>(cost + p.batch);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned bad = 0;
#pragma unroll 1
  for (int b = threadIdx.x; b < p.batch; b += blockDim.x) seq[b] = load_seq(p, b, &bad);
  if (bad && blockIdx.x == 0) atomicOr(status, bad);
  __syncthreads();
#pragma unroll 1
  for (int base = 0; base < p.batch; base += blockDim.x >> 3) {
    const int b = base + (threadIdx.x >> 3);
    long long sum = 0;
    if (b < p.batch) {
      const Seq s = seq[b];
      const int items = n_items(p, s);
#pragma unroll 1
      for (int t = threadIdx.x & 7; t < items; t += 8) sum += item_units(p, s, t);
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (b < p.batch && (threadIdx.x & 7) == 0) cost[b] = sum * p.n_kv;
  }
  __syncthreads();
  if (warp == 0) {  // prefix sums, in place
    long long carry = 0;
#pragma unroll 1
    for (int base = 0; base < p.batch; base += 32) {
      long long v = base + lane < p.batch ? cost[base + lane] : 0;
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      v += carry;
      if (base + lane < p.batch) cost[base + lane] = v;
      carry = __shfl_sync(0xffffffffu, v, 31);
    }
    __syncwarp();
    const int active = active_ctas(p, carry, (int)gridDim.x);
    const int c = (int)blockIdx.x;
    const long long begin = c < active ? bound(carry, active, c) : carry;
    const long long end = c < active ? bound(carry, active, c + 1) : carry;
    int b = 0;
    if (begin < end) {  // the first sequence whose prefix exceeds begin
      int lo = 0, hi = p.batch - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cost[mid] > begin) hi = mid; else lo = mid + 1;
      }
      b = lo;
      const Seq s = seq[b];
      const long long before = b > 0 ? cost[b - 1] : 0;
      const long long per_head = bound(cost[b] - before, p.n_kv, 1);
      int kvh = 0;
      long long rest = begin - before;
      while (rest >= per_head) {  // (n_kv steps at most)
        rest -= per_head;
        ++kvh;
      }
      // the item: scan their costs 32 at a time (their sum fits 31 bits: the capacity does)
      const int items = n_items(p, s);
      int t = 0;
#pragma unroll 1
      for (int base = 0; base < items; base += 32) {
        const int u = base + lane;
        const int w = u < items ? item_units(p, s, u) : 0;
        int v = w;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += x;
        }
        const unsigned past = __ballot_sync(0xffffffffu, v > rest);
        if (past) {
          const int l = __ffs(past) - 1;
          t = base + l;
          rest -= __shfl_sync(0xffffffffu, v - w, l);
          break;
        }
        rest -= __shfl_sync(0xffffffffu, v, 31);
      }
      if (lane == 0) {
        st->kvh = kvh;
        st->t = t;
        st->off = (int)rest;
        st->s = s;
      }
    }
    if (lane == 0) {
      st->begin = begin;
      st->end = end;
      st->total = carry;
      st->ctas = active;
      st->b = b;
    }
  }
  __syncthreads();
}

// One piece of work: key tiles [tile0, tile1) of item t of (b, kvh).
struct Piece {
  int b, kvh, t;
  int row0, n, kv;   // of the sequence
  int k0;            // first key of the item
  int tile0, tile1;
  int slot;          // -1: the whole item; else partial slot 0 or 1 of this CTA
};

// Walks a CTA's share piece by piece (one thread, or all threads of a warp alike).
template <bool TOKENS>
struct Walker {
  Split<TOKENS> p;
  Seq s;
  long long at, end, total;
  int ctas, b, kvh, t, off;
  int4 merge;  // what to merge: {b, kvh, t, pieces}, pieces 0 when nothing was cut here

  __device__ __forceinline__ void init(const Split<TOKENS>& split, const Start& st) {
    p = split;
    at = st.begin;
    end = st.end;
    total = st.total;
    ctas = st.ctas;
    b = st.b;
    kvh = st.kvh;
    t = st.t;
    off = st.off;
    merge = make_int4(0, 0, 0, 0);
    s = st.s;
  }

  __device__ __forceinline__ bool next(Piece* w) {
    while (at < end) {
      const int items = n_items(p, s);
      if (t >= items) {  // next KV head, next sequence
        t = 0;
        if (items == 0 || ++kvh >= p.n_kv) {
          kvh = 0;
          if (++b >= p.batch) return false;
          unsigned ignored = 0;
          s = load_seq(p, b, &ignored);
        }
        continue;
      }
      const int2 keys = item_keys(p, s, t);
      const int tu = tile_units(p, s, t), whole = p.item_cost + tu * keys.y;
      const int take = (int)min((long long)(whole - off), end - at);
      const int tile0 = max(0, off - p.item_cost) / tu;
      const int tile1 = off + take == whole ? keys.y : max(0, off + take - p.item_cost) / tu;
      const bool starts = off == 0;
      w->b = b;
      w->kvh = kvh;
      w->t = t;
      w->row0 = s.row0;
      w->n = s.n;
      w->kv = s.kv;
      w->k0 = keys.x;
      w->tile0 = tile0;
      w->tile1 = tile1;
      w->slot = tile0 == 0 && tile1 == keys.y ? -1 : (tile0 == 0 ? 1 : 0);
      at += take;
      off += take;
      if (w->slot == 1 && tile1 > 0) {
        // the start of an item that goes on: how many CTAs finish it
        const long long item_end = at + (whole - off);
        int c = (int)blockIdx.x + 1, n = 1;
        while (bound(total, ctas, c) < item_end) {
          ++c;
          ++n;
        }
        merge = make_int4(b, kvh, t, n);
      }
      if (off == whole) {
        ++t;
        off = 0;
      }
      if (tile1 > tile0 || (keys.y == 0 && starts)) return true;
    }
    return false;
  }
};

}  // namespace chunk
}  // namespace dflash
