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

// The trees of a step (dflash_tree): which rows of their own tree its rows see.
struct TreeRows {
  const int32_t* nodes;   // [batch]; null: no trees, a row sees every row before it
  const int32_t* depths;  // [batch][max_nodes]
  const uint32_t* masks;  // [batch][max_nodes][max_nodes / 32]
  int max_nodes;
};
constexpr int kTreeMaxBatch = 4096;
constexpr int kTreeMaxNodes = 4096;

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
  TreeRows tree;
};

size_t chunk_attn_workspace(int dtype, int d_h);
// Carves part, part_ml and merge out of the workspace; false when it is too small.
bool chunk_attn_carve(int dtype, int d_h, ChunkAttnParams& p, void* workspace, size_t bytes);
cudaError_t chunk_attn(int dtype, const ChunkAttnParams& p, cudaStream_t s);
int chunk_attn_simt_item_rows(int d_h);
int chunk_attn_simt_ctas(int d_h);
cudaError_t chunk_attn_simt(const ChunkAttnParams& p, cudaStream_t s);  // f32
cudaError_t chunk_attn_tc(const ChunkAttnParams& p, cudaStream_t s);    // bf16
cudaError_t tree_attn_simt(const ChunkAttnParams& p, cudaStream_t s);   // the same with trees
cudaError_t tree_attn_tc(const ChunkAttnParams& p, cudaStream_t s);
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
// TREE: a sequence's last rows are the nodes of a tree (the step's rows the newest of them), the
// rows before them committed. A row sees no key behind its own, as without a tree, so items, spans
// and costs are the same; only a window's first key depends on the tree.
template <bool TOKENS, bool TREE = false>
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
  const int32_t* nodes;  // TREE: nodes of each sequence's tree
  int max_nodes;
};

template <bool TREE>
struct Seq {
  int row0, n, kv;  // first row, new rows, rows held (0: refused)
};
template <>
struct Seq<true> {
  int row0, n, kv;
  int ctx;          // committed rows: kv less the tree's nodes
};

template <bool TOKENS, bool TREE>
__device__ __forceinline__ Seq<TREE> load_seq(const Split<TOKENS, TREE>& p, int b, unsigned* bad) {
  Seq<TREE> s;
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
  if constexpr (TREE) {
    const int nodes = p.nodes[b];
    s.ctx = s.kv - nodes;
    if (s.kv > 0 && (nodes < s.n || nodes > p.max_nodes || s.ctx < 0)) {
      *bad |= DFLASH_DEV_TREE;
      s.kv = 0;
    }
    if (s.kv == 0) s.ctx = 0;
  }
  return s;
}

// (rows * G fits 31 bits)
template <bool TOKENS, bool TREE>
__device__ __forceinline__ int n_items(const Split<TOKENS, TREE>& p, const Seq<TREE>& s) {
  if (TOKENS ? s.n <= p.item_tokens : s.n * p.G <= p.item_rows) return s.n > 0;
  if (TOKENS) return (int)((unsigned)(s.n + p.item_tokens - 1) / (unsigned)p.item_tokens);
  return (int)((unsigned)(s.n * p.G + p.item_rows - 1) / (unsigned)p.item_rows);
}

// Positions of the first and the last row of item t.
template <bool TOKENS, bool TREE>
__device__ __forceinline__ int2 item_span(const Split<TOKENS, TREE>& p, const Seq<TREE>& s, int t) {
  const int p0 = s.kv - s.n;
  if (TOKENS) return make_int2(p0 + t * p.item_tokens, p0 + min((t + 1) * p.item_tokens, s.n) - 1);
  const unsigned r0 = t * p.item_rows, r1 = min(r0 + p.item_rows, (unsigned)(s.n * p.G));
  return make_int2(p0 + (int)(r0 / (unsigned)p.G), p0 + (int)((r1 - 1) / (unsigned)p.G));
}

// First key (a multiple of the tile) and key tiles of item t.
template <bool TOKENS, bool TREE>
__device__ __forceinline__ int2 item_keys(const Split<TOKENS, TREE>& p, const Seq<TREE>& s, int t) {
  const int2 span = item_span(p, s, t);
  if (span.y < 0) return make_int2(0, 0);
  int k0 = 0;
  int least = span.x;  // the lowest position of a row
  if constexpr (TREE) least = s.ctx;
  if (p.window > 0 && least >= p.window) k0 = (least - p.window + 1) >> p.tile_shift << p.tile_shift;
  return make_int2(k0, ((span.y - k0) >> p.tile_shift) + 1);
}

// Cost units of a key tile of item t, and of the whole item.
template <bool TOKENS, bool TREE>
__device__ __forceinline__ int tile_units(const Split<TOKENS, TREE>& p, const Seq<TREE>& s, int t) {
  return s.n * p.G - t * p.item_rows > p.half_rows ? p.tile_cost : p.half_cost;
}
template <bool TOKENS, bool TREE>
__device__ __forceinline__ int item_units(const Split<TOKENS, TREE>& p, const Seq<TREE>& s, int t) {
  return p.item_cost + tile_units(p, s, t) * item_keys(p, s, t).y;
}

// a / b for a >= 0, b > 0.
static __device__ __noinline__ long long divide64(long long a, int b) { return a / b; }
__device__ __forceinline__ long long divide(long long a, int b) {
  return a >> 32 == 0 ? (long long)((unsigned)a / (unsigned)b) : divide64(a, b);
}

// The cost line's shares: CTA c has [from(c), from(c + 1)), none but the first ctas. A share is large
// enough for a key tile, so that every CTA inside a cut item has at least one.
struct Shares {
  long long each;   // units of a share; the first `more` have one more
  int more, ctas;
  template <bool TOKENS, bool TREE>
  __device__ __forceinline__ void init(const Split<TOKENS, TREE>& p, long long total, int tiles = 1) {
    const int least = tiles * max(p.tile_cost, p.half_cost);
    ctas = (int)gridDim.x;
    if (total < (long long)ctas * least) ctas = max(1, (int)total / least);
    each = divide(total, ctas);
    more = (int)(total - each * ctas);
  }
  __device__ __forceinline__ long long from(int c) const { return c < ctas ? c * each + min(c, more) : ctas * each + more; }
};

// A CTA's share and where it starts.
template <bool TREE>
struct Start {
  long long begin, end;  // on the cost line
  Shares shares;
  int b, kvh, t;         // the item that holds `begin`
  int off;               // cost units of it before `begin`
  Seq<TREE> s;           // its sequence
};

// Shared scratch of locate: every sequence and its cost.
template <bool TREE>
constexpr size_t kLocateBytes = sizeof(Seq<TREE>) + sizeof(long long);  // per sequence

// The KV head and the item of a sequence that hold cost unit `rest` of it; per_head: of one of its heads. By a
// whole warp.
template <bool TOKENS, bool TREE>
__device__ __noinline__ void locate_item(const Split<TOKENS, TREE>& p, const Seq<TREE>& s, long long rest,
                                         long long per_head, Start<TREE>* st) {
  const int lane = threadIdx.x & 31;
  int kvh = 0;
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

// locate for at most 32 sequences by one warp, in registers: 32, 16, .. lanes share a sequence. All of this comes
// before the first load, and is run once: an instruction costs about 40 cycles then, as none is in the cache, so
// what counts is how few there are, and that parameters are operands, not loads (16 rows behind 1023 of one
// sequence: 15.8 us with locate, 13.7; 32 blocks of 16 rows 69.4 and 66.8; one token in f32 19.2 and 16.8).
template <bool TOKENS, bool TREE>
__device__ __forceinline__ void locate_by_warp(const Split<TOKENS, TREE>& p, Start<TREE>* st, unsigned* status) {
  const int lane = threadIdx.x & 31;
  const int shift = __clz(p.batch - 1) - 27;  // log2 of a sequence's lanes (one sequence: 32 - 27)
  const int b = lane >> shift, lanes = 1 << shift;
  Seq<TREE> s = {};
  unsigned bad = 0;
  int items = 0;
  if (b < p.batch) {
    s = load_seq(p, b, &bad);
    items = n_items(p, s);
  }
  if (bad && blockIdx.x == 0) atomicOr(status, bad);
  long long sum = 0;
#pragma unroll 1
  for (int t = lane & (lanes - 1); t < items; t += lanes) sum += item_units(p, s, t);
#pragma unroll 1
  for (int o = lanes >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const long long cost = sum * p.n_kv;
  long long upto = (lane & (lanes - 1)) == 0 ? cost : 0;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += u;
  }
  const long long total = __shfl_sync(0xffffffffu, upto, 31);
  // Fewer heads than eight: an item may be cut into as many pieces as there are CTAs, which the merge adds up one
  // after another (0.33 us each, a tile of a share about 1.1): shares of s tiles, T / s pieces of an item that costs
  // as much as T tiles, are the quickest around s = sqrt(0.3 T), here sqrt(T / 4). (A tile as dear as those of two
  // row tiles; an item of few rows has two keys' tiles in one.) 16 rows behind 128 n - 17 of one KV head, bf16, us:
  //   8 query heads, T = n / 2:  n = 64   s 1: 25.5  2: 18.8  4: 19.0  8: 21.2             the rule (2) 19.5
  //                              n = 256  s 1: 56.4  2: 43.1  4: 29.0  6: 25.3  8: 26.0    the rule (5) 25.6
  //                              n = 1024 s 4: 59.2  8: 50.5  12: 44.8  16: 43.4           the rule (11) 44.6
  //   16 query heads, T = n:     n = 256  s 1: 59.2  4: 35.9  6: 32.7  8: 32.3  12: 35.0   the rule (8) 32.4
  // Over 1, 2 and 4 heads or sequences, both caches and n = 8 to 1024 the rule is within 5 % of the best s in 146 of
  // 160 cases, and 11 % behind it at most. (f32, whose items are cut by rows, keeps shares of a tile and more.)
  int tiles = 1;
  if (TOKENS && p.batch * p.n_kv < 8) {
    const int item = __reduce_max_sync(0xffffffffu, items > 0 ? (int)__fdividef((float)sum, (float)items) : 1);
    tiles = max(1, (int)__fdividef(1.f, rsqrtf((float)(item / (4 * p.tile_cost)))));  // (0: 1 / infinity)
  }
  Shares shares;
  shares.init(p, total, tiles);
  const long long begin = shares.from(blockIdx.x), end = shares.from(blockIdx.x + 1);
  int l = 0;
  if (begin < end) {  // the first sequence whose prefix exceeds begin
    l = __ffs(__ballot_sync(0xffffffffu, upto > begin)) - 1;
    long long rest = begin - (upto - cost);
    if (__any_sync(0xffffffffu, lane == l && items > 1)) {
      s.row0 = __shfl_sync(0xffffffffu, s.row0, l);
      s.n = __shfl_sync(0xffffffffu, s.n, l);
      s.kv = __shfl_sync(0xffffffffu, s.kv, l);
      if constexpr (TREE) s.ctx = __shfl_sync(0xffffffffu, s.ctx, l);
      locate_item(p, s, __shfl_sync(0xffffffffu, rest, l), __shfl_sync(0xffffffffu, sum, l), st);
    } else if (lane == l) {  // one item a head
      int kvh = 0;
      for (; rest >= sum; rest -= sum) ++kvh;
      st->kvh = kvh;
      st->t = 0;
      st->off = (int)rest;
      st->s = s;
    }
  }
  if (lane == 0) {
    st->begin = begin;
    st->end = end;
    st->shares = shares;
    st->b = l >> shift;
  }
  __syncwarp();
}

// Run by all threads of the CTA; `scratch` is 16-byte aligned shared memory of kLocateBytes per
// sequence (free again after the call and a __syncthreads), `st` shared. A thread per sequence
// reads the lengths; then eight lanes per sequence add up its items.
template <bool TOKENS, bool TREE>
__device__ __noinline__ void locate(const Split<TOKENS, TREE>& p, void* scratch, Start<TREE>* st, unsigned* status) {
  long long* cost = reinterpret_cast<long long*>(scratch);
  Seq<TREE>* seq = reinterpret_cast<Seq<TREE>*>(cost + p.batch);
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
      const Seq<TREE> s = seq[b];
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
    Shares shares;
    shares.init(p, carry);
    const long long begin = shares.from(blockIdx.x), end = shares.from(blockIdx.x + 1);
    int b = 0;
    if (begin < end) {  // the first sequence whose prefix exceeds begin
      int lo = 0, hi = p.batch - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cost[mid] > begin) hi = mid; else lo = mid + 1;
      }
      b = lo;
      const Seq<TREE> s = seq[b];
      const long long before = b > 0 ? cost[b - 1] : 0;
      locate_item(p, s, begin - before, divide(cost[b] - before, p.n_kv), st);
    }
    if (lane == 0) {
      st->begin = begin;
      st->end = end;
      st->shares = shares;
      st->b = b;
    }
  }
  __syncthreads();
}

// One piece of work: key tiles [tile0, tile1) of item t of (b, kvh).
struct PieceOf {
  int b, kvh, t;
  int row0, n, kv;   // of the sequence
  int k0;            // first key of the item
  int tile0, tile1;
  int slot;          // -1: the whole item; else partial slot 0 or 1 of this CTA
};
template <bool TREE>
struct Piece : PieceOf {};
template <>
struct Piece<true> : PieceOf {
  int ctx;
};

// Walks a CTA's share piece by piece (one thread, or all threads of a warp alike).
template <bool TOKENS, bool TREE>
struct Walker {
  const Split<TOKENS, TREE>& p;
  Seq<TREE> s;
  long long at, end;
  Shares shares;
  int b, kvh, t, off;
  int4 merge;  // what to merge: {b, kvh, t, pieces}, pieces 0 when nothing was cut here

  __device__ __forceinline__ Walker(const Split<TOKENS, TREE>& split, const Start<TREE>& st) : p(split) {
    at = st.begin;
    end = st.end;
    shares = st.shares;
    b = st.b;
    kvh = st.kvh;
    t = st.t;
    off = st.off;
    merge = make_int4(0, 0, 0, 0);
    s = st.s;
  }

  __device__ __forceinline__ bool next(Piece<TREE>* w) {
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
      if constexpr (TREE) w->ctx = s.ctx;
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
        while (shares.from(c) < item_end) {
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

// Which of the keys k .. k + 127 the node `node` (none: -1) of sequence b's tree sees, as bits of four
// words. Committed keys by the window alone; keys of the tree by the node's mask, up to its own, and
// by the window: a node's position is the committed rows plus its depth. (A window as deep as
// the node cuts nothing from its tree, so depths are compared where it is not.) One call for a tile, so
// that the five words a tile can straddle are loaded at once; not inlined, as the kernels have little
// room for code.
static __device__ __noinline__ uint4 tree_bits(const TreeRows& t, int b, int node, int ctx, int k, int window) {
  uint32_t m[4] = {0, 0, 0, 0};
  if (node >= 0) {
    const size_t row = (size_t)b * t.max_nodes;
    const int u0 = k - ctx, i0 = u0 >> 5;  // node of bit 0; the word it is in (below 0: committed keys)
    const uint32_t* mask = t.masks + (row + node) * (t.max_nodes >> 5);
    const int depth = window > 0 ? t.depths[row + node] : 0;
    uint32_t w[5];
#pragma unroll
    for (int c = 0; c < 5; ++c) w[c] = i0 + c >= 0 && 32 * (i0 + c) <= node ? mask[i0 + c] : 0u;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int last = node - u0 - 32 * c;  // bit of the own node
      m[c] = __funnelshift_r(w[c], w[c + 1], u0 & 31) & (last < 0 ? 0u : last >= 31 ? 0xffffffffu : (2u << last) - 1u);
    }
    if (window > 0 && depth >= window) {
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t bits = c == 0 ? m[0] : c == 1 ? m[1] : c == 2 ? m[2] : m[3], keep = bits;
#pragma unroll 1
        for (; bits; bits &= bits - 1) {
          const int e = __ffs(bits) - 1;
          if (depth - t.depths[row + u0 + 32 * c + e] >= window) keep &= ~(1u << e);
        }
        (c == 0 ? m[0] : c == 1 ? m[1] : c == 2 ? m[2] : m[3]) = keep;
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int n = -u0 - 32 * c;                                                 // committed keys
      const int l0 = window > 0 ? ctx + depth - window + 1 - k - 32 * c : 0;      // the first the window leaves
      m[c] |= (n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u) & (l0 <= 0 ? 0xffffffffu : l0 > 31 ? 0u : 0xffffffffu << l0);
    }
  }
  return make_uint4(m[0], m[1], m[2], m[3]);
}

}  // namespace chunk
}  // namespace dflash
