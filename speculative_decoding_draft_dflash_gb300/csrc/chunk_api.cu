// Entry points of the chunk step: argument checks and launches.
#include <math.h>
#include <string.h>

#include "chunk.cuh"

using namespace dflash;

namespace {

bool aligned4(const void* p) { return ((uintptr_t)p & 3) == 0; }

// What every call asks of the step: `slots` and `positions` where the call uses them.
dflash_status check_chunk(const dflash_kv_cache* c, const dflash_chunk* ch, bool rows_arrays) {
  if (!ch || !ch->cu_rows || !ch->kv_lens || !aligned4(ch->cu_rows) || !aligned4(ch->kv_lens))
    return DFLASH_ERR_INVALID_ARG;
  if (ch->batch != c->batch || ch->rows < 0) return DFLASH_ERR_INVALID_ARG;
  if (rows_arrays && ch->rows > 0 &&
      (!ch->slots || !ch->positions || !aligned4(ch->slots) || !aligned4(ch->positions)))
    return DFLASH_ERR_INVALID_ARG;
  if (ch->batch > kChunkMaxBatch) return DFLASH_ERR_UNSUPPORTED;
  return DFLASH_OK;
}

long long cache_slots(const dflash_kv_cache* c) {
  return c->block_table ? (long long)c->n_pages * c->page_size : (long long)c->batch * c->capacity;
}

// Rows of `width` elements `ld` apart.
bool rows_ok(const dflash_dims* d, const void* p, long long ld, long long width) {
  if (!p || ld < width) return false;
  if (d->dtype == DFLASH_BF16) return aligned16(p) && ld % 8 == 0;
  return aligned4(p);
}

}  // namespace

DFLASH_API dflash_status dflash_chunk_map(const dflash_kv_cache* c, int layer,
                                          const dflash_chunk* ch, const dflash_page_pool* pool,
                                          cudaStream_t stream) {
  dflash_status st = check_cache(c, layer);
  if (st != DFLASH_OK) return st;
  st = check_chunk(c, ch, true);
  if (st != DFLASH_OK) return st;
  if (cache_slots(c) > 0x7fffffffll) return DFLASH_ERR_UNSUPPORTED;
  ChunkMapParams p;
  memset(&p, 0, sizeof(p));
  if (c->block_table) {
    if (!pool || pool->block_table != c->block_table || pool->n_free < 0 || !pool->pages_held ||
        !pool->pages_held_out || !pool->taken || !pool->taken_out ||
        (pool->n_free > 0 && !pool->free_pages))
      return DFLASH_ERR_INVALID_ARG;
    const void* ptrs[] = {pool->pages_held, pool->pages_held_out, pool->taken, pool->taken_out,
                          pool->free_pages};
    for (const void* q : ptrs)
      if (!aligned4(q)) return DFLASH_ERR_INVALID_ARG;
    p.paged = true;
    p.table = pool->block_table;
    p.held = pool->pages_held;
    p.held_out = pool->pages_held_out;
    p.free_pages = pool->free_pages;
    p.n_free = pool->n_free;
    p.taken = pool->taken;
    p.taken_out = pool->taken_out;
    p.pages_per_seq = c->capacity / c->page_size;
    p.n_pages = c->n_pages;
    p.alias = pool->pages_held_out == pool->pages_held || pool->taken_out == pool->taken;
  }
  if (ch->kv_lens == c->lens + (size_t)layer * c->batch) return DFLASH_ERR_INVALID_ARG;
  p.status = status_word();
  if (!p.status) return DFLASH_ERR_CUDA;
  p.cu_rows = ch->cu_rows;
  p.lens = c->lens + (size_t)layer * c->batch;
  p.kv_lens = ch->kv_lens;
  p.slots = ch->slots;
  p.positions = ch->positions;
  p.batch = ch->batch;
  p.rows = ch->rows;
  p.capacity = c->capacity;
  return cuda_status(chunk_map(p, stream));
}

DFLASH_API dflash_status dflash_chunk_append(const dflash_dims* d, const dflash_kv_cache* c,
                                             int layer, const dflash_chunk* ch, const void* q,
                                             long long ld_q, const void* k, long long ld_k,
                                             const void* v, long long ld_v, const void* gamma_q,
                                             const void* gamma_k, const float* rope_table,
                                             int table_len, void* q_out, cudaStream_t stream) {
  dflash_status st = check_dims(d);
  if (st != DFLASH_OK) return st;
  st = check_cache(c, layer);
  if (st != DFLASH_OK) return st;
  st = check_layout(d, c);
  if (st != DFLASH_OK) return st;
  st = check_chunk(c, ch, true);
  if (st != DFLASH_OK) return st;
  if (cache_slots(c) > 0x7fffffffll) return DFLASH_ERR_UNSUPPORTED;
  const size_t ra = d->dtype == DFLASH_BF16 ? 15 : 7;
  if (table_len < 0 || (rope_table ? ((uintptr_t)rope_table & ra) != 0 : table_len != 0))
    return DFLASH_ERR_INVALID_ARG;
  if (ch->rows == 0) return DFLASH_OK;
  const long long qw = (long long)d->n_h * d->d_h, kw = (long long)d->n_kv * d->d_h;
  if (!rows_ok(d, k, ld_k, kw) || !rows_ok(d, v, ld_v, kw)) return DFLASH_ERR_INVALID_ARG;
  if ((q != nullptr) != (q_out != nullptr)) return DFLASH_ERR_INVALID_ARG;
  if (q && (!rows_ok(d, q, ld_q, qw) || !rows_ok(d, q_out, qw, qw) || (q == q_out && ld_q != qw)))
    return DFLASH_ERR_INVALID_ARG;
  const size_t ga = d->dtype == DFLASH_BF16 ? 15 : 3;
  if (((uintptr_t)gamma_q & ga) || ((uintptr_t)gamma_k & ga)) return DFLASH_ERR_INVALID_ARG;
  ChunkAppendParams p;
  memset(&p, 0, sizeof(p));
  p.status = status_word();
  if (!p.status) return DFLASH_ERR_CUDA;
  p.slots = ch->slots;
  p.positions = ch->positions;
  p.kv_lens = ch->kv_lens;
  p.lens = c->lens + (size_t)layer * c->batch;
  p.q = q;
  p.k = k;
  p.v = v;
  p.ld_q = ld_q;
  p.ld_k = ld_k;
  p.ld_v = ld_v;
  p.gamma_q = gamma_q;
  p.gamma_k = gamma_k;
  p.rope = (const float2*)rope_table;
  p.q_out = q_out;
  p.unit_rows = c->block_table ? c->page_size : c->capacity;
  p.n_slots = cache_slots(c);
  const size_t layer_bytes = (size_t)p.n_slots * d->n_kv * d->d_h * kv_esize(d, c);
  p.cache_k = (char*)c->k + layer * layer_bytes;
  p.cache_v = (char*)c->v + layer * layer_bytes;
  p.batch = ch->batch;
  p.rows = ch->rows;
  p.capacity = c->capacity;
  p.n_h = d->n_h;
  p.n_kv = d->n_kv;
  p.d_h = d->d_h;
  p.table_len = table_len;
  p.eps = d->eps;
  p.fp8 = kv_fp8(c);
  p.k_inv = 1.f / kv_scale(c, layer, 0);
  p.v_inv = 1.f / kv_scale(c, layer, 1);
  return cuda_status(chunk_append(d->dtype, p, stream));
}

DFLASH_API size_t dflash_chunk_workspace_bytes(const dflash_dims* d) {
  if (check_dims(d) != DFLASH_OK) return 0;
  return chunk_attn_workspace(d->dtype, d->d_h);
}

DFLASH_API dflash_status dflash_chunk_attn(const dflash_dims* d, const dflash_kv_cache* c, int layer,
                                           const dflash_chunk* ch, const void* q, long long ld_q,
                                           int sliding_window, float scaling, void* out,
                                           void* workspace, size_t ws_bytes, cudaStream_t stream) {
  dflash_status st = check_dims(d);
  if (st != DFLASH_OK) return st;
  st = check_cache(c, layer);
  if (st != DFLASH_OK) return st;
  st = check_layout(d, c);
  if (st != DFLASH_OK) return st;
  st = check_chunk(c, ch, false);
  if (st != DFLASH_OK) return st;
  // key rows of one layer are addressed with 32-bit row numbers
  if (cache_slots(c) * d->n_kv > 0x7fffffffll || c->capacity > (1 << 28)) return DFLASH_ERR_UNSUPPORTED;
  if ((long long)ch->rows * (d->n_h / d->n_kv) > (1 << 30)) return DFLASH_ERR_UNSUPPORTED;
  if (sliding_window < 0 || !(scaling < INFINITY)) return DFLASH_ERR_INVALID_ARG;
  if (ch->rows == 0) return DFLASH_OK;
  const long long qw = (long long)d->n_h * d->d_h;
  if (!rows_ok(d, q, ld_q, qw) || !aligned16(q) || !out || !aligned16(out) || !workspace ||
      ((uintptr_t)workspace & 255))
    return DFLASH_ERR_INVALID_ARG;
  ChunkAttnParams p;
  memset(&p, 0, sizeof(p));
  if (!chunk_attn_carve(d->dtype, d->d_h, p, workspace, ws_bytes)) return DFLASH_ERR_WORKSPACE;
  p.status = status_word();
  if (!p.status) return DFLASH_ERR_CUDA;
  p.cu_rows = ch->cu_rows;
  p.kv_lens = ch->kv_lens;
  p.q = q;
  p.ld_q = ld_q;
  const size_t layer_bytes = (size_t)cache_slots(c) * d->n_kv * d->d_h * kv_esize(d, c);
  p.cache_k = (const char*)c->k + layer * layer_bytes;
  p.cache_v = (const char*)c->v + layer * layer_bytes;
  p.block_table = c->block_table;
  p.pages_per_seq = c->block_table ? c->capacity / c->page_size : 0;
  p.n_pages = c->block_table ? c->n_pages : 0;
  p.out = out;
  p.batch = ch->batch;
  p.rows = ch->rows;
  p.n_h = d->n_h;
  p.n_kv = d->n_kv;
  p.d_h = d->d_h;
  p.G = d->n_h / d->n_kv;
  p.capacity = c->capacity;
  // No two rows of a sequence are a capacity apart: a window that large is none, and one that is
  // smaller can be taken from any position without leaving 32 bits.
  p.window = sliding_window < c->capacity ? sliding_window : 0;
  p.scaling = scaling > 0.f ? scaling : 1.f / sqrtf((float)d->d_h);
  p.fp8 = kv_fp8(c);
  p.k_scale = kv_scale(c, layer, 0);
  p.v_scale = kv_scale(c, layer, 1);
  return cuda_status(chunk_attn(d->dtype, p, stream));
}
