// Entry points of the tree and beam calls: argument checks and launches.
#include <math.h>
#include <string.h>

#include "tree.cuh"

using namespace dflash;

namespace {

bool aligned4(const void* p) { return p && ((uintptr_t)p & 3) == 0; }

dflash_status check_tree(const dflash_tree* t, int batch, bool masks) {
  if (!t || !aligned4(t->nodes) || t->batch != batch || t->max_nodes <= 0 || t->max_nodes % 32)
    return DFLASH_ERR_INVALID_ARG;
  if (masks && (!aligned4(t->depths) || !aligned4(t->masks))) return DFLASH_ERR_INVALID_ARG;
  if (t->max_nodes > kTreeMaxNodes || batch > kTreeMaxBatch) return DFLASH_ERR_UNSUPPORTED;
  return DFLASH_OK;
}

dflash_status check_rows(const dflash_chunk* ch) {
  if (!ch || !aligned4(ch->cu_rows) || !aligned4(ch->kv_lens) || ch->batch <= 0 || ch->rows < 0)
    return DFLASH_ERR_INVALID_ARG;
  return DFLASH_OK;
}

}  // namespace

DFLASH_API dflash_status dflash_tree_map(const dflash_chunk* ch, const dflash_tree* tree, const int32_t* parents,
                                         const int32_t* nodes_before, cudaStream_t stream) {
  dflash_status st = check_rows(ch);
  if (st != DFLASH_OK) return st;
  st = check_tree(tree, ch->batch, true);
  if (st != DFLASH_OK) return st;
  if (nodes_before && !aligned4(nodes_before)) return DFLASH_ERR_INVALID_ARG;
  if (ch->rows > 0 && (!aligned4(ch->slots) || !aligned4(ch->positions) || !aligned4(parents)))
    return DFLASH_ERR_INVALID_ARG;
  TreeMapParams p;
  memset(&p, 0, sizeof(p));
  p.status = status_word();
  if (!p.status) return DFLASH_ERR_CUDA;
  p.cu_rows = ch->cu_rows;
  p.kv_lens = ch->kv_lens;
  p.slots = ch->slots;
  p.positions = ch->positions;
  p.parents = parents;
  p.nodes_before = nodes_before;
  p.nodes = tree->nodes;
  p.depths = tree->depths;
  p.masks = tree->masks;
  p.batch = ch->batch;
  p.rows = ch->rows;
  p.max_nodes = tree->max_nodes;
  return cuda_status(tree_map(p, stream));
}

DFLASH_API dflash_status dflash_tree_accept(const dflash_chunk* ch, const int32_t* parents, const int32_t* tokens,
                                            const int32_t* posterior, const int32_t* ctx_len, int max_path,
                                            int32_t* path, int32_t* accept_len, int32_t* next_cu_rows,
                                            int32_t* ctx_next, int32_t* next_anchor, cudaStream_t stream) {
  dflash_status st = check_rows(ch);
  if (st != DFLASH_OK) return st;
  if (max_path <= 0 || !aligned4(ctx_len) || !aligned4(path) || !aligned4(accept_len) ||
      !aligned4(next_cu_rows) || !aligned4(ctx_next) || !aligned4(next_anchor))
    return DFLASH_ERR_INVALID_ARG;
  if (ch->rows > 0 && (!aligned4(parents) || !aligned4(tokens) || !aligned4(posterior)))
    return DFLASH_ERR_INVALID_ARG;
  if (ch->batch > kChunkMaxBatch) return DFLASH_ERR_UNSUPPORTED;
  TreeAcceptParams p;
  memset(&p, 0, sizeof(p));
  p.status = status_word();
  if (!p.status) return DFLASH_ERR_CUDA;
  p.cu_rows = ch->cu_rows;
  p.kv_lens = ch->kv_lens;
  p.parents = parents;
  p.tokens = tokens;
  p.posterior = posterior;
  p.ctx_len = ctx_len;
  p.accept_len = accept_len;
  p.path = path;
  p.next_cu_rows = next_cu_rows;
  p.ctx_next = ctx_next;
  p.next_anchor = next_anchor;
  p.batch = ch->batch;
  p.rows = ch->rows;
  p.max_path = max_path;
  return cuda_status(tree_accept(p, stream));
}

DFLASH_API dflash_status dflash_tree_commit(const dflash_dims* d, const dflash_kv_cache* c, const dflash_tree* tree,
                                            const int32_t* ctx_len, const int32_t* path, int max_path,
                                            const int32_t* accept_len, cudaStream_t stream) {
  dflash_status st = check_dims(d);
  if (st != DFLASH_OK) return st;
  st = check_cache(c, 0);
  if (st != DFLASH_OK) return st;
  st = check_layout(d, c);
  if (st != DFLASH_OK) return st;
  st = check_tree(tree, c->batch, false);
  if (st != DFLASH_OK) return st;
  if (max_path <= 0 || !aligned4(ctx_len) || !aligned4(path) || !aligned4(accept_len)) return DFLASH_ERR_INVALID_ARG;
  if (c->n_layers > 32767) return DFLASH_ERR_UNSUPPORTED;  // (two grid rows a layer)
  // the lengths are written while other CTAs read these
  const size_t n = (size_t)c->batch;
  auto in_lens = [&](const int32_t* a, size_t m) {
    const uintptr_t lo = (uintptr_t)a, from = (uintptr_t)c->lens;
    return lo < from + 4 * n * c->n_layers && from < lo + 4 * m;
  };
  if (in_lens(ctx_len, n) || in_lens(accept_len, n) || in_lens(tree->nodes, n) || in_lens(path, n * max_path))
    return DFLASH_ERR_INVALID_ARG;
  TreeCommitParams p;
  memset(&p, 0, sizeof(p));
  p.status = status_word();
  if (!p.status) return DFLASH_ERR_CUDA;
  p.cache_k = (char*)c->k;
  p.cache_v = (char*)c->v;
  p.block_table = c->block_table;
  p.lens = c->lens;
  p.ctx_len = ctx_len;
  p.nodes = tree->nodes;
  p.path = path;
  p.accept_len = accept_len;
  p.unit_rows = c->block_table ? c->page_size : c->capacity;
  p.n_kv = d->n_kv;
  p.row_bytes = d->d_h * (int)kv_esize(d, c);
  const size_t units = c->block_table ? (size_t)c->n_pages : (size_t)c->batch;
  p.layer_bytes = units * p.unit_rows * d->n_kv * p.row_bytes;
  p.n_layers = c->n_layers;
  p.batch = c->batch;
  p.capacity = c->capacity;
  p.pages_per_seq = c->block_table ? c->capacity / c->page_size : 0;
  p.n_pages = c->block_table ? c->n_pages : 0;
  p.max_path = max_path;
  p.max_nodes = tree->max_nodes;
  return cuda_status(tree_commit(p, stream));
}

namespace {

dflash_status check_beams(int batch, int beams, int vocab, int k) {
  if (batch <= 0 || beams <= 0 || vocab <= 0 || k <= 0) return DFLASH_ERR_INVALID_ARG;
  if ((long long)beams * vocab < k) return DFLASH_ERR_INVALID_ARG;
  if (beams > kBeamMax || k > kBeamMax || (long long)beams * vocab > 0x7fffffffll || vocab > (1 << 28) ||
      (long long)batch * beams > (1 << 20))
    return DFLASH_ERR_UNSUPPORTED;
  return DFLASH_OK;
}

}  // namespace

DFLASH_API size_t dflash_beam_workspace_bytes(int batch, int beams, int vocab, int k) {
  return check_beams(batch, beams, vocab, k) == DFLASH_OK ? beam_workspace(batch, beams, vocab, k) : 0;
}

DFLASH_API dflash_status dflash_beam_select(int dtype, const void* logits, long long ld_seq, long long ld_beam,
                                            const float* scores, int batch, int beams, int vocab, int k,
                                            int parent_base, int32_t* tokens, int32_t* parents, float* scores_out,
                                            long long ld_out, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  if (dtype != DFLASH_F32 && dtype != DFLASH_BF16) return DFLASH_ERR_UNSUPPORTED;
  dflash_status st = check_beams(batch, beams, vocab, k);
  if (st != DFLASH_OK) return st;
  const size_t es = dtype == DFLASH_F32 ? 4 : 2;
  if (!logits || ((uintptr_t)logits & (es - 1)) || ld_seq < 0 || ld_beam < 0 || ld_out < k) return DFLASH_ERR_INVALID_ARG;
  if (parent_base < 0 || parent_base > 0x7fffffff - beams) return DFLASH_ERR_INVALID_ARG;
  if (!aligned4(tokens) || (parents && !aligned4(parents)) || (scores_out && !aligned4(scores_out)) ||
      (scores && !aligned4(scores)) || !workspace || ((uintptr_t)workspace & 255))
    return DFLASH_ERR_INVALID_ARG;
  BeamParams p;
  memset(&p, 0, sizeof(p));
  p.logits = logits;
  p.ld_seq = ld_seq;
  p.ld_beam = ld_beam;
  p.scores = scores;
  p.tokens = tokens;
  p.parents = parents;
  p.scores_out = scores_out;
  p.ld_out = ld_out;
  p.workspace = workspace;
  p.batch = batch;
  p.beams = beams;
  p.vocab = vocab;
  p.k = k;
  p.parent_base = parent_base;
  return beam_select(dtype, p, ws_bytes, stream);
}
