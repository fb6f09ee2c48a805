// Trees of drafted tokens and beams next to the chunk step: parameters of their kernels.
#pragma once

#include "chunk.cuh"

namespace dflash {

struct TreeMapParams {
  const int32_t* cu_rows;
  int32_t* kv_lens;
  int32_t* slots;
  int32_t* positions;
  const int32_t* parents;       // [rows], node of each row's parent
  const int32_t* nodes_before;  // [batch], or null: no tree had a node
  int32_t* nodes;
  int32_t* depths;
  uint32_t* masks;
  unsigned* status;
  int batch, rows, max_nodes;
};
cudaError_t tree_map(const TreeMapParams& p, cudaStream_t s);

struct TreeAcceptParams {
  const int32_t* cu_rows;
  const int32_t* kv_lens;
  const int32_t* parents;
  const int32_t* tokens;
  const int32_t* posterior;
  const int32_t* ctx_len;
  int32_t* accept_len;
  int32_t* path;                // [batch][max_path]
  int32_t* next_cu_rows;
  int32_t* ctx_next;
  int32_t* next_anchor;
  unsigned* status;
  int batch, rows, max_path;
};
cudaError_t tree_accept(const TreeAcceptParams& p, cudaStream_t s);

struct TreeCommitParams {
  char* cache_k;                // layer 0: units of [n_kv][unit_rows][row_bytes] (a page, or a sequence)
  char* cache_v;
  const int32_t* block_table;   // paged, or null
  int32_t* lens;                // [n_layers][batch]
  const int32_t* ctx_len;
  const int32_t* nodes;
  const int32_t* path;
  const int32_t* accept_len;
  unsigned* status;
  size_t layer_bytes;
  int n_layers, batch, capacity, pages_per_seq, n_pages, unit_rows, n_kv, row_bytes, max_path, max_nodes;
};
cudaError_t tree_commit(const TreeCommitParams& p, cudaStream_t s);

constexpr int kBeamMax = 128;  // beams of a sequence, and kept candidates

struct BeamParams {
  const void* logits;           // row of (sequence, beam) at seq * ld_seq + beam * ld_beam elements
  long long ld_seq, ld_beam;
  const float* scores;          // [batch][beams], or null: 0
  int32_t* tokens;              // [batch] rows of k, ld_out elements apart
  int32_t* parents;             // or null
  float* scores_out;            // or null
  long long ld_out;
  void* workspace;
  int batch, beams, vocab, k, parent_base;
};
size_t beam_workspace(int batch, int beams, int vocab, int k);
dflash_status beam_select(int dtype, const BeamParams& p, size_t ws_bytes, cudaStream_t s);  // or DFLASH_ERR_WORKSPACE

}  // namespace dflash
