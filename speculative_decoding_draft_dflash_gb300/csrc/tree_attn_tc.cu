// Attention of drafted trees and beams on tcgen05 tensor cores: the causal kernel with TREE set.
//
//   out_t = sum_j p_tj v_j / sum_j p_tj over the committed keys j < c and the keys c + u of the nodes u that
// the mask of node t has. Nothing else differs: rows lie in the cache in the order of the nodes, so a node sees no
// key behind its own, items, shares and costs are those of causal rows, and only tiles that reach beyond the
// first c keys (or that a window cuts) look at masks. There a thread, which has one row, takes the 128 bits
// of its tile in one look-up (chunk::tree_bits) while the tensor cores work on the scores; a bit is then the
// same select as the causal mask's. Inlined, or word by word after the scores, the look-up cost 8 us of 83.
//
// Bound by HBM and, in items of few tiles, by the start (4 us until the first tile is on its way), an
// item's end and the merge. In a replayed graph, and the causal kernel on the same rows: 32 trees of 64 nodes
// behind 256 to 4096 rows of 8 heads 82.2 us (causal 79.1; 326.9 MB read of 328.8 with what stays in L2), 16
// sequences of 9 to 16 beams behind 1024 to 8192 rows and 100 to 500 nodes, E4M3, window 4096 53.4 (46.0: a
// window reaches further back for a node than for the row at its place), 16 nodes behind 1023 rows 13.8 (13.3).
#include "chunk_attn_tc.cuh"

namespace dflash {

cudaError_t tree_attn_tc(const ChunkAttnParams& p, cudaStream_t s) { return attn_tc<true>(p, s); }

}  // namespace dflash
