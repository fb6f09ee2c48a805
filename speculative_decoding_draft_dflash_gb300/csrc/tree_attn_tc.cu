// Attention of drafted trees and beams on tcgen05 tensor cores.
#include "chunk_attn_tc.cuh"

namespace dflash {

cudaError_t tree_attn_tc(const ChunkAttnParams& p, cudaStream_t s) { return attn_tc<true>(p, s); }

}  // namespace dflash
