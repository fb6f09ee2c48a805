// Causal chunk attention on tcgen05 tensor cores.
#include "chunk_attn_tc.cuh"

namespace dflash {

int chunk_attn_tc_item_rows(int G) { return 2 * (128 / G) * G; }

cudaError_t chunk_attn_tc(const ChunkAttnParams& p, cudaStream_t s) { return attn_tc<false>(p, s); }

}  // namespace dflash
