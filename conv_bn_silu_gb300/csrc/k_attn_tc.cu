// k_attn_tc.cu -- attention of chunks over a paged cache (k_attn_chunk.cuh).
#include "k_attn_chunk.cuh"

namespace cbs {
cbs_status launch_attn_chunk(const AttnLaunch &L, cudaStream_t s) { return launch_attn_chunk_as<kAttnPlain>(L, s); }
}  // namespace cbs
