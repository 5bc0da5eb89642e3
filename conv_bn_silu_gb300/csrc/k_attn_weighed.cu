// k_attn_weighed.cu -- attention that leaves scores and sums for the keys' weights: the kernels of
// k_attn_rows.cuh and k_attn_chunk.cuh in that mode.
#include "k_attn_chunk.cuh"
#include "k_attn_rows.cuh"

namespace cbs {
cbs_status launch_attn_weighed(const AttnLaunch &L, int row_tile, cudaStream_t s) {
    if (row_tile == kAttnChunkRows) return launch_attn_chunk_as<kAttnWeighed>(L, s);
    return cuda_check(launch_attn_rows_as<kAttnWeighed>(L, row_tile, s), "attention launch");
}
}  // namespace cbs
