// k_attn_beside.cu -- the sequences' own part behind a shared prefix, its shares left for
// a join: the kernels of k_attn_rows.cuh and k_attn_chunk.cuh in that mode.
#include "k_attn_chunk.cuh"
#include "k_attn_rows.cuh"

namespace cbs {
cbs_status launch_attn_beside(const AttnLaunch &L, int row_tile, cudaStream_t s) {
    if (row_tile == kAttnChunkRows) return launch_attn_chunk_as<kAttnBeside>(L, s);
    return cuda_check(launch_attn_rows_as<kAttnBeside>(L, row_tile, s), "attention launch");
}
}  // namespace cbs
