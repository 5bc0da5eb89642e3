// k_attn.cu -- attention of few rows over a paged cache (k_attn_rows.cuh).
#include "k_attn_rows.cuh"

namespace cbs {
cudaError_t launch_attn_rows(const AttnLaunch &L, int row_tile, cudaStream_t s) { return launch_attn_rows_as<kAttnPlain>(L, row_tile, s); }
}  // namespace cbs
