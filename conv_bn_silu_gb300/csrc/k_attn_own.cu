// k_attn_own.cu -- the sequences' own part behind a shared prefix: the kernels of
// k_attn_rows.cuh and k_attn_chunk.cuh in that mode, and the join of both parts where
// the own part does not wait for the prefix's.
#include "k_attn_chunk.cuh"
#include "k_attn_rows.cuh"

namespace cbs {
cbs_status launch_attn_own(const AttnLaunch &L, int row_tile, cudaStream_t s) {
    if (row_tile == kAttnChunkRows) return launch_attn_chunk_as<kAttnOwn>(L, s);
    return cuda_check(launch_attn_rows_as<kAttnOwn>(L, row_tile, s), "attention launch");
}

namespace {

// A prefix's and the sequences' own shares of every row, joined.  A thread eight
// dimensions; tokens behind the last sequence's are left as they are.
template <int D>
__global__ void __launch_bounds__(256) join_shares_kernel(const AttnLaunch L, const float *pre, const float2 *pre_stats) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    constexpr int kU = D / 8;
    const int tokens = max(0, min(L.c.new_start[L.c.batch], L.c.total));
    const long long all = (long long)tokens * L.heads * kU;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < all; i += (long long)gridDim.x * 256) {
        const long long row = i / kU;
        const int u = (int)(i - row * kU), token = (int)(row / L.heads), head = (int)(row - (long long)token * L.heads);
        const float2 p = pre_stats[row], o = L.share_stats[row];
        uint32_t w[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const size_t at = (size_t)row * D + u * 8 + h * 4;
            float4 acc = *reinterpret_cast<const float4 *>(L.share + at);
            float sum;
            const bool any = join_shares(p, *reinterpret_cast<const float4 *>(pre + at), o, acc, sum);
            const float inv = __fdiv_rn(1.0f, sum);
            w[2 * h] = any ? frag::pack_bf16(acc.x * inv, acc.y * inv) : 0u;
            w[2 * h + 1] = any ? frag::pack_bf16(acc.z * inv, acc.w * inv) : 0u;
        }
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(L.out) + (size_t)token * L.out_stride + (size_t)head * D + u * 8) =
            make_uint4(w[0], w[1], w[2], w[3]);
    }
}

}  // namespace

cudaError_t launch_join_shares(const AttnLaunch &L, const float *pre, const float2 *pre_stats, cudaStream_t s) {
    const long long units = ((long long)L.c.total * L.heads * L.c.head_dim / 8 + 255) / 256, most = current_device_sms() * 8ll;
    const int grid = (int)(units < most ? units : most);
    if (L.c.head_dim == 64) return launch_kernel(join_shares_kernel<64>, grid, 256, 0, s, L, pre, pre_stats);
    return launch_kernel(join_shares_kernel<128>, grid, 256, 0, s, L, pre, pre_stats);
}
}  // namespace cbs
