// k_w8_few.cu -- products of 8-bit integers (the formula is in k_w8.cu) for a few input
// rows, where the weights' bytes bound the call and each is used once.
//
// Y^T = W X^T on m16n8k16: sixteen outputs of a warp fill the MMA's rows, the input rows
// its columns; a CTA's eight warps lie along k.  The contraction's order is free, so a
// lane's share of an output is sixteen consecutive codes, loaded at once; both sides
// widen exactly to f16.  No shared memory, barrier or hand-off before the end, where
// the warps' sums meet in order: whole numbers, exact below 2^24 in any order.
//
// Measured, one row: 6144 x 4096 6.6 us, 3.8 TB/s; 8192 x 8192 14.6 us, 4.6 TB/s; 60% of the
// issue slots.  (Of more than 96 MB of weights k_w8.cu takes over.)
#include <cuda_bf16.h>

#include "mma_frag.cuh"
#include "tc_ptx.cuh"
#include "tokens.cuh"
#include "w8.cuh"

namespace cbs {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps, kStep = 64;   // codes along k of a warp's step: sixteen a lane

__device__ __forceinline__ uint4 load_once(const int8_t *p) {   // weights: past L1, which the inputs use
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// NR: tiles of eight input rows.  kCtas: of an SM.  kAhead: steps on their way.  wk:
// warps side by side along k.
template <int NR, int kCtas, int kAhead>
__global__ void __launch_bounds__(kThreads, kCtas) w8_few_kernel(const W8Launch L, int wk) {
    __shared__ float s_sum[kWarps][NR * 8][17];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, j = lane & 3;
    const int part = warp % wk, n0 = (blockIdx.x * (kWarps / wk) + warp / wk) * 16, m0 = blockIdx.y * (NR * 8);
    const int steps = (L.k + kStep - 1) / kStep;
    const int s0 = (int)((long long)steps * part / wk), s1 = (int)((long long)steps * (part + 1) / wk);
    // Outputs g and g + 8 (past n: the last one again), input rows g and g + 8.
    const int8_t *wp[2], *xp[NR];
    bool on[NR];
#pragma unroll
    for (int i = 0; i < 2; ++i) wp[i] = L.w + (size_t)min(n0 + g + 8 * i, L.n - 1) * L.k + 16 * j;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        on[i] = m0 + g + 8 * i < L.rows;
        xp[i] = L.x + (size_t)min(m0 + g + 8 * i, L.rows - 1) * L.k + 16 * j;
    }
    struct Step { uint4 w[2], x[NR]; };
    const auto load = [&](int s) {
        Step t;
        const int at = s * kStep;
        const bool in = s < s1 && at + 16 * j < L.k;   // (k is a multiple of sixteen)
#pragma unroll
        for (int i = 0; i < 2; ++i) t.w[i] = in ? load_once(wp[i] + at) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < NR; ++i) t.x[i] = in && on[i] ? __ldg(reinterpret_cast<const uint4 *>(xp[i] + at)) : make_uint4(0, 0, 0, 0);
        return t;
    };
    float acc[NR][4] = {};
    Step ring[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) ring[i] = load(s0 + i);
    for (int sb = s0; sb < s1; sb += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {   // (past the share's end: zeros)
            const Step t = ring[i];
            ring[i] = load(sb + i + kAhead);
            const uint32_t a[4] = {t.w[0].x, t.w[0].y, t.w[0].z, t.w[0].w}, b[4] = {t.w[1].x, t.w[1].y, t.w[1].z, t.w[1].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t a0, a1, a2, a3;
                frag::i8_halves(a[q], a0, a2);
                frag::i8_halves(b[q], a1, a3);
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const uint32_t x[4] = {t.x[r].x, t.x[r].y, t.x[r].z, t.x[r].w};
                    uint32_t b0, b1;
                    frag::i8_halves(x[q], b0, b1);
                    frag::mma_half(acc[r], a0, a1, a2, a3, b0, b1);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) s_sum[warp][r * 8 + 2 * j + (i & 1)][g + 8 * (i >> 1)] = acc[r][i];
    __syncthreads();
    const int outs = kWarps / wk * 16;
    for (int i = tid; i < NR * 8 * outs; i += kThreads) {
        const int r = i / outs, o = i % outs, m = m0 + r, n = blockIdx.x * outs + o;
        if (m >= L.rows || n >= L.n) continue;
        float y = 0.0f;
        for (int w = o / 16 * wk; w < (o / 16 + 1) * wk; ++w) y += s_sum[w][r][o % 16];
        y = w8::Channel(L.w_scale[n], L.bias ? L.bias[n] : 0.0f)(y, L.x_scale[m]);
        if (L.act == CBS_ACT_SILU) y = silu(y);
        const size_t at = (size_t)m * L.n + n;
        if (L.out_bf16) static_cast<__nv_bfloat16 *>(L.y)[at] = __float2bfloat16_rn(y);
        else static_cast<float *>(L.y)[at] = y;
    }
}

}  // namespace

cudaError_t launch_w8_few(const W8Launch &L, cudaStream_t s) {
    // As many warps along k as leave each four steps, or until every SM has twelve.
    const int tiles = (L.n + 15) / 16, steps = (L.k + kStep - 1) / kStep;
    int wk = 1;
    while (wk < kWarps && (wk * 8 <= steps || tiles * wk < current_device_sms() * 12) && wk * 2 <= steps) wk *= 2;
    const int per = kWarps / wk, grid = (tiles + per - 1) / per;
    if (L.rows > 8) return launch_kernel(w8_few_kernel<2, 2, 3>, dim3(grid, (L.rows + 15) / 16), kThreads, 0, s, L, wk);
    // What is in flight is about as much with two CTAs an SM, four steps ahead, as with
    // three or four, two ahead; so as many as take the grid in one round, or four.  Two,
    // three and four, one row: 4096 x 4096 (256 CTAs) 5.1, 5.9, 6.2 us; 6144 x 4096 (384)
    // 8.4, 6.6, 8.2; 8192 x 8192 (512) 15.7, 19.1, 14.6; and, past what is sent here, 16384 x
    // 8192 (1024) 28.8, 30.0, 27.2.
    const int sms = current_device_sms();
    if (grid <= 2 * sms) return launch_kernel(w8_few_kernel<1, 2, 4>, grid, kThreads, 0, s, L, wk);
    if (grid <= 3 * sms) return launch_kernel(w8_few_kernel<1, 3, 2>, grid, kThreads, 0, s, L, wk);
    return launch_kernel(w8_few_kernel<1, 4, 2>, grid, kThreads, 0, s, L, wk);
}

}  // namespace cbs
