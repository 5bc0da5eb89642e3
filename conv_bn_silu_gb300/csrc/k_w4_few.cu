// k_w4_few.cu -- products with 4-bit weights for up to eight input rows of small
// layers (the formula is in k_w4.cu), where latency counts more than rate.
//
// Y^T = W X^T on m16n8k16: sixteen outputs of a warp fill the MMA's rows, the
// input rows its columns; a CTA's eight warps lie along the outputs or along k.
// Everything goes from global memory to the lane that uses it: its packed words
// through a ring of its own in shared memory (cp.async, three stages ahead, no
// barrier), X and the scales through registers.  There is no tensor memory to
// allocate, no cluster and no hand-off between warps, so a call of 6144 x 4096
// ends in 8.7 us and one of 1001 x 2048 in 3.4, where k_w4.cu takes 10.4 and 5.1;
// per weight it spends half as many instructions again (16384 x 8192: 42 us
// against 33).
//
// A nibble becomes bf16 as in k_w4.cu; for 8-bit inputs the zero point comes off
// the group's whole-number sum (sum x (128 + q) - (128 + z) sum x, exact below
// 2^24) instead of every weight.
#include <type_traits>

#include <cuda_bf16.h>

#include "mma_frag.cuh"
#include "tc_ptx.cuh"
#include "tokens.cuh"

namespace cbs {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kStageK = 128;    // weights along k in one stage of the ring
constexpr int kStages = 4;
constexpr int kSlotBytes = 2 * kThreads * 16;   // a stage: two rows a lane, 16 bytes each

// GROUP: weights a scale covers.  FULL: k is a multiple of the stage's 128, so no
// stage ends early.  wk: warps side by side along k.
template <int GROUP, bool XI8, bool FULL>
__global__ void __launch_bounds__(kThreads, 2) w4_few_kernel(const W4Launch L, int wk) {
    constexpr int V = GROUP / 32;            // words a lane, row and group
    constexpr int kGroups = kStageK / GROUP; // groups in a stage
    constexpr int kXB = XI8 ? 1 : 2;         // bytes of an input
    extern __shared__ __align__(16) unsigned char smem[];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, j = lane & 3;
    const int part = warp % wk;              // which share of k
    const int n0 = (blockIdx.x * (kWarps / wk) + warp / wk) * 16;
    const int stages = (L.k + kStageK - 1) / kStageK;
    const int st0 = (int)((long long)stages * part / wk), st1 = (int)((long long)stages * (part + 1) / wk);
    const int left = L.k - st0 * kStageK;    // weights from this share's start to the row's end

    // This lane's outputs g and g + 8 (past n: the last one again) at its bytes of
    // the first group, and its input row (past the end: the last one again).
    int nrow[2];
    const uint8_t *wp[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        nrow[i] = min(n0 + i * 8 + g, L.n - 1);
        wp[i] = L.w + (size_t)nrow[i] * (L.k / 2) + st0 * (kStageK / 2) + j * 4 * V;
    }
    const char *xp = static_cast<const char *>(L.x) + ((size_t)min(g, L.rows - 1) * L.k + st0 * kStageK + j * 8 * V) * kXB;

    unsigned char *const ring = smem + tid * 16;   // [stage][row][thread], 16 bytes each
    const uint32_t ring32 = ptx::smem_u32(ring);
    const auto copy = [&](int st, int s) {   // stage st into place s of the ring
        if (st < st1) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t dst = ring32 + s * kSlotBytes + i * kThreads * 16;
#pragma unroll
                for (int gi = 0; gi < kGroups; ++gi) {
                    const bool in = FULL || (st - st0) * kStageK + gi * GROUP < left;
                    const uint8_t *src = in ? wp[i] + gi * (GROUP / 2) : L.w;
                    const uint32_t bytes = in ? 4 * V : 0;
                    if constexpr (V == 4) ptx::cp_async_16(dst, src, bytes);
                    else if constexpr (V == 2) ptx::cp_async_8(dst + gi * 8, src, bytes);
                    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + gi * 4), "l"(src), "r"(bytes) : "memory");
                }
                wp[i] += kStageK / 2;
            }
        }
        ptx::cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) copy(st0 + s, s);

    // The groups' scales and zero points: lane j of a row's four holds those of
    // the stage's group j, four stages ahead and as they were loaded (arithmetic
    // on them would wait for the loads); the row's lanes get a group's by a shuffle.
    struct Scale { uint16_t s; uint8_t z; };
    Scale sz[kStages][2];
    const int groups = L.k / GROUP;
    const auto load_scales = [&](int st, Scale (&to)[2]) {
        if (st >= st1) return;
        const int gr = st * kGroups + j % kGroups;
        const size_t at = (size_t)(FULL || gr < groups ? gr : groups - 1) * L.n;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            to[i].s = __ldg(static_cast<const uint16_t *>(L.scales) + at + nrow[i]);
            if (L.zeros) to[i].z = __ldg(L.zeros + at + nrow[i]);
        }
    };
#pragma unroll
    for (int s = 0; s < kStages; ++s) load_scales(st0 + s, sz[s]);

    using XWord = typename std::conditional<XI8, uint2, uint4>::type;   // eight consecutive inputs
    XWord xs[4];   // a stage ahead
    const auto load_x = [&](int gi, int v) -> XWord { return __ldg(reinterpret_cast<const XWord *>(xp + (gi * GROUP + v * 8) * kXB)); };
#pragma unroll
    for (int gi = 0; gi < kGroups; ++gi)
        if (st0 < st1 && (FULL || gi * GROUP < left)) {
#pragma unroll
            for (int v = 0; v < V; ++v) xs[gi * V + v] = load_x(gi, v);
        }
    xp += kStageK * kXB;

    float total[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int sb = st0; sb < st1; sb += kStages) {
#pragma unroll
        for (int su = 0; su < kStages; ++su) {
            const int st = sb + su;
            if (st >= st1) break;
            copy(st + kStages - 1, (su + kStages - 1) % kStages);
            ptx::cp_async_wait<kStages - 1>();
            uint32_t wv[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 w = *reinterpret_cast<const uint4 *>(ring + su * kSlotBytes + i * kThreads * 16);
                wv[i][0] = w.x; wv[i][1] = w.y; wv[i][2] = w.z; wv[i][3] = w.w;
            }
            const int past = (st - st0) * kStageK;   // weights of the share before this stage
#pragma unroll
            for (int gi = 0; gi < kGroups; ++gi) {
                if (!FULL && past + gi * GROUP >= left) break;
                float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f}, sx[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                uint32_t zp[2];   // 128 + z, a pair of bf16
                float sc[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const Scale &o = sz[su][i];
                    const uint32_t mine = (uint32_t)o.s << 16 | (L.zeros ? o.z & 15u : 8u);
                    const uint32_t w = __shfl_sync(~0u, mine, (lane & ~3) | gi);
                    zp[i] = __byte_perm(w, 0x43u, 0x4040);
                    sc[i] = __uint_as_float(w & 0xffff0000u);
                }
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    uint32_t x[4];
                    const XWord y = xs[gi * V + v];
                    if (st + 1 < st1 && (FULL || past + kStageK + gi * GROUP < left)) xs[gi * V + v] = load_x(gi, v);
                    if constexpr (XI8) {
                        x[0] = frag::i8_pair(__byte_perm(y.x, 0, 0x4140));
                        x[1] = frag::i8_pair(__byte_perm(y.x, 0, 0x4342));
                        x[2] = frag::i8_pair(__byte_perm(y.y, 0, 0x4140));
                        x[3] = frag::i8_pair(__byte_perm(y.y, 0, 0x4342));
                        // a row of ones: the group's sum of x in every output's place
                        constexpr uint32_t kOnes = 0x3f803f80u;
                        frag::mma(sx, kOnes, kOnes, kOnes, kOnes, x[0], x[1]);
                        frag::mma(sx, kOnes, kOnes, kOnes, kOnes, x[2], x[3]);
                    } else {
                        x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
                    }
                    uint32_t a[2][4];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int p = 0; p < 4; ++p) {
                            a[i][p] = ((wv[i][gi * V + v] >> (4 * p)) & 0x000f000fu) | 0x43004300u;
                            if constexpr (!XI8) a[i][p] = frag::sub_bf16x2(a[i][p], zp[i]);
                        }
                    frag::mma(acc, a[0][0], a[1][0], a[0][1], a[1][1], x[0], x[1]);
                    frag::mma(acc, a[0][2], a[1][2], a[0][3], a[1][3], x[2], x[3]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (XI8) acc[i] = fmaf(-__uint_as_float(zp[i >> 1] & 0xffff0000u), sx[i], acc[i]);
                    total[i] = fmaf(acc[i], sc[i >> 1], total[i]);
                }
            }
            load_scales(st + kStages, sz[su]);
            xp += kStageK * kXB;
        }
    }
    ptx::cp_async_wait<0>();
    __syncthreads();   // the ring is free: the shares of k meet in it

    // [warp][input row][output], then summed in the order of the shares.
    constexpr int kPitch = 17;
    float *sum = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[(warp * 8 + 2 * j + (i & 1)) * kPitch + (i >> 1) * 8 + g] = total[i];
    __syncthreads();
    const int outs = (kWarps / wk) * 16;
    for (int i = tid; i < outs * L.rows; i += kThreads) {
        const int m = i / outs, nn = i % outs, w0 = (nn / 16) * wk, n = blockIdx.x * outs + nn;
        if (n >= L.n) continue;
        float y = 0.0f;
        for (int p = 0; p < wk; ++p) y += sum[((w0 + p) * 8 + m) * kPitch + nn % 16];
        if (XI8) y *= L.x_scale[m];
        if (L.bias) y += L.bias[n];
        if (L.act == CBS_ACT_SILU) y = silu(y);
        const size_t at = (size_t)m * L.n + n;
        if (L.out_bf16) static_cast<__nv_bfloat16 *>(L.y)[at] = __float2bfloat16_rn(y);
        else static_cast<float *>(L.y)[at] = y;
    }
}

template <int GROUP, bool XI8>
cudaError_t launch_few(const W4Launch &L, cudaStream_t s) {
    static_assert(kWarps * 8 * 17 * 4 <= kStages * kSlotBytes, "sums fit the ring");
    // Warps along k until the outputs' tiles times that give each SM twelve warps.
    const int tiles = (L.n + 15) / 16, stages = (L.k + kStageK - 1) / kStageK;
    int wk = 1;
    while (wk < kWarps && tiles * wk < current_device_sms() * 12 && wk * 2 <= stages) wk *= 2;
    const int per = kWarps / wk, grid = (tiles + per - 1) / per;
    if (L.k % kStageK == 0) return launch_kernel(w4_few_kernel<GROUP, XI8, true>, grid, kThreads, kStages * kSlotBytes, s, L, wk);
    return launch_kernel(w4_few_kernel<GROUP, XI8, false>, grid, kThreads, kStages * kSlotBytes, s, L, wk);
}

}  // namespace

cudaError_t launch_w4_few(const W4Launch &L, cudaStream_t s) {
    switch (L.group) {
    case 32: return L.x_int8 ? launch_few<32, true>(L, s) : launch_few<32, false>(L, s);
    case 64: return L.x_int8 ? launch_few<64, true>(L, s) : launch_few<64, false>(L, s);
    default: return L.x_int8 ? launch_few<128, true>(L, s) : launch_few<128, false>(L, s);
    }
}

}  // namespace cbs
