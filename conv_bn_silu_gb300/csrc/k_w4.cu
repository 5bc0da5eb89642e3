// k_w4.cu -- products with 4-bit weights in groups along k, for few rows:
//
//   y[m, n] = act( xs[m] * sum_g s[g, n] * sum_{k in g} x[m, k] (q[n, k] - z[g, n]) + bias[n] )
//
// The weights are read once: half a byte each, so HBM (L2, for small layers)
// bounds the call.  Y^T = W X^T: sixteen outputs fill the rows of an m16n8k16
// MMA and the few input rows its columns.  A packed word holds eight weights
// of one output with weights 2i and 2i + 1 in nibbles i and i + 4, so a shift
// and a mask give a pair in the two halves of a register; 0x4300 | q is the
// bf16 value 128 + q, and taking 128 + z away leaves q - z exactly.  Group
// sums stay apart (exact whole numbers for 8-bit inputs), are scaled in 32
// bits and added to the running total in 32 bits.
//
// Each lane copies the words it will use itself into a ring of its own in
// shared memory (cp.async), several stages ahead, so no thread waits for
// another's copy and the bytes in flight cost no registers.
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

__device__ __forceinline__ float silu(float z) { return __fdiv_rn(z, 1.0f + expf(-z)); }

// GROUP: weights a scale covers (32, 64 or 128).  NT: tiles of eight input
// rows.  RB: tiles of sixteen outputs a warp.  FULL: k is a multiple of the
// stage's 128, so no stage ends early.
//
// What the loop costs is instructions (a weight is half a byte: at HBM's rate an
// SM has a dozen issue slots for a warp's 64 weights), so rows past the ends
// are clamped instead of masked, pointers advance, and for 8-bit inputs the zero
// point comes off the group's whole-number sum (sum x (128 + q) - (128 + z)
// sum x, exact below 2^24) instead of every weight.
template <int GROUP, int NT, int RB, bool XI8, bool FULL>
__global__ void __launch_bounds__(kThreads, NT > 2 ? 1 : 2) w4_kernel(const W4Launch L, int wk) {
    constexpr int V = GROUP / 32;            // words a lane, row and group
    constexpr int kGroups = kStageK / GROUP; // groups in a stage
    constexpr int kRowBytes = 16;            // a lane's bytes of one row in a stage
    constexpr int kXB = XI8 ? 1 : 2;         // bytes of an input
    constexpr bool kEarlyX = NT * kXB <= 2;  // X one stage ahead: 8 NT kXB registers
    extern __shared__ __align__(16) unsigned char smem[];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, j = lane & 3;
    const int wr = warp / wk, part = warp % wk;   // which outputs, which share of k
    const int n0 = (blockIdx.x * (kWarps / wk) + wr) * 16 * RB;
    const int m0 = blockIdx.y * 8 * NT;
    const int stages = (L.k + kStageK - 1) / kStageK;
    const int st0 = (int)((long long)stages * part / wk), st1 = (int)((long long)stages * (part + 1) / wk);
    const int left = L.k - st0 * kStageK;         // weights from this share's start to the row's end

    // This lane's rows: g and g + 8 of each tile (rows past n repeat the last one),
    // at its bytes of the first group; X's row g of each tile (likewise).
    const uint8_t *wp[2 * RB];
    int nrow[2 * RB];
#pragma unroll
    for (int i = 0; i < 2 * RB; ++i) {
        nrow[i] = min(n0 + (i >> 1) * 16 + (i & 1) * 8 + g, L.n - 1);
        wp[i] = L.w + (size_t)nrow[i] * (L.k / 2) + st0 * (kStageK / 2) + j * 4 * V;
    }
    const char *xp[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
        xp[t] = static_cast<const char *>(L.x) + ((size_t)min(m0 + t * 8 + g, L.rows - 1) * L.k + st0 * kStageK + j * 8 * V) * kXB;

    unsigned char *const ring = smem + (size_t)tid * kRowBytes;   // [stage][row][thread], 16 bytes each
    const uint32_t ring32 = ptx::smem_u32(ring);
    const auto copy = [&](int st, int s) {   // stage st into place s of the ring
        if (st < st1) {
#pragma unroll
            for (int i = 0; i < 2 * RB; ++i) {
                const uint32_t dst = ring32 + (s * 2 * RB + i) * kThreads * kRowBytes;
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

    float total[RB][NT][4];
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) total[r][t][i] = 0.0f;

    // The groups' scales and zero points: lane j of a row's four holds those of
    // the stage's group j, some stages ahead and as they were loaded (arithmetic
    // on them here would wait for the loads), and the row's lanes get a group's by
    // a shuffle.
    constexpr int kAhead = RB == 1 ? 4 : 2;
    static_assert(kStages % kAhead == 0, "the rings turn together");
    struct Scale { uint16_t s; uint8_t z; };
    Scale sz[kAhead][2 * RB];
    const uint16_t *sp = static_cast<const uint16_t *>(L.scales);
    const uint8_t *zpt = L.zeros;
    const int groups = L.k / GROUP;
    const auto load_scales = [&](int st, Scale (&to)[2 * RB]) {
        if (st >= st1) return;
        const int gr = st * kGroups + j % kGroups;
        const size_t at = (size_t)(FULL || gr < groups ? gr : groups - 1) * L.n;
#pragma unroll
        for (int i = 0; i < 2 * RB; ++i) {
            to[i].s = __ldg(sp + at + nrow[i]);
            if (zpt) to[i].z = __ldg(zpt + at + nrow[i]);
        }
    };
#pragma unroll
    for (int s = 0; s < kAhead; ++s) load_scales(st0 + s, sz[s]);

    using XWord = typename std::conditional<XI8, uint2, uint4>::type;   // eight consecutive inputs
    XWord xs[kEarlyX ? NT : 1][4];
    const auto load_x = [&](int t, int gi, int v) -> XWord {   // word v of group gi of xp's stage
        return __ldg(reinterpret_cast<const XWord *>(xp[t] + (gi * GROUP + v * 8) * kXB));
    };
    if constexpr (kEarlyX) {
#pragma unroll
        for (int gi = 0; gi < kGroups; ++gi)
            if (st0 < st1 && (FULL || gi * GROUP < left)) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int v = 0; v < V; ++v) xs[t][gi * V + v] = load_x(t, gi, v);
            }
#pragma unroll
        for (int t = 0; t < NT; ++t) xp[t] += kStageK * kXB;
    }
    for (int sb = st0; sb < st1; sb += kStages) {
#pragma unroll
        for (int su = 0; su < kStages; ++su) {
            const int st = sb + su;
            if (st >= st1) break;
            copy(st + kStages - 1, (su + kStages - 1) % kStages);
            ptx::cp_async_wait<kStages - 1>();
            uint32_t wv[2 * RB][4];
#pragma unroll
            for (int i = 0; i < 2 * RB; ++i) {
                const uint4 w = *reinterpret_cast<const uint4 *>(ring + (su * 2 * RB + i) * kThreads * kRowBytes);
                wv[i][0] = w.x; wv[i][1] = w.y; wv[i][2] = w.z; wv[i][3] = w.w;
            }
            const int past = (st - st0) * kStageK;   // weights of the share before this stage
#pragma unroll
            for (int gi = 0; gi < kGroups; ++gi) {
                if (!FULL && past + gi * GROUP >= left) break;
                float acc[RB][NT][4], sx[NT][4];
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        sx[t][i] = 0.0f;
#pragma unroll
                        for (int r = 0; r < RB; ++r) acc[r][t][i] = 0.0f;
                    }
                uint32_t zp[2 * RB];   // 128 + z, a pair of bf16
                float sc[2 * RB];
#pragma unroll
                for (int i = 0; i < 2 * RB; ++i) {
                    const Scale &o = sz[su % kAhead][i];
                    const uint32_t mine = (uint32_t)o.s << 16 | (zpt ? o.z & 15u : 8u);
                    const uint32_t w = kGroups == 1 ? mine : __shfl_sync(~0u, mine, (lane & ~3) | gi);
                    zp[i] = __byte_perm(w, 0x43u, 0x4040);
                    sc[i] = __uint_as_float(w & 0xffff0000u);
                }
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    uint32_t x[NT][4];
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        XWord w;
                        if constexpr (kEarlyX) {
                            w = xs[t][gi * V + v];
                            if (st + 1 < st1 && (FULL || past + kStageK + gi * GROUP < left)) xs[t][gi * V + v] = load_x(t, gi, v);
                        } else {
                            w = load_x(t, gi, v);
                        }
                        if constexpr (XI8) {
                            x[t][0] = frag::i8_pair(__byte_perm(w.x, 0, 0x4140));
                            x[t][1] = frag::i8_pair(__byte_perm(w.x, 0, 0x4342));
                            x[t][2] = frag::i8_pair(__byte_perm(w.y, 0, 0x4140));
                            x[t][3] = frag::i8_pair(__byte_perm(w.y, 0, 0x4342));
                            // a row of ones: the group's sum of x in every output's place
                            constexpr uint32_t kOnes = 0x3f803f80u;
                            frag::mma(sx[t], kOnes, kOnes, kOnes, kOnes, x[t][0], x[t][1]);
                            frag::mma(sx[t], kOnes, kOnes, kOnes, kOnes, x[t][2], x[t][3]);
                        } else {
                            x[t][0] = w.x; x[t][1] = w.y; x[t][2] = w.z; x[t][3] = w.w;
                        }
                    }
#pragma unroll
                    for (int r = 0; r < RB; ++r) {
                        uint32_t a[2][4];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t w = wv[2 * r + i][gi * V + v];
#pragma unroll
                            for (int p = 0; p < 4; ++p) {
                                a[i][p] = ((w >> (4 * p)) & 0x000f000fu) | 0x43004300u;
                                if constexpr (!XI8) a[i][p] = frag::sub_bf16x2(a[i][p], zp[2 * r + i]);
                            }
                        }
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            frag::mma(acc[r][t], a[0][0], a[1][0], a[0][1], a[1][1], x[t][0], x[t][1]);
                            frag::mma(acc[r][t], a[0][2], a[1][2], a[0][3], a[1][3], x[t][2], x[t][3]);
                        }
                    }
                }
#pragma unroll
                for (int r = 0; r < RB; ++r)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if constexpr (XI8)
                                acc[r][t][i] = fmaf(-__uint_as_float(zp[2 * r + (i >> 1)] & 0xffff0000u), sx[t][i], acc[r][t][i]);
                            total[r][t][i] = fmaf(acc[r][t][i], sc[2 * r + (i >> 1)], total[r][t][i]);
                        }
            }
            load_scales(st + kAhead, sz[su % kAhead]);
#pragma unroll
            for (int t = 0; t < NT; ++t) xp[t] += kStageK * kXB;
        }
    }
    ptx::cp_async_wait<0>();
    __syncthreads();   // the ring is free: the shares of k meet in it

    // [warp][input row][output], then summed in the order of the shares.
    constexpr int kN = 16 * RB, kM = 8 * NT, kPitch = kN + 1;
    float *sum = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sum[((size_t)warp * kM + t * 8 + 2 * j + (i & 1)) * kPitch + r * 16 + (i >> 1) * 8 + g] = total[r][t][i];
    __syncthreads();
    const int outs = (kWarps / wk) * kN;
    for (int i = tid; i < outs * kM; i += kThreads) {
        const int m = i / outs, nn = i % outs, w0 = (nn / kN) * wk;
        const int n = blockIdx.x * outs + nn;
        if (m0 + m >= L.rows || n >= L.n) continue;
        float y = 0.0f;
        for (int p = 0; p < wk; ++p) y += sum[((size_t)(w0 + p) * kM + m) * kPitch + nn % kN];
        if (XI8) y *= L.x_scale[m0 + m];
        if (L.bias) y += L.bias[n];
        if (L.act == CBS_ACT_SILU) y = silu(y);
        const size_t at = (size_t)(m0 + m) * L.n + n;
        if (L.out_bf16) static_cast<__nv_bfloat16 *>(L.y)[at] = __float2bfloat16_rn(y);
        else static_cast<float *>(L.y)[at] = y;
    }
}

template <int GROUP, int NT, int RB, bool XI8, bool FULL>
cudaError_t launch_w4_one(const W4Launch &L, cudaStream_t s) {
    const int ring = kStages * 2 * RB * kThreads * 16;
    const int join = kWarps * 8 * NT * (16 * RB + 1) * 4;
    const int smem = ring > join ? ring : join;
    // Warps side by side along k: as few as give every SM one and a half CTAs,
    // since a CTA's warps along n share X (its bytes are 4 rows / (outputs of the
    // CTA) of the weights').
    const int tiles = (L.n + 16 * RB - 1) / (16 * RB), stages = (L.k + kStageK - 1) / kStageK;
    int wk = 1;
    while (wk < kWarps && tiles * wk < current_device_sms() * 12 && wk * 2 <= stages) wk *= 2;
    const int per = kWarps / wk;
    const dim3 grid((tiles + per - 1) / per, (L.rows + 8 * NT - 1) / (8 * NT));
    auto kern = w4_kernel<GROUP, NT, RB, XI8, FULL>;
    cudaError_t e = set_max_dyn_smem(kern, smem);
    if (e != cudaSuccess) return e;
    return launch_kernel(kern, grid, kThreads, smem, s, L, wk);
}

template <int GROUP, bool XI8>
cudaError_t launch_w4_rows(const W4Launch &L, cudaStream_t s) {
    const bool full = L.k % kStageK == 0;
    const auto run = [&](auto nt, auto rb) {
        return full ? launch_w4_one<GROUP, nt, rb, XI8, true>(L, s) : launch_w4_one<GROUP, nt, rb, XI8, false>(L, s);
    };
    using std::integral_constant;
    if (L.rows <= 8) return run(integral_constant<int, 1>{}, integral_constant<int, 1>{});
    if (L.rows <= 16) return run(integral_constant<int, 2>{}, integral_constant<int, 2>{});
    return run(integral_constant<int, 4>{}, integral_constant<int, 2>{});
}

// One-time weight transform: symmetric codes q in 1..15 (zero point 8) with
// s = bf16(max|w| / 7) over each group, q = 8 + clamp(rne(w / s), -7, 7).  A
// warp per group of one output.
__global__ void quantize_w4_kernel(const float *__restrict__ w, int n, int k, int group, uint32_t *__restrict__ packed,
                                   __nv_bfloat16 *__restrict__ scales) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int groups = k / group, lane = threadIdx.x & 31;
    const long long tasks = (long long)n * groups;
    const long long step = (long long)gridDim.x * (blockDim.x >> 5);
    for (long long t = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); t < tasks; t += step) {
        const int row = (int)(t / groups), gi = (int)(t % groups);
        const float *src = w + (size_t)row * k + (size_t)gi * group;
        float top = 0.0f;
        for (int i = lane; i < group; i += 32) top = fmaxf(top, fabsf(src[i]));
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(top, 7.0f));
        const float s = __bfloat162float(sb);
        if (lane == 0) scales[(size_t)gi * n + row] = sb;
        if (lane < group / 8) {
            uint32_t word = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float q = s > 0.0f ? rintf(__fdiv_rn(src[lane * 8 + i], s)) : 0.0f;
                q = q != q ? 0.0f : fminf(fmaxf(q, -7.0f), 7.0f);
                const int nibble = (i >> 1) + 4 * (i & 1);
                word |= (uint32_t)((int)q + 8) << (4 * nibble);
            }
            packed[((size_t)row * k + (size_t)gi * group) / 8 + lane] = word;
        }
    }
}

}  // namespace

cudaError_t launch_w4(const W4Launch &L, cudaStream_t s) {
    switch (L.group) {
    case 32: return L.x_int8 ? launch_w4_rows<32, true>(L, s) : launch_w4_rows<32, false>(L, s);
    case 64: return L.x_int8 ? launch_w4_rows<64, true>(L, s) : launch_w4_rows<64, false>(L, s);
    default: return L.x_int8 ? launch_w4_rows<128, true>(L, s) : launch_w4_rows<128, false>(L, s);
    }
}

cudaError_t launch_quantize_w4(const float *w, int n, int k, int group, uint8_t *packed, void *scales, cudaStream_t s) {
    const long long tasks = (long long)n * (k / group);
    long long grid = (tasks + 7) / 8;
    const long long cap = (long long)current_device_sms() * 16;
    if (grid > cap) grid = cap;
    return launch_kernel(quantize_w4_kernel, (int)grid, 256, 0, s, w, n, k, group, reinterpret_cast<uint32_t *>(packed),
                         static_cast<__nv_bfloat16 *>(scales));
}

}  // namespace cbs
