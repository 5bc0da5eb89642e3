// k_w8.cu -- products of 8-bit integers with a scale for each token and each channel:
//
//   y[m, n] = act( xs[m] ws[n] sum_k x[m, k] w[n, k] + bias[n] )
//
// Y^T = W X^T on tcgen05: 128 outputs of a CTA are the lanes of tensor memory, its
// input rows the product's columns.  Codes are widened to f16, which holds them
// exactly, and sums of products are kept in 32 bits: whole numbers, exact below
// 2^24, past which each of an MMA's additions (sixteen products) rounds or cuts after 23
// bits.  (The card's 8-bit integer tensor rate is far below its f16 one.)
//
// TMA brings the codes, one byte each.  Two warpgroups in turn widen a stage's
// weights and store them to tensor memory as the MMA's A operand; other warps widen
// the inputs into the swizzled rows of B.  Shared memory's bandwidth bounds it: a
// byte is written by TMA, read by a thread, and B's twofold written and read again.
// So many rows go to k_w8_pair.cu, where two CTAs share a tile.
//
// For few rows the weights' bytes bound it.  Shares of k are then CTAs of a cluster,
// which add their sums in order through distributed shared memory.
//
// Measured with the weights in turn (not in L2), 16384 x 8192: 32 rows 28 us, 4.8 TB/s;
// 64 rows 34 us; 128 rows 37 us, 0.94 PFLOP/s.  1001 x 2064, 400 rows 9.7 us: starts and ends.
#include <algorithm>

#include "w8.cuh"

namespace cbs {

using namespace w8;

namespace {

constexpr int kShareMost = 8;                // shares of k: CTAs of a cluster
constexpr int kPitch = kOut + 4;             // floats of a row of a share's sums

// kN: input rows of a tile.
template <int kN>
struct W8Tile {
    static constexpr int kW = kOut * 128, kRaw = kW + kN * 128;
    static constexpr int kOp = kN * 256;                  // a stage of B: two panels of 64
    // (64 rows with two stages let two CTAs on an SM, which waited for their loads: 64 rows
    // of 16384 x 8192 38.7 us, with four 33.3; of 6144 x 4096 12.0 and 12.3.)
    static constexpr int kStages = 4;
    static constexpr int kOps = kN <= 32 ? 2 : 3;
    // Warps that widen inputs, and the groups of them that take stages in turn: a
    // group then has two stages' time for its loads, stores and fence.
    static constexpr int kWiden = kN >= 128 ? 8 : kN / 16, kTurns = kN >= 32 ? 2 : 1;
    // A wait knows a barrier's turns apart only while it is less than two behind.  Loads
    // land out of order, so whoever takes stages in turn has to see every turn of its
    // slots: their number is a multiple of two (weights) and of kTurns.  A group's last
    // stage waited for an MMA kTurns + kOps stages back, and MMAs end in order: with no
    // more groups than places of B, that place's turn before the last one has ended.  So
    // too the two groups of weights and the places of A.
    static_assert(kStages % 2 == 0 && kStages % kTurns == 0 && kTurns <= kOps, "turns");
    static constexpr int kStoreWarps = kWiden >= 8 ? 16 : 8;   // at the end: each has 32 outputs of its part of the rows
    static constexpr int kWarpMma = 8 + kWiden, kWarpTma = kWarpMma + 1, kThreads = (kWarpTma + 1) * 32;
    static constexpr int kOpAt = kStages * kRaw, kBars = kOpAt + kOps * kOp;
    // Places of A in tensor memory, a stage each: from a place's MMA back to its next one
    // takes some 2500 cycles of hand-offs, so as many as fit.
    static constexpr int kABufs = kN >= 128 ? 4 : 3, kACols = kStageK / 2;
    static_assert(2 <= kABufs, "turns");
    static constexpr int kTmem = kABufs * kACols + kN <= 256 ? 256 : 512;
    // raw_full[], raw_empty[], b_ready[], b_free[], a_ready[], a_free[], done;
    // TMEM address, flag; the input rows' scales
    static constexpr int kNumBars = 2 * kStages + 2 * kOps + 2 * kABufs + 1;
    static constexpr int kScales = kBars + kNumBars * 8 + 16, kSmem = kScales + kN * 4;
    static_assert(kABufs * kACols + kN <= 512 && kScales % 8 == 0 && kRaw % 1024 == 0 && kOp % 1024 == 0, "tensor memory; operands at multiples of 1 KB");
    static_assert(kSmem <= kMaxDynSmem, "shared memory");
    static_assert(kN * kPitch * 4 <= kBars, "a share's sums fit where the stages were");
};

template <int kN>
__global__ void __launch_bounds__(W8Tile<kN>::kThreads, W8Tile<kN>::kSmem <= 113 * 1024 ? 2 : 1)
w8_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, const W8Launch L, int split) {
    using C = W8Tile<kN>;
    extern __shared__ __align__(1024) unsigned char smem[];   // the only shared memory: starts at a multiple of 1 KB
    const uint32_t sbase = ptx::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int share = split > 1 ? (int)cluster_rank() : 0;   // of k
    const int n0 = (blockIdx.x / split) * kOut, m0 = blockIdx.y * kN;
    const int stages = (L.k + kStageK - 1) / kStageK;
    const int st0 = (int)((long long)stages * share / split), ns = (int)((long long)stages * (share + 1) / split) - st0;
    const auto bar = [&](int i) { return sbase + C::kBars + 8u * i; };
    const auto raw_full = [&](int s) { return bar(s); };
    const auto raw_empty = [&](int s) { return bar(C::kStages + s); };
    const auto b_ready = [&](int s) { return bar(2 * C::kStages + s); };
    const auto b_free = [&](int s) { return bar(2 * C::kStages + C::kOps + s); };
    const auto a_ready = [&](int w) { return bar(2 * C::kStages + 2 * C::kOps + w); };
    const auto a_free = [&](int w) { return bar(2 * C::kStages + 2 * C::kOps + C::kABufs + w); };
    const uint32_t done = bar(2 * C::kStages + 2 * C::kOps + 2 * C::kABufs);
    volatile uint32_t *const words = reinterpret_cast<volatile uint32_t *>(smem + C::kBars + 8 * C::kNumBars);
    // words[0]: TMEM address; [1]: a wait ran out

    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            ptx::mbar_init(raw_full(s), 1);
            ptx::mbar_init(raw_empty(s), 4 + C::kWiden / C::kTurns);   // the warps whose turn it is
        }
        for (int s = 0; s < C::kOps; ++s) {
            ptx::mbar_init(b_ready(s), C::kWiden / C::kTurns);
            ptx::mbar_init(b_free(s), 1);
        }
        for (int w = 0; w < C::kABufs; ++w) {
            ptx::mbar_init(a_ready(w), 4);
            ptx::mbar_init(a_free(w), 1);
        }
        ptx::mbar_init(done, 1);
        ptx::fence_mbar_init();
        words[1] = 0;
    }
    if (warp == C::kWarpMma) {
        ptx::tmem_alloc(sbase + C::kBars + 8 * C::kNumBars, C::kTmem);
        ptx::tmem_relinquish();
    }
    if (warp == C::kWarpTma && lane < 2) ptx::prefetch_tmap(lane ? &tm_x : &tm_w);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const uint32_t tmem = words[0];
    const auto t_a = [&](int w) { return tmem + (uint32_t)(w * C::kACols); };
    const uint32_t t_d = tmem + C::kABufs * C::kACols;

    const auto wait = [&](uint32_t bar_, uint32_t parity) -> bool {
        if (ptx::mbar_wait_bounded(bar_, parity, kWaitNs)) return true;
        words[1] = 1;
        atomicOr(L.status, kStatusTimeout);
        return false;
    };
    const auto lost = [&] { return words[1] != 0; };
    float *const xs = reinterpret_cast<float *>(smem + C::kScales);
    float ws = 0.0f, bias = 0.0f;   // of a thread's output
    if (warp < C::kStoreWarps) {
        for (int i = tid; i < kN; i += C::kStoreWarps * 32) xs[i] = m0 + i < L.rows ? L.x_scale[m0 + i] : 0.0f;
        if (n0 + (tid & 127) < L.n) {
            ws = L.w_scale[n0 + (tid & 127)];
            if (L.bias) bias = L.bias[n0 + (tid & 127)];
        }
    }

    if (warp == C::kWarpMma) {
        // ------------------------------------------------------- MMA issue
        constexpr uint32_t idesc = (1u << 4) | ((kN >> 3) << 17) | ((kOut >> 4) << 24);   // f16 operands
        const uint32_t lead = elect_one();
        const uint64_t d_b = ptx::smem_desc(sbase + C::kOpAt, 16, 1024, 2);
        int op = 0;
        uint32_t op_parity = 0;
        for (int i = 0; i < ns; ++i) {
            const bool ok = wait(a_ready(i % C::kABufs), (i / C::kABufs) & 1) && wait(b_ready(op), op_parity) && !lost();
            if (!__all_sync(~0u, ok)) break;
            ptx::tc_fence_after();
            const uint64_t b = d_b + (uint32_t)(op * C::kOp) / 16;
#pragma unroll
            for (int x = 0; x < kStageK / 16; ++x)
                mma_ts(lead, t_d, t_a(i % C::kABufs) + 8 * x, b + (uint32_t)((x >> 2) * kN * 8 + (x & 3) * 2), idesc, i > 0 || x > 0);
            mma_commit(lead, a_free(i % C::kABufs));
            mma_commit(lead, b_free(op));
            if (++op == C::kOps) op = 0, op_parity ^= 1;
        }
        __syncwarp();
        mma_commit(lead, done);   // all that was issued, however the loop ended
    } else if (warp == C::kWarpTma) {
        // ------------------------------------------------------- TMA
        if (lane == 0) {
            int slot = 0, count = 0;
            uint32_t parity = 1;
            for (int i = 0; i < ns; ++i) {
                if (!wait(raw_empty(slot), parity) || lost()) break;
                const uint32_t at = sbase + slot * C::kRaw;
                ptx::mbar_arrive_expect_tx(raw_full(slot), C::kRaw);
                ptx::tma_load_2d(at, &tm_w, raw_full(slot), (st0 + i) * kStageK, n0);
                ptx::tma_load_2d(at + C::kW, &tm_x, raw_full(slot), (st0 + i) * kStageK, m0);
                ++count;
                if (++slot == C::kStages) slot = 0, parity ^= 1;
            }
            // The copies in flight land before the CTA leaves, whoever gives up, and when.
            for (int x = max(0, count - C::kStages); x < count; ++x)
                ptx::mbar_wait_bounded(raw_full(x % C::kStages), (x / C::kStages) & 1, kWaitNs);
        }
    } else if (warp >= 8) {
        // ------------------------------------------------------- inputs
        // Sixteen codes a unit, eight units a row.
        constexpr int kLanes = C::kWiden / C::kTurns * 32, kPer = kN * 8 / kLanes, kOnce = kPer < 8 ? kPer : 8;
        const int turn = (tid - 256) / kLanes, t = (tid - 256) % kLanes, u = t & 7, row0 = t >> 3;
        for (int i = turn; i < ns; i += C::kTurns) {
            const int slot = i % C::kStages, op = i % C::kOps;
            bool ok = wait(raw_full(slot), (i / C::kStages) & 1);
            if (!__all_sync(~0u, ok)) break;
            unsigned char *const to = smem + C::kOpAt + op * C::kOp + (u >> 2) * kN * 128;
#pragma unroll
            for (int pass = 0; pass < kPer / kOnce; ++pass) {
                uint4 raw[kOnce];
#pragma unroll
                for (int x = 0; x < kOnce; ++x) {
                    const int row = row0 + (pass * kOnce + x) * (kLanes / 8);
                    raw[x] = *reinterpret_cast<const uint4 *>(smem + slot * C::kRaw + C::kW + row * 128 + ((u ^ (row & 7)) << 4));
                }
                if (pass == kPer / kOnce - 1) {
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(raw_empty(slot));
                }
                if (pass == 0) {
                    ok = wait(b_free(op), (i / C::kOps + 1) & 1) && !lost();
                    if (!__all_sync(~0u, ok)) break;
                }
#pragma unroll
                for (int x = 0; x < kOnce; ++x) {
                    const int row = row0 + (pass * kOnce + x) * (kLanes / 8);
                    widen_input(to, row, u, raw[x]);
                }
            }
            if (!__all_sync(~0u, ok)) break;
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(b_ready(op));
        }
    } else {
        // ------------------------------------------------------- weights
        const int wg = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        for (int i = wg; i < ns; i += 2) {
            const int slot = i % C::kStages, buf = i % C::kABufs;
            bool ok = wait(raw_full(slot), (i / C::kStages) & 1);
            if (!__all_sync(~0u, ok)) break;
            const unsigned char *const from = smem + slot * C::kRaw + row * 128;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t a[32];
                widen_weights(from, row, h, a);
                if (h == 0) {
                    ok = wait(a_free(buf), (i / C::kABufs + 1) & 1) && !lost();
                    if (!__all_sync(~0u, ok)) break;
                    ptx::tc_fence_after();
                }
                tmem_st32(t_a(buf) + lanes + 32 * h, a);
            }
            if (!__all_sync(~0u, ok)) break;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(raw_empty(slot));
            tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(a_ready(buf));
        }
    }
    __syncwarp();
    // Nothing goes on while an MMA reads shared or tensor memory.
    if (!ptx::mbar_wait_bounded(done, 0, kWaitNs)) atomicOr(L.status, kStatusTimeout);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();

    // ------------------------------------------------------------ output
    if (warp < C::kStoreWarps) {
        // A thread has one output of some of the input rows.
        const int part = warp >> 2, row = tid & 127, n = n0 + row;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        constexpr int kCols = kN / (C::kStoreWarps / 4), kPart = kCols < 16 ? 8 : 16;
        float *const sum = reinterpret_cast<float *>(smem);   // [input row][output] of this share
#pragma unroll 1
        for (int q = 0; q < kCols / kPart; ++q) {
            uint32_t v[kPart];
            const int col = part * kCols + q * kPart;
            if (ns > 0) {
                if constexpr (kPart == 8) ptx::tmem_ld8(t_d + lanes + col, v);
                else ptx::tmem_ld16(t_d + lanes + col, v);
                ptx::tmem_ld_wait();
            } else {
#pragma unroll
                for (int e = 0; e < kPart; ++e) v[e] = 0;
            }
            if (split > 1) {
#pragma unroll
                for (int e = 0; e < kPart; ++e) sum[(col + e) * kPitch + row] = __uint_as_float(v[e]);
            } else if (n < L.n) {
                store_rows(L, m0 + col, n, v, xs + col, Channel(ws, bias));
            }
        }
    }
    ptx::tc_fence_before();
    if (split > 1) cluster_sync();
    else __syncthreads();
    if (warp == C::kWarpMma) ptx::tmem_dealloc(tmem, C::kTmem);
    if (split == 1) return;
    // Four outputs of a row at a time, every share's on their way together.
    const int rows = min(kN, L.rows - m0);
    for (int i = tid + share * C::kThreads; i < kOut / 4 * rows; i += C::kThreads * split) {
        const int m = i / (kOut / 4), nn = i % (kOut / 4) * 4, n = n0 + nn;
        if (n >= L.n) continue;
        const uint32_t from = sbase + (m * kPitch + nn) * 4;
        float4 v[kShareMost];
#pragma unroll
        for (int p = 0; p < kShareMost; ++p)
            if (p < split) v[p] = ld_cluster4(from, p);
        float y[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
        for (int p = 1; p < kShareMost; ++p)
            if (p < split) y[0] += v[p].x, y[1] += v[p].y, y[2] += v[p].z, y[3] += v[p].w;
        const float x_scale = xs[m];
        const size_t at = (size_t)(m0 + m) * L.n + n;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (n + e >= L.n) break;
            y[e] = Channel(L.w_scale[n + e], L.bias ? L.bias[n + e] : 0.0f)(y[e], x_scale);
            if (L.act == CBS_ACT_SILU) y[e] = silu(y[e]);
        }
        if (L.n % 4 == 0) {
            if (L.out_bf16) *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(L.y) + at) = make_uint2(frag::pack_bf16(y[0], y[1]), frag::pack_bf16(y[2], y[3]));
            else *reinterpret_cast<float4 *>(static_cast<float *>(L.y) + at) = make_float4(y[0], y[1], y[2], y[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (n + e >= L.n) break;
                if (L.out_bf16) static_cast<__nv_bfloat16 *>(L.y)[at + e] = __float2bfloat16_rn(y[e]);
                else static_cast<float *>(L.y)[at + e] = y[e];
            }
        }
    }
    cluster_sync();   // nobody's sums go while another CTA reads them
}

template <int kN>
cbs_status launch_w8_one(const W8Launch &L, int split, cudaStream_t s) {
    using C = W8Tile<kN>;
    alignas(64) CUtensorMap tw, tx;
    CBS_TRY(codes_map(&tw, L.w, L.k, L.n, kOut));
    CBS_TRY(codes_map(&tx, L.x, L.k, L.rows, kN));
    const int tiles = (L.n + kOut - 1) / kOut, row_tiles = (L.rows + kN - 1) / kN;
    auto kern = w8_kernel<kN>;
    static ContextOfDevice set;
    cudaError_t e = set_max_dyn_smem_once(kern, C::kSmem, set);
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(tiles * split, row_tiles);
        cfg.blockDim = dim3(C::kThreads);
        cfg.dynamicSmemBytes = C::kSmem;
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = split;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = (launch_options() & CBS_LAUNCH_PDL) ? 2 : 1;
        e = cudaLaunchKernelEx(&cfg, kern, tw, tx, L, split);
    }
    return cuda_check(e, "8-bit product launch");
}

// One-time weight transform: s = max|w| / 127 over an output's weights, code =
// clamp(rne(w / s), -127, 127).  A warp an output.  A NaN or an infinity among them
// makes the scale NaN, and with it the output.
__global__ void quantize_w8_kernel(const float *__restrict__ w, int n, int k, int8_t *__restrict__ codes, float *__restrict__ scales) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31, step = gridDim.x * (blockDim.x >> 5);
    for (int row = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); row < n; row += step) {
        const float *src = w + (size_t)row * k;
        float top = 0.0f;
        for (int i = lane; i < k; i += 32) top = most_or_nan(top, fabsf(src[i]));
#pragma unroll
        for (int o = 16; o; o >>= 1) top = most_or_nan(top, __shfl_xor_sync(~0u, top, o));
        const float s = top < INFINITY ? __fdiv_rn(top, 127.0f) : __int_as_float(0x7fc00000);
        if (lane == 0) scales[row] = s;
        for (int i = lane; i < k; i += 32) {
            const float q = s > 0.0f ? rintf(__fdiv_rn(src[i], s)) : 0.0f;
            codes[(size_t)row * k + i] = (int8_t)fminf(fmaxf(q, -127.0f), 127.0f);
        }
    }
}

}  // namespace

// The tile and the shares of k, by what was measured (hundredths of a microsecond; 60
// sizes of 256 x 1024 to 16384 x 8192, 1 to 6400 rows, every tile with 1 to 8 shares):
// a CTA's start and end and each of its stages, alone on its SM and, for the tiles of
// which two fit, for two side by side; and the join of shares.  What it takes is 1%
// slower than the best on average and 19% at worst (1024 x 256, 6400 rows: 14.9 us for
// 12.6).
struct W8Cost { int rows, alone, stage, two, stage2, share; };
constexpr W8Cost kCosts[] = {{16, 88, 45, 72, 68, 0}, {32, 128, 36, 128, 65, 0}, {64, 155, 46, 0, 0, 5},
                             {128, 227, 49, 0, 0, 22}, {256, 142, 55, 0, 0, 0}};
constexpr int kJoin = 146;
constexpr int kPairTile = 373;   // of a tile of 256, beside its stages: where the next one's begin late
// Of 152 SMs with a CTA each, that many clusters of 1, 2, 4 and 8 run at once.
constexpr int kAtOnce[] = {152, 76, 36, 15};
//
// Few rows go to k_w8_few.cu: its time and this file's, one row: 1001 x 2064 4.0 and 5.6
// us, 4096 x 4096 5.1 and 8.1, 6144 x 4096 6.6 and 9.1, 8192 x 8192 14.6 and 15.9, 16384 x
// 8192 27.2 and 26.6; sixteen rows: 4.0 and 6.0, 6.6 and 8.6, 9.7 and 10.0, 20 and 17; 70000
// x 256 14 and 9.0.
constexpr long long kFewMost8 = 96ll << 20, kFewMost16 = 28ll << 20;
constexpr int kFewMostOutputs16 = 16384;
constexpr long long kGridMost = 65535;   // row tiles of a launch

cbs_status launch_w8(const W8Launch &L, cudaStream_t s) {
    const long long weights = (long long)L.n * L.k;
    if (L.rows <= 8 ? weights <= kFewMost8 : L.rows <= 16 && weights <= kFewMost16 && L.n <= kFewMostOutputs16)
        return cuda_check(launch_w8_few(L, s), "8-bit product launch");
    const long long sms = current_device_sms(), stages = (L.k + kStageK - 1) / kStageK;
    long long best = 0;
    int rows = 0, split = 1;
    for (const W8Cost &c : kCosts) {
        if (rows && c.rows >= 2 * L.rows) break;   // (half of a larger tile would be empty)
        const long long row_tiles = ((long long)L.rows + c.rows - 1) / c.rows;
        if (row_tiles > kGridMost) continue;
        for (int i = 0; i < (c.rows == 256 ? 1 : 4) && (i == 0 || 2 << i <= stages); ++i) {
            const int x = 1 << i;
            const long long each = (stages + x - 1) / x;
            long long cost;
            if (c.rows == 256) {   // pairs of CTAs
                const long long pairs = std::max(sms / 2, 1ll), tiles = (L.n + 2 * kOut - 1) / (2 * kOut) * row_tiles;
                cost = c.alone + (tiles + pairs - 1) / pairs * (kPairTile + each * c.stage);
            } else {
                const long long at_once = std::max(kAtOnce[i] * sms / 152, 1ll), per = ((L.n + kOut - 1) / kOut * row_tiles + at_once - 1) / at_once;
                const long long join = x > 1 ? kJoin + x * c.share : 0;
                cost = c.two ? per / 2 * (c.two + each * c.stage2 + join) + per % 2 * (c.alone + each * c.stage + join) : per * (c.alone + each * c.stage + join);
            }
            if (!rows || cost < best) best = cost, rows = c.rows, split = x;
        }
    }
    switch (rows) {
    case 16: return launch_w8_one<16>(L, split, s);
    case 32: return launch_w8_one<32>(L, split, s);
    case 64: return launch_w8_one<64>(L, split, s);
    case 128: return launch_w8_one<128>(L, split, s);
    default: return launch_w8_pair(L, s);
    }
}

cudaError_t launch_quantize_w8(const float *w, int n, int k, int8_t *codes, float *scales, cudaStream_t s) {
    const int cap = current_device_sms() * 16, grid = (n + 7) / 8;
    return launch_kernel(quantize_w8_kernel, grid < cap ? grid : cap, 256, 0, s, w, n, k, codes, scales);
}

}  // namespace cbs
