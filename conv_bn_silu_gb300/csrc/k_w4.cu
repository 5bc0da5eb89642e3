// k_w4.cu -- products with 4-bit weights in groups along k, for few rows:
//
//   y[m, n] = act( xs[m] * sum_g s[g, n] * sum_{k in g} x[m, k] (q[n, k] - z[g, n]) + bias[n] )
//
// The weights are read once: half a byte each, so HBM (L2, for small layers)
// bounds the call, and after it the instructions that turn nibbles into
// operands.  Y^T = W X^T on tcgen05: 128 outputs are the rows of the product (the
// lanes of tensor memory) and the input rows its 16, 32 or 64 columns.  A thread
// owns an output: it takes 128 of its weights from shared memory, turns them into
// bf16 and stores them to tensor memory as the MMA's A operand; X comes by TMA as
// B (8-bit X is widened by the threads).  A piece's sums come back through tensor
// memory, are scaled in 32 bits and added to the thread's running totals, so
// every weight costs about two instructions and the MMA none of the threads'.
// (On mma.sync the same product spent as many again on fragments of X and on
// the MMAs: 38 us for 16 rows of 8192 x 16384.)
//
// A packed word holds eight weights of one output with weights 2i and 2i + 1 in
// nibbles i and i + 4, so a shift and a mask-and-or give a pair in the two halves
// of a register: 0x4300 | q is the bf16 value 128 + q, and taking 128 + z away
// leaves q - z exactly.  Products of bf16 pairs are exact in 32 bits, and sums of
// 8-bit inputs are whole numbers below 2^24.
//
// Two warpgroups take a half of every stage of k each: while the MMA of a
// group's piece runs, it dequantises the next.  A handshake costs 150 to 250
// cycles and 64 weights about 300, so pieces are of 128.
// 16 rows of 16384 x 8192, groups of 64: 29 us, 2.5 TB/s of its 73 MB; the issue
// slots that dequantise are half full, and the hand-offs between the threads and
// the MMA take most of the rest.  Made for few rows: from 17 on a thread's running
// totals are 32 or 64, and where two CTAs an SM leave it 80 registers (by tensor
// memory they could), some of them are spilled.
// Shares of k are CTAs of a cluster, which add their sums in order through
// distributed shared memory.
#include <type_traits>

#include <cuda_bf16.h>

#include "mma_frag.cuh"
#include "tc_ptx.cuh"
#include "tc_warp.cuh"
#include "tokens.cuh"

namespace cbs {

namespace {

constexpr int kOut = 128;                    // outputs of a CTA: tensor memory's lanes
constexpr int kStageK = 256, kPiece = 128;   // weights along k in a stage (128 bytes a row) and in a warpgroup's piece of it
constexpr int kPanels = kStageK / 64;        // of X in a stage: 64 inputs, 128 bytes a row
constexpr int kWorkers = 256, kThreads = kWorkers + 96;    // two warpgroups; MMA, TMA and scales
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s per wait

// Largest layer that k_w4_few.cu takes, for up to eight input rows.  One row,
// k_w4_few.cu's time and this file's: 0.4 M weights 2.8 and 4.0 us, 2 M 2.9 and 4.6,
// 16 M 6.6 and 9.8, 24 M 8.6 and 10.7, 32 M 10.4 and 10.8, 64 M 22 and 19, 128 M 42
// and 33.
constexpr long long kFewMost = 48ll << 20;

// GROUP: weights a scale covers.  kN: input rows of a CTA.
template <int GROUP, int kN>
struct W4Tile {
    static constexpr int kSubs = kPiece / GROUP;                        // groups in a piece
    static constexpr int kW = kOut * 128, kX = kPanels * kN * 128;      // a stage's weights; inputs
    static constexpr int kGroups = kStageK / GROUP;
    // Scales [group][output], then zero points; each group's from the word that
    // holds its first, so a row may start a few elements late.
    static constexpr int kSPitch = kOut * 2 + 8, kZPitch = kOut + 4, kZAt = kGroups * kSPitch;
    static constexpr int kS = (kZAt + kGroups * kZPitch + 1023) / 1024 * 1024;
    static constexpr int kSlot = kW + kX + kS;
    static constexpr int kStages = kN == 16 ? 4 : kN == 32 ? 3 : 2;
    static_assert(kSlot % 1024 == 0, "operands start at multiples of 1 KB");
    // full[], x_ready[], empty[], a_ready[2], d_ready[2], drain; TMEM address, flag
    static constexpr int kBars = kStages * kSlot, kNumBars = 3 * kStages + 5;
    static constexpr int kSmem = kBars + kNumBars * 8 + 16;
    // tensor memory: A [warpgroup][64], then the results [warpgroup][sub][kN]
    static constexpr int kACols = 2 * (kPiece / 2), kDCols = 2 * kSubs * kN;
    static constexpr int kTmem = kACols + kDCols <= 256 ? 256 : 512;
    static_assert(kACols + kDCols <= 512, "tensor memory");
    // at the end: each group's sums [2][kN][kOut + 1]
    static_assert(2 * kN * (kOut + 1) * 4 <= kBars, "sums fit where the stages were");
};

// A float of another CTA's shared memory (this CTA's address, that CTA's rank).
__device__ __forceinline__ float ld_cluster(uint32_t addr, uint32_t rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

template <int GROUP, int kN, bool XI8>
__global__ void __launch_bounds__(kThreads, W4Tile<GROUP, kN>::kTmem == 256 ? 2 : 1)
w4_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, const W4Launch L, int split) {
    using C = W4Tile<GROUP, kN>;
    extern __shared__ __align__(1024) unsigned char smem[];   // the only shared memory: starts at a multiple of 1 KB
    const uint32_t sbase = ptx::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = split > 1 ? (int)cluster_rank() : 0;
    const int n0 = (blockIdx.x / split) * kOut, m0 = blockIdx.y * kN;
    const int stages = (L.k + kStageK - 1) / kStageK;
    const int st0 = (int)((long long)stages * rank / split), ns = (int)((long long)stages * (rank + 1) / split) - st0;
    const auto bar = [&](int i) { return sbase + C::kBars + 8u * i; };
    const auto full = [&](int s) { return bar(s); };                          // a stage has arrived
    const auto x_ready = [&](int s) { return bar(C::kStages + s); };          // its 8-bit inputs are widened
    const auto empty = [&](int s) { return bar(2 * C::kStages + s); };        // and it has been used
    const auto a_ready = [&](int w) { return bar(3 * C::kStages + w); };       // a piece's operand is stored
    const auto d_ready = [&](int w) { return bar(3 * C::kStages + 2 + w); };   // and its sums are there
    const uint32_t drain = bar(3 * C::kStages + 4);
    volatile uint32_t *const words = reinterpret_cast<volatile uint32_t *>(smem + C::kBars + 8 * C::kNumBars);
    // words[0]: TMEM address; [1]: a wait ran out

    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            ptx::mbar_init(full(s), 1 + 32);               // TMA's, and the scale warp's lanes'
            ptx::mbar_init(x_ready(s), kWorkers / 32);
            ptx::mbar_init(empty(s), kWorkers / 32 + 1);   // every worker warp, and the MMAs
        }
        for (int w = 0; w < 2; ++w) {
            ptx::mbar_init(a_ready(w), 4);
            ptx::mbar_init(d_ready(w), 1);
        }
        ptx::mbar_init(drain, 1);
        ptx::fence_mbar_init();
        words[1] = 0;
    }
    if (warp == 8) {
        ptx::tmem_alloc(sbase + C::kBars + 8 * C::kNumBars, C::kTmem);
        ptx::tmem_relinquish();
    }
    if (warp == 9 && lane < 2) ptx::prefetch_tmap(lane ? &tm_x : &tm_w);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const uint32_t tmem = words[0];
    const auto t_a = [&](int w) { return tmem + (uint32_t)w * (kPiece / 2); };
    const auto t_d = [&](int w, int sub) { return tmem + C::kACols + (uint32_t)(w * C::kSubs + sub) * kN; };

    const auto wait = [&](uint32_t bar_, uint32_t parity) -> bool {
        if (ptx::mbar_wait_bounded(bar_, parity, kWaitNs)) return true;
        words[1] = 1;
        atomicOr(L.status, kStatusTimeout);
        return false;
    };
    const auto lost = [&] { return words[1] != 0; };

    float total[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) total[i] = 0.0f;
    const int wg = warp >> 2, row = tid & 127;

    if (warp == 8) {
        // ------------------------------------------------------- MMA issue
        constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((kN >> 3) << 17) | ((kOut >> 4) << 24);
        const uint32_t lead = elect_one();
        const uint64_t d_x = ptx::smem_desc(sbase + C::kW, 16, 1024, 2);
        int slot = 0;
        uint32_t parity = 0;
        bool ok = true;
        for (int i = 0; i < ns && ok; ++i) {
            ok = wait(XI8 ? x_ready(slot) : full(slot), parity) && !lost();
            ok = __all_sync(~0u, ok);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                if (ok) ok = wait(a_ready(w), i & 1);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint64_t x = d_x + (uint32_t)(slot * C::kSlot + w * (kPiece / 64) * kN * 128) / 16;
#pragma unroll
                for (int k = 0; k < kPiece / 16; ++k) {
                    constexpr int kPer = GROUP / 16;   // MMAs of a group
                    mma_ts(lead, t_d(w, k / kPer), t_a(w) + 8 * k, x + (uint32_t)((k >> 2) * kN * 8 + (k & 3) * 2), idesc, k % kPer > 0);
                }
                mma_commit(lead, d_ready(w));
            }
            if (!ok) break;
            mma_commit(lead, empty(slot));
            if (++slot == C::kStages) slot = 0, parity ^= 1;
        }
        __syncwarp();
        mma_commit(lead, drain);   // nothing leaves while an MMA reads shared memory
        if (!ptx::mbar_wait_bounded(drain, 0, kWaitNs)) atomicOr(L.status, kStatusTimeout);
    } else if (warp == 9) {
        // ------------------------------------------------------- TMA
        if (lane == 0) {
            int slot = 0, done = 0;
            uint32_t parity = 1;
            for (int i = 0; i < ns; ++i) {
                if (!wait(empty(slot), parity) || lost()) break;
                const uint32_t at = sbase + slot * C::kSlot;
                ptx::mbar_arrive_expect_tx(full(slot), XI8 ? C::kW : C::kW + C::kX);
                ptx::tma_load_2d(at, &tm_w, full(slot), (st0 + i) * (kStageK / 2), n0);
                if (!XI8)
#pragma unroll
                    for (int x = 0; x < kPanels; ++x)
                        ptx::tma_load_2d(at + C::kW + x * kN * 128, &tm_x, full(slot), (st0 + i) * kStageK + x * 64, m0);
                ++done;
                if (++slot == C::kStages) slot = 0, parity ^= 1;
            }
            // The copies in flight land before the CTA leaves, whoever gives up, and when.
            for (int x = max(0, done - C::kStages); x < done; ++x)
                ptx::mbar_wait_bounded(full(x % C::kStages), (x / C::kStages) & 1, kWaitNs);
        }
    } else if (warp == 10) {
        // ------------------------------------------------------- scales
        // Copied as far ahead as the ring is deep: they come from HBM a row of
        // [k / group][n] at a time, later than the threads that need them could ask.
        // Four outputs a lane where every row starts at a multiple of four (n does);
        // else words of four bytes from the one that holds the row's first element.
        // (9 rows of 4897 x 2944, bf16: 10.5 us; element by element 15.2 us; 4896
        // outputs 8.5 us.)
        const int n = n0 + 4 * lane;
        const bool fours = L.n % 4 == 0;
        const char *sp = static_cast<const char *>(L.scales), *zp = reinterpret_cast<const char *>(L.zeros);
        const long long all = (long long)(L.k / GROUP) * L.n;   // scales
        const auto copy4 = [](uint32_t to, const char *from, int bytes) {
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
        };
        const auto word = [&](uint32_t to, const char *from, long long at, long long bytes, bool in) {   // zeros past the end
            const int left = in ? (int)max(0ll, min(4ll, bytes - at)) : 0;
            copy4(to, from + (left ? at : 0), left);
        };
        int slot = 0;
        uint32_t parity = 1;
        for (int i = 0; i < ns; ++i) {
            if (!__all_sync(~0u, wait(empty(slot), parity))) break;
            const uint32_t to = sbase + slot * C::kSlot + C::kW + C::kX;
            if (fours) {
#pragma unroll
                for (int gr = 0; gr < C::kGroups; ++gr) {
                    const int k = (st0 + i) * kStageK + gr * GROUP;
                    const bool on = k < L.k && n < L.n;   // groups past k: scale zero
                    const size_t at = on ? (size_t)(k / GROUP) * L.n + n : 0;
                    ptx::cp_async_8(to + gr * C::kSPitch + 8 * lane, sp + 2 * at, on ? 8 : 0);
                    if (L.zeros) copy4(to + C::kZAt + gr * C::kZPitch + 4 * lane, zp + at, on ? 4 : 0);
                }
            } else {
#pragma unroll 1
                for (int gr = 0; gr < C::kGroups; ++gr) {
                    const int k = (st0 + i) * kStageK + gr * GROUP;
                    const bool in = k < L.k;
                    const long long at = (long long)(in ? k / GROUP : 0) * L.n + n0, s_at = 2 * at & ~3ll, z_at = at & ~3ll;
                    const uint32_t s_to = to + gr * C::kSPitch, z_to = to + C::kZAt + gr * C::kZPitch;
                    word(s_to + 4 * lane, sp, s_at + 4 * lane, 2 * all, in);
                    word(s_to + 128 + 4 * lane, sp, s_at + 128 + 4 * lane, 2 * all, in);
                    if (lane == 0) word(s_to + 256, sp, s_at + 256, 2 * all, in);
                    if (L.zeros) {
                        word(z_to + 4 * lane, zp, z_at + 4 * lane, all, in);
                        if (lane == 0) word(z_to + 128, zp, z_at + 128, all, in);
                    }
                }
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(full(slot)) : "memory");
            if (++slot == C::kStages) slot = 0, parity ^= 1;
        }
        ptx::cp_async_commit();
        ptx::cp_async_wait<0>();   // nothing leaves while a copy is in flight
    } else {
        // ------------------------------------------------------- workers
        // 8-bit inputs: 16 codes a unit, a stage ahead.
        constexpr int kXPer = XI8 ? kN * 16 / kWorkers : 1;
        uint4 xr[kXPer];
        const auto load_x = [&](int i) {
#pragma unroll
            for (int x = 0; x < kXPer; ++x) {
                const int unit = x * kWorkers + tid, m = m0 + (unit >> 4), k = (st0 + i) * kStageK + (unit & 15) * 16;
                xr[x] = make_uint4(0, 0, 0, 0);
                if (i < ns && m < L.rows && k < L.k)
                    xr[x] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const int8_t *>(L.x) + (size_t)m * L.k + k));
            }
        };
        if (XI8) load_x(0);
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        float sc[C::kSubs];
        // The sums of the group's last piece, scaled into the totals.
        const auto take = [&] {
#pragma unroll
            for (int u = 0; u < C::kSubs; ++u)
#pragma unroll
                for (int q = 0; q < kN / 16; ++q) {
                    uint32_t v[16];
                    ptx::tmem_ld16(t_d(wg, u) + lanes + 16 * q, v);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) total[16 * q + e] = fmaf(__uint_as_float(v[e]), sc[u], total[16 * q + e]);
                }
        };
        int slot = 0;
        uint32_t parity = 0;
        bool ok = true;
        for (int i = 0; i < ns; ++i) {
            ok = __all_sync(~0u, wait(full(slot), parity));
            if (!ok) break;
            const unsigned char *wt = smem + slot * C::kSlot + row * 128;
            if constexpr (XI8) {
                unsigned char *xt = smem + slot * C::kSlot + C::kW;
#pragma unroll
                for (int x = 0; x < kXPer; ++x) {
                    const int unit = x * kWorkers + tid, m = unit >> 4, c = unit & 15;
                    const uint32_t w[4] = {xr[x].x, xr[x].y, xr[x].z, xr[x].w};
                    uint32_t o[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        o[2 * e] = frag::i8_pair(__byte_perm(w[e], 0, 0x4140));
                        o[2 * e + 1] = frag::i8_pair(__byte_perm(w[e], 0, 0x4342));
                    }
                    unsigned char *p = xt + (c >> 2) * kN * 128 + m * 128;
                    const int ch = (c & 3) * 2;
                    *reinterpret_cast<uint4 *>(p + ((ch ^ (m & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4 *>(p + (((ch + 1) ^ (m & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(x_ready(slot));
                load_x(i + 1);
            }
            uint16_t sn[C::kSubs];
            uint32_t zp[C::kSubs];   // 128 + z, a pair of bf16
#pragma unroll
            for (int u = 0; u < C::kSubs; ++u) {
                const unsigned char *from = smem + slot * C::kSlot + C::kW + C::kX;
                const int gr = wg * C::kSubs + u;
                const uint32_t late = (uint32_t)(((st0 + i) * C::kGroups + gr) * L.n) & 3u;   // the group's first element in its word
                sn[u] = reinterpret_cast<const uint16_t *>(from + gr * C::kSPitch)[row + (late & 1u)];
                zp[u] = 0x43004300u | (L.zeros ? (from[C::kZAt + gr * C::kZPitch + row + late] & 15u) * 0x00010001u : 0x00080008u);
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t w[8], a[32];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint4 y = *reinterpret_cast<const uint4 *>(wt + (((4 * wg + 2 * b + q) ^ (row & 7)) << 4));
                    w[4 * q] = y.x; w[4 * q + 1] = y.y; w[4 * q + 2] = y.z; w[4 * q + 3] = y.w;
                }
#pragma unroll
                for (int q = 0; q < 8; ++q)
#pragma unroll
                    for (int p = 0; p < 4; ++p)
                        a[4 * q + p] = frag::sub_bf16x2(((w[q] >> (4 * p)) & 0x000f000fu) | 0x43004300u, zp[(64 * b + 8 * q) / GROUP]);
                if (b == 0 && i > 0) {
                    // The operand's place is free once the last piece's MMA is done,
                    // and its sums are there.
                    ok = __all_sync(~0u, wait(d_ready(wg), (i - 1) & 1));
                    if (!ok) break;
                    ptx::tc_fence_after();
                }
                tmem_st32(t_a(wg) + lanes + 32 * b, a);
                if (b == 0 && i > 0) take();
            }
            if (!ok) break;
            tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(a_ready(wg));
                ptx::mbar_arrive(empty(slot));   // the warp has read all it needs of the stage
            }
#pragma unroll
            for (int u = 0; u < C::kSubs; ++u) sc[u] = __uint_as_float((uint32_t)sn[u] << 16);
            if (++slot == C::kStages) slot = 0, parity ^= 1;
        }
        if (ok && ns > 0) {
            ok = __all_sync(~0u, wait(d_ready(wg), (ns - 1) & 1));
            ptx::tc_fence_after();
            if (ok) take();
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 8) ptx::tmem_dealloc(tmem, C::kTmem);

    // The groups' sums, [group][input row][output] where the stages were, then the
    // shares of k in order: each CTA of the cluster finishes its part.
    constexpr int kPitch = kOut + 1;
    float *sum = reinterpret_cast<float *>(smem);
    if (warp < 8) {
#pragma unroll
        for (int m = 0; m < kN; ++m) sum[(wg * kN + m) * kPitch + row] = total[m];
    }
    if (split > 1) cluster_sync();
    else __syncthreads();
    const int rows = min(kN, L.rows - m0);
    for (int i = tid + rank * kThreads; i < kOut * rows; i += kThreads * split) {
        const int m = i / kOut, nn = i % kOut, n = n0 + nn;
        if (n >= L.n) continue;
        float y = 0.0f;
        if (split > 1) {
            for (int p = 0; p < split; ++p) {
                const uint32_t at = sbase + (m * kPitch + nn) * 4;
                y += ld_cluster(at, p);
                y += ld_cluster(at + kN * kPitch * 4, p);
            }
        } else {
            y = sum[m * kPitch + nn] + sum[(kN + m) * kPitch + nn];
        }
        if (XI8) y *= L.x_scale[m0 + m];
        if (L.bias) y += L.bias[n];
        if (L.act == CBS_ACT_SILU) y = silu(y);
        const size_t at = (size_t)(m0 + m) * L.n + n;
        if (L.out_bf16) static_cast<__nv_bfloat16 *>(L.y)[at] = __float2bfloat16_rn(y);
        else static_cast<float *>(L.y)[at] = y;
    }
    if (split > 1) cluster_sync();   // nobody's sums go while another CTA reads them
}

template <int GROUP, int kN, bool XI8>
cbs_status launch_w4_one(const W4Launch &L, cudaStream_t s) {
    using C = W4Tile<GROUP, kN>;
    EncodeTiledFn fn = encode_tiled();
    if (!fn) return fail(CBS_ERR_CUDA, "cannot resolve cuTensorMapEncodeTiled from the driver");
    // Rows of k / 2 bytes by the CTA's outputs, and of inputs by its rows: boxes of
    // 128 bytes a row.
    alignas(64) CUtensorMap tw, tx;
    const auto map = [&](CUtensorMap *tm, CUtensorMapDataType type, const void *p, int cols, int rows, int elem, int box_rows) {
        const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)cols * elem};
        const cuuint32_t box[2] = {(cuuint32_t)(128 / elem), (cuuint32_t)box_rows}, es[2] = {1u, 1u};
        return fn(tm, type, 2, const_cast<void *>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = map(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, L.w, L.k / 2, L.n, 1, kOut);
    if (r != CUDA_SUCCESS) return fail(CBS_ERR_CUDA, "cuTensorMapEncodeTiled (weights) failed (%d)", (int)r);
    tx = tw;   // 8-bit inputs need no map
    if (!XI8) {
        r = map(&tx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, L.x, L.k, L.rows, 2, kN);
        if (r != CUDA_SUCCESS) return fail(CBS_ERR_CUDA, "cuTensorMapEncodeTiled (inputs) failed (%d)", (int)r);
    }

    // Shares of k, by what was measured: an SM's CTAs take 0.72 us a stage between
    // them (two run at a time), a CTA's start and end 1.6 us (two at a time), a
    // cluster of eight half a microsecond more; of shares that cost the same, the
    // fewest.  Groups of 64, 1, 2, 4, 8 shares in us, the one taken in brackets.  16
    // rows: 16384 x 8192 [28.6], 25.9, 29.5, 37.1; 6144 x 4096 15.7, [10.4], 9.6, 12.8;
    // 4096 x 4096 15.7, 10.4, [7.2], 8.1; 1001 x 2048 12.0, 8.5, 6.0, [5.1].  32 rows:
    // [36.5], 32.9, 36.9, 49; 20.2, [13.3], 12.3, 17.9; 20.1, 13.2, [8.7], 10.6; 13.9,
    // 10.1, 6.9, [6.2].  64 rows: [37.7], 45.6, 54, 92; 21.0, [14.9], 19.2, 33; 21.1,
    // 14.7, [10.1], 24; 16.0, 12.1, 7.9, [7.6].  So up to 32 rows two layers get a share
    // 8% to 11% slower than their best, where two cost the same by the rule; with 64
    // the fewest is right.
    const int tiles = (L.n + kOut - 1) / kOut, stages = (L.k + kStageK - 1) / kStageK;
    const int row_tiles = (L.rows + kN - 1) / kN, sms = current_device_sms();
    int split = 1;
    long long best = 0;
    for (int x = 1; x <= 8 && x <= stages; x *= 2) {
        const long long ctas = ((long long)tiles * row_tiles * x + sms - 1) / sms;
        const long long cost = ctas * ((stages + x - 1) / x) * 72 + (ctas + 1) / 2 * 160 + (x == 8 ? 50 : 0);
        if (x == 1 || cost < best) best = cost, split = x;
    }
    auto kern = w4_kernel<GROUP, kN, XI8>;
    static ContextOfDevice set;
    cudaError_t e = set_max_dyn_smem_once(kern, C::kSmem, set);
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(tiles * split, row_tiles);
        cfg.blockDim = dim3(kThreads);
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
    return cuda_check(e, "4-bit product launch");
}

template <int GROUP, bool XI8>
cbs_status launch_w4_rows(const W4Launch &L, cudaStream_t s) {
    if (L.rows <= 16) return launch_w4_one<GROUP, 16, XI8>(L, s);
    // (groups of 32 have four results a piece: 64 columns of each would not fit tensor memory)
    if (L.rows <= 32 || GROUP == 32) return launch_w4_one<GROUP, 32, XI8>(L, s);
    return launch_w4_one<GROUP, GROUP == 32 ? 32 : 64, XI8>(L, s);
}

// One-time weight transform: symmetric codes q in 1..15 (zero point 8) with
// s = bf16(max|w| / 7) over each group, q = 8 + clamp(rne(w / s), -7, 7).  A
// warp per group of one output.  A NaN in a group is its scale (and an infinity
// its own), so what the group adds to is NaN.
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
        for (int i = lane; i < group; i += 32) top = most_or_nan(top, fabsf(src[i]));
#pragma unroll
        for (int o = 16; o; o >>= 1) top = most_or_nan(top, __shfl_xor_sync(~0u, top, o));
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

cbs_status launch_w4(const W4Launch &L, cudaStream_t s) {
    if (L.rows <= 8 && (long long)L.n * L.k <= kFewMost) return cuda_check(launch_w4_few(L, s), "4-bit product launch");
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
