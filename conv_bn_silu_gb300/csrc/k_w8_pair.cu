// k_w8_pair.cu -- products of 8-bit integers (k_w8.cu) for many rows: tiles of 256
// outputs by 256 input rows that two CTAs share (cta_group::2).  Each keeps the widened
// half of the rows and its own 128 outputs' weights; the pair's MMA reads both halves,
// so what a CTA moves through shared memory for a tile is half of what it would alone.
//
// Persistent: a pair takes tiles in turn.  The loads and the widening run on into the
// next tile, whose first MMA waits only until warps of their own have read the last
// one's sums; a CTA's start (tensor memory, barriers, the first loads) is paid once.
//
// Measured: 8192 rows of 8192 x 8192 549 us, 2.0 PFLOP/s, and 611 us, 1.80, with the card warm
// from the calls before; 1024 rows 82 us, 1.67; 2048 rows of 4096 x 8192 80 us, with the tensor
// pipe 84% active and 55% of the issue slots (widening).
#include <algorithm>

#include "w8.cuh"

namespace cbs {

using namespace w8;

namespace {

constexpr int kTileRows = 256, kRows = kTileRows / 2;     // of a tile; that a CTA widens
constexpr int kW = kOut * 128, kRaw = kW + kRows * 128;   // a stage's codes: weights, inputs
constexpr int kOp = kRows * 256;                          // a stage of B: two panels of 64
constexpr int kStages = 4, kOps = 3, kABufs = 4, kACols = kStageK / 2;
constexpr int kTurns = 2;   // groups of warps that take stages in turn, of weights and of inputs (as in k_w8.cu)
static_assert(kStages % kTurns == 0 && kTurns <= kOps && kTurns <= kABufs, "turns");
static_assert(kABufs * kACols + kTileRows == 512, "tensor memory");
constexpr int kStoreWarps = 8, kWarpStore = 16, kWarpMma = kWarpStore + kStoreWarps, kWarpTma = kWarpMma + 1;
constexpr int kThreads = (kWarpTma + 1) * 32;
// raw_full[], raw_empty[], b_ready[], b_free[], peer[], a_ready[], a_free[], d_full, d_free,
// peer_free, done; TMEM address, flag; two tiles' input scales
constexpr int kOpAt = kStages * kRaw, kBars = kOpAt + kOps * kOp, kNumBars = 2 * kStages + 3 * kOps + 2 * kABufs + 4;
constexpr int kScales = kBars + kNumBars * 8 + 16, kSmem = kScales + 2 * kTileRows * 4;
static_assert(kSmem <= kMaxDynSmem && kScales % 8 == 0, "shared memory");
constexpr int kGroupRows = 8;   // row tiles side by side: what pairs read at one time is near a square of the product

// Another CTA's barrier.  What this announces lies in the sender's own shared and
// tensor memory, where its writers' fences have made it visible to the MMA's reads
// before they arrived here; no thread of the other CTA reads it.  So nothing is
// released in the cluster's scope, which took the sender some 1700 cycles a stage (256
// rows of 8192 x 8192: 62.6 us, and 43.7 without).
__device__ __forceinline__ void arrive_at(uint32_t bar, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(bar), "r"(rank));
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(a) : "memory");
}
// As mbar_wait_bounded, for the arrival of the pair's other CTA.
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
    uint64_t t0 = 0;
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\nselp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(1000u)
            : "memory");
        if (ok) return true;
        const uint64_t t = ptx::globaltimer();
        if (t0 == 0) t0 = t;
        else if (t - t0 > limit_ns) return false;
    }
}
// The instructions for two CTAs (a kernel uses one form throughout).
__device__ __forceinline__ void mma_pair(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
// Arrives on `bar` of both CTAs.
__device__ __forceinline__ void commit_pair(uint32_t lead, uint32_t bar) {
    asm volatile(
        "{\n.reg .pred q;\nsetp.ne.b32 q, %1, 0;\n"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2;\n}\n" ::"r"(bar),
        "r"(lead), "h"((uint16_t)3)
        : "memory");
}

struct Grid { int n_tiles, m_tiles, pairs; };

__global__ void __launch_bounds__(kThreads, 1)
w8_pair_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, const W8Launch L, const Grid G) {
    extern __shared__ __align__(1024) unsigned char smem[];   // the only shared memory: starts at a multiple of 1 KB
    const uint32_t sbase = ptx::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_rank(), pair = blockIdx.x >> 1;
    const int ns = (L.k + kStageK - 1) / kStageK, all = G.n_tiles * G.m_tiles;
    const int mine = (all - pair + G.pairs - 1) / G.pairs;   // tiles pair, pair + pairs, ...
    const int total = mine * ns;                             // stages, numbered on through the tiles
    struct Tile { int n0, m0; };
    const auto tile_of = [&](int it) {
        const int t = pair + it * G.pairs, band = kGroupRows * G.n_tiles, first = t / band * kGroupRows;
        const int rows = min(kGroupRows, G.m_tiles - first), in = t % band;
        return Tile{(in / rows) * 2 * kOut + rank * kOut, (first + in % rows) * kTileRows};
    };
    const auto bar = [&](int i) { return sbase + kBars + 8u * i; };
    const auto raw_full = [&](int s) { return bar(s); };
    const auto raw_empty = [&](int s) { return bar(kStages + s); };
    const auto b_ready = [&](int s) { return bar(2 * kStages + s); };
    const auto b_free = [&](int s) { return bar(2 * kStages + kOps + s); };
    const auto peer = [&](int s) { return bar(2 * kStages + 2 * kOps + s); };   // the other CTA's operands are ready
    const auto a_ready = [&](int w) { return bar(2 * kStages + 3 * kOps + w); };
    const auto a_free = [&](int w) { return bar(2 * kStages + 3 * kOps + kABufs + w); };
    constexpr int kLast = 2 * kStages + 3 * kOps + 2 * kABufs;
    const uint32_t d_full = bar(kLast), d_free = bar(kLast + 1), peer_free = bar(kLast + 2), done = bar(kLast + 3);
    volatile uint32_t *const words = reinterpret_cast<volatile uint32_t *>(smem + kBars + 8 * kNumBars);
    // words[0]: TMEM address; [1]: a wait ran out

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(raw_full(s), 1);
            ptx::mbar_init(raw_empty(s), 4 + 4);   // the warps whose turn it is
        }
        for (int s = 0; s < kOps; ++s) {
            ptx::mbar_init(b_ready(s), 4);
            ptx::mbar_init(b_free(s), 1);
            ptx::mbar_init(peer(s), 1);
        }
        for (int w = 0; w < kABufs; ++w) {
            ptx::mbar_init(a_ready(w), 4);
            ptx::mbar_init(a_free(w), 1);
        }
        ptx::mbar_init(d_full, 1);
        ptx::mbar_init(d_free, kStoreWarps);
        ptx::mbar_init(peer_free, 1);
        ptx::mbar_init(done, 1);
        ptx::fence_mbar_init();
        words[1] = 0;
    }
    if (warp == kWarpMma) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sbase + kBars + 8 * kNumBars), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (warp == kWarpTma && lane < 2) ptx::prefetch_tmap(lane ? &tm_x : &tm_w);
    ptx::tc_fence_before();
    cluster_sync();   // both CTAs' barriers are ready for each other's arrivals
    ptx::tc_fence_after();
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const uint32_t tmem = words[0];
    const auto t_a = [&](int w) { return tmem + (uint32_t)(w * kACols); };
    const uint32_t t_d = tmem + kABufs * kACols;

    const auto ran_out = [&] {
        words[1] = 1;
        atomicOr(L.status, kStatusTimeout);
        return false;
    };
    const auto wait = [&](uint32_t bar_, uint32_t parity) -> bool { return ptx::mbar_wait_bounded(bar_, parity, kWaitNs) || ran_out(); };
    const auto wait_peer = [&](uint32_t bar_, uint32_t parity) -> bool { return wait_cluster(bar_, parity, kWaitNs) || ran_out(); };
    const auto lost = [&] { return words[1] != 0; };

    if (warp == kWarpMma) {
        // One CTA issues for both; the other one announces its operands, a stage at a
        // time, and that its sums have been read.
        constexpr uint32_t idesc = (1u << 4) | ((kTileRows >> 3) << 17) | ((2 * kOut >> 4) << 24);   // f16 operands
        const uint32_t lead = elect_one();
        const uint64_t d_b = ptx::smem_desc(sbase + kOpAt, 16, 1024, 2);
        int op = 0;
        uint32_t op_parity = 0;
        bool ok = true;
        for (int it = 0; it < mine && ok; ++it) {
            if (it > 0) {
                ok = wait(d_free, (it - 1) & 1) && (rank != 0 || wait_peer(peer_free, (it - 1) & 1));
                ok = __all_sync(~0u, ok);
                ptx::tc_fence_after();
                if (ok && rank != 0) {
                    ptx::tc_fence_before();
                    if (lane == 0) arrive_at(peer_free, 0);
                }
            }
            for (int i = 0; i < ns && ok; ++i) {
                const int g = it * ns + i, a = g % kABufs;
                ok = wait(a_ready(a), (g / kABufs) & 1) && wait(b_ready(op), op_parity) && (rank != 0 || wait_peer(peer(op), op_parity)) && !lost();
                ok = __all_sync(~0u, ok);
                if (!ok) break;
                ptx::tc_fence_after();
                if (rank == 0) {
                    const uint64_t b = d_b + (uint32_t)(op * kOp) / 16;
#pragma unroll
                    for (int x = 0; x < kStageK / 16; ++x)
                        mma_pair(lead, t_d, t_a(a) + 8 * x, b + (uint32_t)((x >> 2) * kRows * 8 + (x & 3) * 2), idesc, i > 0 || x > 0);
                    commit_pair(lead, a_free(a));
                    commit_pair(lead, b_free(op));
                } else {
                    ptx::tc_fence_before();
                    if (lane == 0) arrive_at(peer(op), 0);
                }
                if (++op == kOps) op = 0, op_parity ^= 1;
            }
            if (ok && rank == 0) commit_pair(lead, d_full);
        }
        __syncwarp();
        if (rank == 0) commit_pair(lead, done);   // all that was issued, however the loop ended
    } else if (warp == kWarpTma) {
        // ------------------------------------------------------- TMA
        if (lane == 0) {
            int count = 0;
            bool ok = true;
            for (int it = 0; it < mine && ok; ++it) {
                const Tile t = tile_of(it);
                for (int i = 0; i < ns; ++i) {
                    const int g = it * ns + i, slot = g % kStages;
                    ok = wait(raw_empty(slot), (g / kStages + 1) & 1) && !lost();
                    if (!ok) break;
                    const uint32_t at = sbase + slot * kRaw;
                    ptx::mbar_arrive_expect_tx(raw_full(slot), kRaw);
                    ptx::tma_load_2d(at, &tm_w, raw_full(slot), i * kStageK, t.n0);
                    ptx::tma_load_2d(at + kW, &tm_x, raw_full(slot), i * kStageK, t.m0 + rank * kRows);
                    ++count;
                }
            }
            // The copies in flight land before the CTA leaves, whoever gives up, and when.
            for (int x = max(0, count - kStages); x < count; ++x) ptx::mbar_wait_bounded(raw_full(x % kStages), (x / kStages) & 1, kWaitNs);
        }
    } else if (warp >= kWarpStore) {
        // ------------------------------------------------------- output
        // A thread has one output of half of a tile's rows.
        const int t = tid - kWarpStore * 32, row = t & 127, half = t >> 7;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        for (int it = 0; it < mine; ++it) {
            const Tile tile = tile_of(it);
            const int n = tile.n0 + row;
            float *const xs = reinterpret_cast<float *>(smem + kScales) + (it & 1) * kTileRows;
            xs[t] = tile.m0 + t < L.rows ? L.x_scale[tile.m0 + t] : 0.0f;
            const Channel channel(n < L.n ? L.w_scale[n] : 0.0f, n < L.n && L.bias ? L.bias[n] : 0.0f);
            const bool ok = wait(d_full, it & 1) && !lost();
            if (ptx::bar_red_or(1, kStoreWarps * 32, !ok)) break;   // (together, whatever ran out; and the scales are there)
            ptx::tc_fence_after();
            constexpr int kCols = kTileRows / 2, kPart = 16;
#pragma unroll 1
            for (int q = 0; q < kCols / kPart; ++q) {
                uint32_t v[kPart];
                const int col = half * kCols + q * kPart;
                __syncwarp();
                ptx::tmem_ld16(t_d + lanes + col, v);
                ptx::tmem_ld_wait();
                if (q == kCols / kPart - 1) {
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(d_free);
                }
                if (n < L.n) store_rows(L, tile.m0 + col, n, v, xs + col, channel);
            }
        }
    } else if (warp >= 8) {
        // ------------------------------------------------------- inputs
        constexpr int kLanes = 128, kPer = kRows * 8 / kLanes;
        const int turn = (warp - 8) >> 2, t = tid & 127, u = t & 7, row0 = t >> 3;
        for (int g = turn; g < total; g += kTurns) {
            const int slot = g % kStages, op = g % kOps;
            bool ok = wait(raw_full(slot), (g / kStages) & 1);
            if (!__all_sync(~0u, ok)) break;
            uint4 raw[kPer];
#pragma unroll
            for (int x = 0; x < kPer; ++x) {
                const int row = row0 + x * (kLanes / 8);
                raw[x] = *reinterpret_cast<const uint4 *>(smem + slot * kRaw + kW + row * 128 + ((u ^ (row & 7)) << 4));
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(raw_empty(slot));
            ok = wait(b_free(op), (g / kOps + 1) & 1) && !lost();
            if (!__all_sync(~0u, ok)) break;
            unsigned char *const to = smem + kOpAt + op * kOp + (u >> 2) * kRows * 128;
#pragma unroll
            for (int x = 0; x < kPer; ++x) widen_input(to, row0 + x * (kLanes / 8), u, raw[x]);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(b_ready(op));
        }
    } else {
        // ------------------------------------------------------- weights
        const int turn = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        for (int g = turn; g < total; g += kTurns) {
            const int slot = g % kStages, buf = g % kABufs;
            bool ok = wait(raw_full(slot), (g / kStages) & 1);
            if (!__all_sync(~0u, ok)) break;
            const unsigned char *const from = smem + slot * kRaw + row * 128;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t a[32];
                widen_weights(from, row, h, a);
                if (h == 0) {
                    ok = wait(a_free(buf), (g / kABufs + 1) & 1) && !lost();
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
    // Nothing leaves while an MMA reads shared or tensor memory.
    if (!ptx::mbar_wait_bounded(done, 0, kWaitNs)) atomicOr(L.status, kStatusTimeout);
    ptx::tc_fence_before();
    cluster_sync();
    if (warp == kWarpMma) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

}  // namespace

cbs_status launch_w8_pair(const W8Launch &L, cudaStream_t s) {
    alignas(64) CUtensorMap tw, tx;
    CBS_TRY(codes_map(&tw, L.w, L.k, L.n, kOut));
    CBS_TRY(codes_map(&tx, L.x, L.k, L.rows, kRows));
    Grid G;
    G.n_tiles = (L.n + 2 * kOut - 1) / (2 * kOut);
    G.m_tiles = (L.rows + kTileRows - 1) / kTileRows;
    if ((long long)G.n_tiles * G.m_tiles * ((L.k + kStageK - 1) / kStageK) >= 1ll << 30)   // (a pair numbers its stages)
        return fail(CBS_ERR_UNSUPPORTED, "%d rows of %d x %d", L.rows, L.n, L.k);
    G.pairs = std::max(1, std::min(G.n_tiles * G.m_tiles, current_device_sms() / 2));
    static ContextOfDevice set;
    CBS_TRY(cuda_check(set_max_dyn_smem_once(w8_pair_kernel, kSmem, set), "8-bit product shared memory"));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * G.pairs);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (launch_options() & CBS_LAUNCH_PDL) ? 2 : 1;
    return cuda_check(cudaLaunchKernelEx(&cfg, w8_pair_kernel, tw, tx, L, G), "8-bit product launch");
}

}  // namespace cbs
