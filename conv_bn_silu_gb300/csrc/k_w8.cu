// k_w8.cu -- products of 8-bit integers with a scale for each token and each channel:
//
//   y[m, n] = act( xs[m] ws[n] sum_k x[m, k] w[n, k] + bias[n] )
//
// Y^T = W X^T on tcgen05: 128 outputs of a CTA are the lanes of tensor memory, its
// input rows the product's columns.  Codes are widened to f16, which holds them
// exactly, and sums of products are kept in 32 bits: whole numbers, exact below
// 2^24.  (The card's 8-bit integer tensor rate is far below its f16 one.)
//
// TMA brings the codes, one byte each.  Two warpgroups in turn widen a stage's
// weights and store them to tensor memory as the MMA's A operand; other warps widen
// the inputs into the swizzled rows of B.  Shared memory's bandwidth bounds it: a
// byte is written by TMA, read by a thread, and B's twofold written and read again.
// So the wide form pairs two CTAs (cta_group::2): each keeps the widened half of the
// 256 input rows, the pair's MMA reads both, and what a CTA moves for a product of
// 256 x 256 is half of what it would alone.
//
// For few rows the weights' bytes bound it.  Shares of k are then CTAs of a cluster,
// which add their sums in order through distributed shared memory.
#include <cuda_bf16.h>

#include "mma_frag.cuh"
#include "tc_ptx.cuh"
#include "tc_warp.cuh"
#include "tokens.cuh"

namespace cbs {

namespace {

constexpr int kOut = 128;                    // outputs of a CTA: tensor memory's lanes
constexpr int kStageK = 128;                 // codes along k in a stage: a row of 128 bytes
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s per wait
constexpr int kShareMost = 8;                // shares of k: CTAs of a cluster

// kN: input rows of a tile; kPair: CTAs that share it.
template <int kN, int kPair>
struct W8Tile {
    static constexpr int kRows = kN / kPair;                 // input rows a CTA widens
    static constexpr int kW = kOut * 128, kRaw = kW + kRows * 128;
    static constexpr int kOp = kRows * 256;                  // a stage of B: two panels of 64
    static constexpr int kStages = kN == 16 ? 5 : kN == 32 ? 4 : kN == 64 ? 3 : 4;
    static constexpr int kOps = kN <= 64 ? 2 : 3;
    static constexpr int kWiden = kRows >= 128 ? 8 : kRows / 16;   // warps that widen inputs
    static constexpr int kWarpMma = 8 + kWiden, kWarpTma = kWarpMma + 1, kThreads = (kWarpTma + 1) * 32;
    static constexpr int kOpAt = kStages * kRaw, kBars = kOpAt + kOps * kOp;
    // raw_full[], raw_empty[], b_ready[], b_free[], a_ready[2], a_free[2], done; TMEM address, flag
    static constexpr int kNumBars = 2 * kStages + 2 * kOps + 5;
    static constexpr int kSmem = kBars + kNumBars * 8 + 16;
    static constexpr int kACols = kStageK / 2, kTmem = 2 * kACols + kN <= 256 ? 256 : 512;
    static_assert(2 * kACols + kN <= 512 && kRaw % 1024 == 0 && kOp % 1024 == 0, "tensor memory; operands at multiples of 1 KB");
    static_assert(kSmem <= kMaxDynSmem, "shared memory");
    static_assert(kPair == 2 || kN * (kOut + 1) * 4 <= kBars, "a share's sums fit where the stages were");
};

__device__ __forceinline__ void arrive_at(uint32_t bar, uint32_t rank) {   // another CTA's barrier (or this one's)
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(bar), "r"(rank));
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(a) : "memory");
}
// As mbar_wait_bounded, for arrivals from both CTAs of a pair.
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
// The instructions whose form names the number of CTAs (one kernel uses one form).
template <int kPair>
struct Tc {
    static __device__ __forceinline__ void alloc(uint32_t at, uint32_t cols) {
        if constexpr (kPair == 1) {
            ptx::tmem_alloc(at, cols);
            ptx::tmem_relinquish();
        } else {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(at), "r"(cols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        }
    }
    static __device__ __forceinline__ void dealloc(uint32_t t, uint32_t cols) {
        if constexpr (kPair == 1) ptx::tmem_dealloc(t, cols);
        else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(t), "r"(cols) : "memory");
    }
    static __device__ __forceinline__ void mma(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
        if constexpr (kPair == 1) {
            mma_ts(lead, d, a, b, idesc, accumulate);
        } else {
            asm volatile(
                "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
                "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
                "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
                : "memory");
        }
    }
    // Arrives on `bar` of every CTA of the tile.
    static __device__ __forceinline__ void commit(uint32_t lead, uint32_t bar) {
        if constexpr (kPair == 1) {
            mma_commit(lead, bar);
        } else {
            asm volatile(
                "{\n.reg .pred q;\nsetp.ne.b32 q, %1, 0;\n"
                "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2;\n}\n" ::"r"(bar),
                "r"(lead), "h"((uint16_t)3)
                : "memory");
        }
    }
};

template <int kN, int kPair>
__global__ void __launch_bounds__(W8Tile<kN, kPair>::kThreads, W8Tile<kN, kPair>::kSmem <= 113 * 1024 ? 2 : 1)
w8_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, const W8Launch L, int split) {
    using C = W8Tile<kN, kPair>;
    using T = Tc<kPair>;
    extern __shared__ __align__(1024) unsigned char smem[];   // the only shared memory: starts at a multiple of 1 KB
    const uint32_t sbase = ptx::smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = kPair > 1 || split > 1 ? (int)cluster_rank() : 0;
    const int share = kPair > 1 ? 0 : rank;                  // of k
    const int n0 = (kPair > 1 ? blockIdx.x : blockIdx.x / split) * kOut, m0 = blockIdx.y * kN;
    const int stages = (L.k + kStageK - 1) / kStageK;
    const int st0 = (int)((long long)stages * share / split), ns = (int)((long long)stages * (share + 1) / split) - st0;
    const auto bar = [&](int i) { return sbase + C::kBars + 8u * i; };
    const auto raw_full = [&](int s) { return bar(s); };
    const auto raw_empty = [&](int s) { return bar(C::kStages + s); };
    const auto b_ready = [&](int s) { return bar(2 * C::kStages + s); };
    const auto b_free = [&](int s) { return bar(2 * C::kStages + C::kOps + s); };
    const auto a_ready = [&](int w) { return bar(2 * C::kStages + 2 * C::kOps + w); };
    const auto a_free = [&](int w) { return bar(2 * C::kStages + 2 * C::kOps + 2 + w); };
    const uint32_t done = bar(2 * C::kStages + 2 * C::kOps + 4);
    volatile uint32_t *const words = reinterpret_cast<volatile uint32_t *>(smem + C::kBars + 8 * C::kNumBars);
    // words[0]: TMEM address; [1]: a wait ran out

    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            ptx::mbar_init(raw_full(s), 1);
            ptx::mbar_init(raw_empty(s), 4 + C::kWiden);   // the warpgroup whose turn it is, and the inputs' warps
        }
        for (int s = 0; s < C::kOps; ++s) {
            ptx::mbar_init(b_ready(s), C::kWiden * kPair);
            ptx::mbar_init(b_free(s), 1);
        }
        for (int w = 0; w < 2; ++w) {
            ptx::mbar_init(a_ready(w), 4 * kPair);
            ptx::mbar_init(a_free(w), 1);
        }
        ptx::mbar_init(done, 1);
        ptx::fence_mbar_init();
        words[1] = 0;
    }
    if (warp == C::kWarpMma) T::alloc(sbase + C::kBars + 8 * C::kNumBars, C::kTmem);
    if (warp == C::kWarpTma && lane < 2) ptx::prefetch_tmap(lane ? &tm_x : &tm_w);
    ptx::tc_fence_before();
    if (kPair > 1) cluster_sync();   // both CTAs' barriers are ready for each other's arrivals
    else __syncthreads();
    ptx::tc_fence_after();
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const uint32_t tmem = words[0];
    const auto t_a = [&](int w) { return tmem + (uint32_t)(w * C::kACols); };
    const uint32_t t_d = tmem + 2 * C::kACols;

    const auto wait = [&](uint32_t bar_, uint32_t parity) -> bool {
        if (ptx::mbar_wait_bounded(bar_, parity, kWaitNs)) return true;
        words[1] = 1;
        atomicOr(L.status, kStatusTimeout);
        return false;
    };
    const auto wait_both = [&](uint32_t bar_, uint32_t parity) -> bool {
        if (kPair == 1) return wait(bar_, parity);
        if (wait_cluster(bar_, parity, kWaitNs)) return true;
        words[1] = 1;
        atomicOr(L.status, kStatusTimeout);
        return false;
    };
    const auto lost = [&] { return words[1] != 0; };
    const auto arrive = [&](uint32_t bar_) {   // at the CTA that issues
        if (kPair == 1) ptx::mbar_arrive(bar_);
        else arrive_at(bar_, 0);
    };

    if (warp == C::kWarpMma) {
        // ------------------------------------------------------- MMA issue
        if (kPair == 1 || rank == 0) {
            constexpr uint32_t idesc = (1u << 4) | ((kN >> 3) << 17) | ((kOut * kPair >> 4) << 24);   // f16 operands
            const uint32_t lead = elect_one();
            const uint64_t d_b = ptx::smem_desc(sbase + C::kOpAt, 16, 1024, 2);
            int op = 0;
            uint32_t op_parity = 0;
            for (int i = 0; i < ns; ++i) {
                bool ok = wait_both(a_ready(i & 1), (i >> 1) & 1) && wait_both(b_ready(op), op_parity) && !lost();
                if (!__all_sync(~0u, ok)) break;
                ptx::tc_fence_after();
                const uint64_t b = d_b + (uint32_t)(op * C::kOp) / 16;
#pragma unroll
                for (int x = 0; x < kStageK / 16; ++x)
                    T::mma(lead, t_d, t_a(i & 1) + 8 * x, b + (uint32_t)((x >> 2) * C::kRows * 8 + (x & 3) * 2), idesc, i > 0 || x > 0);
                T::commit(lead, a_free(i & 1));
                T::commit(lead, b_free(op));
                if (++op == C::kOps) op = 0, op_parity ^= 1;
            }
            __syncwarp();
            T::commit(lead, done);   // all that was issued, however the loop ended
        }
    } else if (warp == C::kWarpTma) {
        // ------------------------------------------------------- TMA
        if (lane == 0) {
            int slot = 0, count = 0;
            uint32_t parity = 1;
            const int row = m0 + (kPair > 1 ? rank * C::kRows : 0);
            for (int i = 0; i < ns; ++i) {
                if (!wait(raw_empty(slot), parity) || lost()) break;
                const uint32_t at = sbase + slot * C::kRaw;
                ptx::mbar_arrive_expect_tx(raw_full(slot), C::kRaw);
                ptx::tma_load_2d(at, &tm_w, raw_full(slot), (st0 + i) * kStageK, n0);
                ptx::tma_load_2d(at + C::kW, &tm_x, raw_full(slot), (st0 + i) * kStageK, row);
                ++count;
                if (++slot == C::kStages) slot = 0, parity ^= 1;
            }
            // The copies in flight land before the CTA leaves, whoever gives up, and when.
            for (int x = max(0, count - C::kStages); x < count; ++x)
                ptx::mbar_wait_bounded(raw_full(x % C::kStages), (x / C::kStages) & 1, kWaitNs);
        }
    } else if (warp >= 8) {
        // ------------------------------------------------------- inputs
        // Sixteen codes a unit, eight units a row.  Lanes of a row's second 64 write
        // their upper half first: eight lanes are then in eight different sixteen-byte
        // banks.
        constexpr int kLanes = C::kWiden * 32, kPer = C::kRows * 8 / kLanes;
        const int t = tid - 256, u = t & 7, row0 = t >> 3;
        const uint32_t second = u >> 2;
        int slot = 0, op = 0;
        uint32_t parity = 0, op_parity = 1;
        for (int i = 0; i < ns; ++i) {
            bool ok = wait(raw_full(slot), parity);
            if (!__all_sync(~0u, ok)) break;
            uint4 raw[kPer];
#pragma unroll
            for (int x = 0; x < kPer; ++x) {
                const int row = row0 + x * (kLanes / 8);
                raw[x] = *reinterpret_cast<const uint4 *>(smem + slot * C::kRaw + C::kW + row * 128 + ((u ^ (row & 7)) << 4));
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(raw_empty(slot));
            ok = wait_both(b_free(op), op_parity) && !lost();
            if (!__all_sync(~0u, ok)) break;
            unsigned char *const to = smem + C::kOpAt + op * C::kOp + (u >> 2) * C::kRows * 128;
#pragma unroll
            for (int x = 0; x < kPer; ++x) {
                const int row = row0 + x * (kLanes / 8);
                uint32_t o[8];
                frag::i8_halves(raw[x].x, o[0], o[1]);
                frag::i8_halves(raw[x].y, o[2], o[3]);
                frag::i8_halves(raw[x].z, o[4], o[5]);
                frag::i8_halves(raw[x].w, o[6], o[7]);
                const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
                const uint32_t at = row * 128 + ((((u & 3) * 2 + second) ^ (row & 7)) << 4);
                *reinterpret_cast<uint4 *>(to + at) = second ? hi : lo;
                *reinterpret_cast<uint4 *>(to + (at ^ 16)) = second ? lo : hi;
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive(b_ready(op));
            if (++slot == C::kStages) slot = 0, parity ^= 1;
            if (++op == C::kOps) op = 0, op_parity ^= 1;
        }
    } else {
        // ------------------------------------------------------- weights
        const int wg = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        for (int i = wg; i < ns; i += 2) {
            const int slot = i % C::kStages;
            bool ok = wait(raw_full(slot), (i / C::kStages) & 1);
            if (!__all_sync(~0u, ok)) break;
            const unsigned char *const from = smem + slot * C::kRaw + row * 128;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t a[32];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(from + (((4 * h + q) ^ (row & 7)) << 4));
                    frag::i8_halves(w.x, a[8 * q], a[8 * q + 1]);
                    frag::i8_halves(w.y, a[8 * q + 2], a[8 * q + 3]);
                    frag::i8_halves(w.z, a[8 * q + 4], a[8 * q + 5]);
                    frag::i8_halves(w.w, a[8 * q + 6], a[8 * q + 7]);
                }
                if (h == 0 && i >= 2) {
                    ok = wait_both(a_free(wg), ((i >> 1) - 1) & 1) && !lost();
                    if (!__all_sync(~0u, ok)) break;
                    ptx::tc_fence_after();
                }
                tmem_st32(t_a(wg) + lanes + 32 * h, a);
            }
            if (!__all_sync(~0u, ok)) break;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(raw_empty(slot));
            tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive(a_ready(wg));
        }
    }
    __syncwarp();
    // Nothing goes on while an MMA reads shared or tensor memory.
    if (!(kPair == 1 ? ptx::mbar_wait_bounded(done, 0, kWaitNs) : wait_cluster(done, 0, kWaitNs)))
        atomicOr(L.status, kStatusTimeout);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();

    // ------------------------------------------------------------ output
    if (warp < 8) {
        // A thread has one output of half the input rows.
        const int wg = warp >> 2, row = tid & 127, n = n0 + row;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const float ws = n < L.n ? L.w_scale[n] : 0.0f, bias = n < L.n && L.bias ? L.bias[n] : 0.0f;
        constexpr int kCols = kN / 2, kPart = kCols < 16 ? 8 : 16;
        float *const sum = reinterpret_cast<float *>(smem);   // [input row][output] of this share
#pragma unroll 1
        for (int q = 0; q < kCols / kPart; ++q) {
            uint32_t v[kPart];
            const int col = wg * kCols + q * kPart;
            if (ns > 0) {
                if constexpr (kPart == 8) ptx::tmem_ld8(t_d + lanes + col, v);
                else ptx::tmem_ld16(t_d + lanes + col, v);
                ptx::tmem_ld_wait();
            } else {
#pragma unroll
                for (int e = 0; e < kPart; ++e) v[e] = 0;
            }
#pragma unroll
            for (int e = 0; e < kPart; ++e) {
                const int m = m0 + col + e;
                if (kPair == 1 && split > 1) {
                    sum[(col + e) * (kOut + 1) + row] = __uint_as_float(v[e]);
                } else if (m < L.rows && n < L.n) {
                    float y = __uint_as_float(v[e]) * (L.x_scale[m] * ws) + bias;
                    if (L.act == CBS_ACT_SILU) y = silu(y);
                    const size_t at = (size_t)m * L.n + n;
                    if (L.out_bf16) static_cast<__nv_bfloat16 *>(L.y)[at] = __float2bfloat16_rn(y);
                    else static_cast<float *>(L.y)[at] = y;
                }
            }
        }
    }
    ptx::tc_fence_before();
    if (kPair > 1 || split > 1) cluster_sync();
    else __syncthreads();
    if (warp == C::kWarpMma) T::dealloc(tmem, C::kTmem);
    if (kPair > 1 || split == 1) return;
    const int rows = min(kN, L.rows - m0);
    for (int i = tid + share * C::kThreads; i < kOut * rows; i += C::kThreads * split) {
        const int m = i / kOut, nn = i % kOut, n = n0 + nn;
        if (n >= L.n) continue;
        float y = 0.0f;
        for (int p = 0; p < split; ++p) y += ld_cluster1(sbase + (m * (kOut + 1) + nn) * 4, p);
        y = y * (L.x_scale[m0 + m] * L.w_scale[n]) + (L.bias ? L.bias[n] : 0.0f);
        if (L.act == CBS_ACT_SILU) y = silu(y);
        const size_t at = (size_t)(m0 + m) * L.n + n;
        if (L.out_bf16) static_cast<__nv_bfloat16 *>(L.y)[at] = __float2bfloat16_rn(y);
        else static_cast<float *>(L.y)[at] = y;
    }
    cluster_sync();   // nobody's sums go while another CTA reads them
}

template <int kN, int kPair>
cbs_status launch_w8_one(const W8Launch &L, cudaStream_t s) {
    using C = W8Tile<kN, kPair>;
    EncodeTiledFn fn = encode_tiled();
    if (!fn) return fail(CBS_ERR_CUDA, "cannot resolve cuTensorMapEncodeTiled from the driver");
    alignas(64) CUtensorMap tw, tx;
    const auto map = [&](CUtensorMap *tm, const void *p, int rows, int box_rows) {
        const cuuint64_t dims[2] = {(cuuint64_t)L.k, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)L.k};
        const cuuint32_t box[2] = {(cuuint32_t)kStageK, (cuuint32_t)box_rows}, es[2] = {1u, 1u};
        return fn(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = map(&tw, L.w, L.n, kOut);
    if (r != CUDA_SUCCESS) return fail(CBS_ERR_CUDA, "cuTensorMapEncodeTiled (weights) failed (%d)", (int)r);
    r = map(&tx, L.x, L.rows, C::kRows);
    if (r != CUDA_SUCCESS) return fail(CBS_ERR_CUDA, "cuTensorMapEncodeTiled (inputs) failed (%d)", (int)r);
    const int tiles = (L.n + kOut * kPair - 1) / (kOut * kPair), stages = (L.k + kStageK - 1) / kStageK;
    const int row_tiles = (L.rows + kN - 1) / kN, sms = current_device_sms();
    // Shares of k until every SM has a CTA.
    int split = 1;
    if (kPair == 1)
        while (split < kShareMost && split * 4 <= stages && tiles * row_tiles * split < sms) split *= 2;
    auto kern = w8_kernel<kN, kPair>;
    static ContextOfDevice set;
    cudaError_t e = set_max_dyn_smem_once(kern, C::kSmem, set);
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(tiles * split * kPair, row_tiles);
        cfg.blockDim = dim3(C::kThreads);
        cfg.dynamicSmemBytes = C::kSmem;
        cfg.stream = s;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = split * kPair;
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

cbs_status launch_w8(const W8Launch &L, cudaStream_t s) {
    if (L.rows <= 16) return launch_w8_one<16, 1>(L, s);
    if (L.rows <= 32) return launch_w8_one<32, 1>(L, s);
    if (L.rows <= 64) return launch_w8_one<64, 1>(L, s);
    if (L.rows <= 128) return launch_w8_one<128, 1>(L, s);
    return launch_w8_one<256, 2>(L, s);
}

cudaError_t launch_quantize_w8(const float *w, int n, int k, int8_t *codes, float *scales, cudaStream_t s) {
    const int cap = current_device_sms() * 16, grid = (n + 7) / 8;
    return launch_kernel(quantize_w8_kernel, grid < cap ? grid : cap, 256, 0, s, w, n, k, codes, scales);
}

}  // namespace cbs
