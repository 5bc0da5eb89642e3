// k_attn_tc.cu -- attention of chunks over a paged cache on the tensor cores:
// one pass over keys and values with the running maximum and sum of a softmax,
//
//   S = Q K^T,   P = 2^(scale log2(e) S - m),   O += P V
//
// with S, P and O in tensor memory.  A CTA takes 256 (token, query head) rows of
// one key/value head as two halves of 128, and a range of keys in tiles of
// 128.  One thread issues the MMAs; while a half's four softmax warps (a thread
// a row) turn its scores into probabilities, the tensor cores work on the other
// half, and K and V tiles are shared by both.  P replaces S in place as bf16
// and is the A operand of the second product straight from tensor memory.
//
// bf16 cache: TMA brings each page's rows (a box a page and 64 dimensions);
// positions past the sequence's pages are boxes outside the tensor, which read
// as zeros.  int8 cache: four converter warps widen codes to bf16 (exact) and
// write the operands' swizzled rows; the scales of a tile's keys lie beside it.
//
// The maximum is raised only when a score passes it by 2^8, so one pass over
// the scores usually does: no second read, no rescaling of O.
#include <cuda.h>
#include <mutex>

#include "attn_common.cuh"
#include "tc_ptx.cuh"

namespace cbs {

namespace {

constexpr int kHalf = 128, kRows = kAttnChunkRows, kTile = kAttnChunkKeys;   // rows of a half and of a CTA; keys of a tile
static_assert(kRows == 2 * kHalf, "two halves");
constexpr int kStages = 2;
constexpr uint64_t kWaitNs = 2000000000ull;   // 2 s per wait

template <int D, bool I8>
struct Chunk {
    // Warps 0-3: MMA issue, TMA, and two that check values; 4-11: softmax of
    // the halves; 12-15 (int8): converters.
    static constexpr int kThreads = I8 ? 512 : 384;
    static constexpr int kPanel = kTile * 128;                 // 64 dimensions of 128 rows
    static constexpr int kOperand = (D / 64) * kPanel;         // one Q half, K tile or V tile
    static constexpr int kQ = 0, kK = 2 * kOperand, kV = kK + kStages * kOperand;
    static constexpr int kScale = kV + kStages * kOperand;     // [K, V][stage][128] floats
    static constexpr int kBars = kScale + (I8 ? 2 * kStages * kTile * 4 : 0);
    // q_full[2], k_full[2], k_empty[2], v_full[2], v_ready[2], v_empty[2],
    // s_full[2], p_ready[2], pv_done[2], drain; then the TMEM address and flags.
    static constexpr int kNumBars = 19;
    static constexpr int kSmem = kBars + kNumBars * 8 + 16 + 1024;   // 1 KB to align the operands
};

// D[tmem] (+)= A[tmem] B[smem desc], bf16 operands.
__device__ __forceinline__ void mma_f16_ta(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
        "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]),
        "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
        "r"(v[29]), "r"(v[30]), "r"(v[31]), "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The rows the halves of a CTA hold and the keys they see.
struct Span { int lo, hi, all_lo, all_hi; };   // seen by some row; seen by every row
__device__ __forceinline__ Span span_of(const AttnLaunch &L, const Rows &s, int r0, int r1) {
    const Seen a = s.seen(L, r0), b = s.seen(L, r1 - 1);
    return Span{a.lo, b.hi, b.lo, a.hi};
}

template <int D, bool I8>
__global__ void __launch_bounds__(Chunk<D, I8>::kThreads, 1)
attn_chunk_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const AttnLaunch L) {
    using C = Chunk<D, I8>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t sbase = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char *const sgen = smem_raw + (sbase - ptx::smem_u32(smem_raw));
    const CacheArgs &c = L.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    ptx::griddep_wait();
    const int b = blockIdx.z, head = blockIdx.y % c.kv_heads;
    const int rt = L.row_tiles - 1 - blockIdx.y / c.kv_heads;   // later rows see more keys: they start first
    const Rows rs = rows_of(L, b, head);
    const int r0 = rt * kRows;
    if (r0 >= rs.R) return;
    const int halves = r0 + kHalf < rs.R ? 2 : 1, r1 = min(rs.R, r0 + kRows);
    const Span all = span_of(L, rs, r0, r1);
    const int lo = all.lo & ~(kTile - 1);
    const int tiles = all.hi > all.lo ? (all.hi - lo + kTile - 1) / kTile : 0;
    const int per = (tiles + L.split - 1) / L.split;
    const int active = per ? (tiles + per - 1) / per : 1;
    const int sp = blockIdx.x;
    if (sp >= active) return;
    const int i0 = sp * per, n = min(tiles, i0 + per) - i0;   // this CTA's key tiles
    const int key0 = lo + i0 * kTile;

    const auto bar = [&](int i) { return sbase + C::kBars + 8u * i; };
    const auto q_full = [&](int h) { return bar(h); };
    const auto k_full = [&](int s) { return bar(2 + s); };
    const auto k_empty = [&](int s) { return bar(4 + s); };
    const auto v_full = [&](int s) { return bar(6 + s); };
    const auto v_ready = [&](int s) { return bar(8 + s); };
    const auto v_empty = [&](int s) { return bar(10 + s); };
    const auto s_full = [&](int h) { return bar(12 + h); };
    const auto p_ready = [&](int h) { return bar(14 + h); };
    const auto pv_done = [&](int h) { return bar(16 + h); };
    const uint32_t drain = bar(18);
    volatile uint32_t *const words = reinterpret_cast<volatile uint32_t *>(sgen + C::kBars + 8 * C::kNumBars);
    // words[0]: TMEM address; [1]: a wait ran out; [2]: a value is not finite; [3]: the join's flag

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(q_full(i), 4);
            ptx::mbar_init(k_full(i), I8 ? 4 : 1);
            ptx::mbar_init(k_empty(i), 1);
            ptx::mbar_init(v_full(i), I8 ? 4 : 1);
            ptx::mbar_init(v_ready(i), 2);
            ptx::mbar_init(v_empty(i), 1);
            ptx::mbar_init(s_full(i), 1);
            ptx::mbar_init(p_ready(i), 4);
            ptx::mbar_init(pv_done(i), 1);
        }
        ptx::mbar_init(drain, 1);
        ptx::fence_mbar_init();
        words[1] = words[2] = words[3] = 0;
    }
    if (warp == 1) {
        ptx::tmem_alloc(sbase + C::kBars + 8 * C::kNumBars, 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    ptx::griddep_launch_dependents();
    const uint32_t tmem = words[0];
    const auto t_s = [&](int h) { return tmem + 128u * h; };         // scores, then probabilities
    const auto t_o = [&](int h) { return tmem + 256u + 128u * h; };  // output

    // A wait of every role: false once any wait has run out.
    const auto wait = [&](uint32_t bar_, uint32_t parity) -> bool {
        if (ptx::mbar_wait_bounded(bar_, parity, kWaitNs)) return true;
        words[1] = 1;
        atomicOr(c.status, kStatusTimeout);
        return false;
    };
    const auto lost = [&] { return words[1] != 0; };

    if (warp == 0) {
        // ------------------------------------------------------- MMA issue
        if (lane == 0 && n > 0) {
            constexpr uint32_t idesc0 = (1u << 4) | (1u << 7) | (1u << 10) | ((kHalf >> 4) << 24);
            constexpr uint32_t idesc_s = idesc0 | ((kTile >> 3) << 17);
            constexpr uint32_t idesc_o = idesc0 | ((D >> 3) << 17) | (1u << 16);   // V: dimensions contiguous
            const auto scores = [&](int h, int st) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (k >> 2) * C::kPanel + (k & 3) * 32;
                    ptx::mma_f16(t_s(h), ptx::smem_desc(sbase + C::kQ + h * C::kOperand + off, 16, 1024, 2),
                                 ptx::smem_desc(sbase + C::kK + st * C::kOperand + off, 16, 1024, 2), idesc_s, k > 0);
                }
                ptx::mma_commit(s_full(h));
            };
            const auto output = [&](int h, int st, bool more) {
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    mma_f16_ta(t_o(h), t_s(h) + 8 * k,
                               ptx::smem_desc(sbase + C::kV + st * C::kOperand + k * 2048, C::kPanel, 1024, 2), idesc_o,
                               more || k > 0);
                ptx::mma_commit(pv_done(h));
            };
            bool ok = wait(k_full(0), 0);
            for (int h = 0; ok && h < halves; ++h) {
                ok = wait(q_full(h), 0);
                if (!ok) break;
                ptx::tc_fence_after();
                scores(h, 0);
            }
            if (ok) ptx::mma_commit(k_empty(0));
            for (int i = 0; ok && i < n && !lost(); ++i) {
                const int st = i & 1, nx = (i + 1) & 1;
                ok = wait(I8 ? v_full(st) : v_ready(st), (i >> 1) & 1);
                for (int h = 0; ok && h < halves; ++h) {
                    ok = wait(p_ready(h), i & 1);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    output(h, st, i > 0);
                    if (h == halves - 1) ptx::mma_commit(v_empty(st));
                    if (i + 1 < n) {
                        if (h == 0) ok = wait(k_full(nx), ((i + 1) >> 1) & 1);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        scores(h, nx);
                        if (h == halves - 1) ptx::mma_commit(k_empty(nx));
                    }
                }
            }
            ptx::mma_commit(drain);   // nothing leaves while an MMA reads shared memory
            if (!ptx::mbar_wait_bounded(drain, 0, kWaitNs)) atomicOr(c.status, kStatusTimeout);
        }
    } else if (warp == 1 && !I8) {
        // ------------------------------------------------------- TMA
        const int page = 1 << c.page_shift, box = min(page, kTile), boxes = kTile / box;
        const int none = c.num_pages * c.kv_heads << c.page_shift;   // a row past the pool: reads as zeros
        const int pages = (rs.len + page - 1) >> c.page_shift;
        int done = 0;
        for (int i = 0; i < n; ++i) {
            const int st = i & 1;
            int row = none;
            const int pos = key0 + i * kTile + lane * box;
            if (lane < boxes && (pos >> c.page_shift) < pages) {
                const int p = page_of(c, b, pos);
                if (p >= 0) row = ((p * c.kv_heads + head) << c.page_shift) + (pos & (page - 1));
            }
            bool ok = true;
#pragma unroll
            for (int side = 0; side < 2 && ok; ++side) {
                if (lane == 0) {
                    ok = wait(side ? v_empty(st) : k_empty(st), ((i >> 1) & 1) ^ 1) && !lost();
                    if (ok) ptx::mbar_arrive_expect_tx(side ? v_full(st) : k_full(st), C::kOperand);
                }
                ok = __shfl_sync(~0u, (int)ok, 0) != 0;
                if (ok && lane < boxes) {
                    const uint32_t dst = sbase + (side ? C::kV : C::kK) + st * C::kOperand + lane * box * 128;
#pragma unroll
                    for (int p = 0; p < D / 64; ++p)
                        ptx::tma_load_2d(dst + p * C::kPanel, side ? &tm_v : &tm_k, side ? v_full(st) : k_full(st), p * 64, row);
                }
                if (ok) ++done;
            }
            if (!ok) break;
        }
        if (lane == 0 && lost()) {   // the copies in flight land before the CTA leaves
            for (int x = max(0, done - 4); x < done; ++x) {
                const int i = x >> 1;
                ptx::mbar_wait_bounded((x & 1) ? v_full(i & 1) : k_full(i & 1), (i >> 1) & 1, kWaitNs);
            }
        }
    } else if (warp == 2 || (warp == 3 && !I8)) {
        // ------------------------- values some row must not see (bf16 cache)
        if (!I8) {
            for (int i = 0; i < n; ++i) {
                const int st = i & 1, pos = key0 + i * kTile;
                if (!wait(v_full(st), (i >> 1) & 1)) break;
                if (pos < all.all_lo || pos + kTile > all.all_hi) {
                    // Rows that nobody sees become zeros (a page's slots past the
                    // length may hold anything, and 0 x NaN is NaN); a value that is
                    // not finite among the others sends the CTA down the slow path.
                    unsigned char *v = sgen + C::kV + st * C::kOperand;
                    bool bad = false;
                    for (int u = (warp - 2) * 32 + lane; u < C::kOperand / 16; u += 64) {
                        const int key = pos + ((u >> 3) & (kTile - 1));
                        uint4 *p = reinterpret_cast<uint4 *>(v + u * 16);
                        if (key < all.lo || key >= all.hi) {
                            *p = make_uint4(0, 0, 0, 0);
                        } else {
                            const uint4 w = *p;
                            const auto odd = [](uint32_t x) { return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u; };
                            bad |= odd(w.x) || odd(w.y) || odd(w.z) || odd(w.w);
                        }
                    }
                    if (bad) words[2] = 1;
                    ptx::fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(v_ready(st));
            }
        }
    } else if (I8 && warp >= 12) {
        // ------------------------------------------------------- converters
        if constexpr (I8) {
            constexpr int kU = D / 16;                  // 16-code units of a row
            constexpr int kPer = kTile * kU / 128;      // units a thread
            const int ct = tid - 384;
            uint4 raw[2][kPer];
            float sc[2];
            // Tile i's codes and scales (zeros for positions nobody sees).
            const auto load = [&](int i, int side) {
                const int pos = key0 + i * kTile;
                const int8_t *pool = static_cast<const int8_t *>(side ? c.v : c.k);
#pragma unroll
                for (int x = 0; x < kPer; ++x) {
                    const int unit = x * 128 + ct, key = pos + unit / kU;
                    raw[side][x] = make_uint4(0, 0, 0, 0);
                    if (i < n && key >= all.lo && key < all.hi) {
                        const int p = page_of(c, b, key);
                        if (p >= 0) {
                            const size_t at = (((size_t)p * c.kv_heads + head) << c.page_shift) + (key & ((1 << c.page_shift) - 1));
                            raw[side][x] = __ldg(reinterpret_cast<const uint4 *>(pool + at * D + (unit % kU) * 16));
                        }
                    }
                }
                if (side) {
                    sc[0] = sc[1] = 0.0f;
                    const int key = pos + ct;
                    const int p = i < n && key >= all.lo && key < all.hi ? page_of(c, b, key) : -1;
                    if (p >= 0) {
                        const size_t at = (((size_t)p * c.kv_heads + head) << c.page_shift) + (key & ((1 << c.page_shift) - 1));
                        sc[0] = c.k_scale[at];
                        sc[1] = c.v_scale[at];
                    }
                }
            };
            const auto store = [&](int st, int side) {
#pragma unroll
                for (int x = 0; x < kPer; ++x) {
                    const int unit = x * 128 + ct, row = unit / kU, u = unit % kU;
                    const uint32_t w[4] = {raw[side][x].x, raw[side][x].y, raw[side][x].z, raw[side][x].w};
                    uint32_t o[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        o[2 * e] = frag::i8_pair(__byte_perm(w[e], 0, 0x4140));
                        o[2 * e + 1] = frag::i8_pair(__byte_perm(w[e], 0, 0x4342));
                    }
                    unsigned char *base = sgen + (side ? C::kV : C::kK) + st * C::kOperand + (u >> 2) * C::kPanel + row * 128;
                    const int ch = (u & 3) * 2;
                    *reinterpret_cast<uint4 *>(base + ((ch ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4 *>(base + (((ch + 1) ^ (row & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
                }
                if (side) {
                    // Both sides' scales go with the values: the softmax warps read
                    // them until the tile's last product, which is what v_empty waits for.
                    float *at = reinterpret_cast<float *>(sgen + C::kScale) + st * kTile + ct;
                    at[0] = sc[0] * L.scale_log2;
                    at[kStages * kTile] = sc[1];
                }
            };
            load(0, 0);
            load(0, 1);
            for (int i = 0; i < n; ++i) {
                const int st = i & 1;
                bool ok = true;
#pragma unroll
                for (int side = 0; side < 2; ++side) {
                    if (ok) ok = wait(side ? v_empty(st) : k_empty(st), ((i >> 1) & 1) ^ 1) && !lost();
                    ok = __all_sync(~0u, ok);
                    if (!ok) break;
                    store(st, side);
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(side ? v_full(st) : k_full(st));
                    load(i + 1, side);
                }
                if (!ok) break;
            }
        }
    }

    __syncwarp();

    float m = -INFINITY, l = 0.0f;
    const int h = (warp - 4) >> 2;                       // this softmax warp's half
    const int r = r0 + h * kHalf + (warp & 3) * 32 + lane;   // and its thread's row
    const uint32_t lanes = (uint32_t)(warp & 3) * 32u << 16;
    const bool softmax = warp >= 4 && warp < 12 && h < halves;
    if (softmax) {
        // ------------------------------------------------------- softmax
        {   // this thread's row of Q, in the operand's swizzled rows
            const int qr = r - r0 - h * kHalf;
            unsigned char *base = sgen + C::kQ + h * C::kOperand + qr * 128;
            const __nv_bfloat16 *p = rs.query(L, r, D);
#pragma unroll
            for (int u = 0; u < D / 8; ++u) {
                const uint4 w = r < rs.R ? __ldg(reinterpret_cast<const uint4 *>(p + u * 8)) : make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4 *>(base + (u >> 3) * C::kPanel + (((u & 7) ^ (qr & 7)) << 4)) = w;
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(q_full(h));
        }
        const int last = min(r1, r0 + (h + 1) * kHalf);
        const Span mine = span_of(L, rs, r0 + h * kHalf, last);
        const Seen z = rs.seen(L, min(r, rs.R - 1));
        for (int i = 0; i < n; ++i) {
            if (!__all_sync(~0u, wait(s_full(h), i & 1) && !lost())) break;
            ptx::tc_fence_after();
            const int pos = key0 + i * kTile;
            const bool partial = pos < mine.all_lo || pos + kTile > mine.all_hi;
            const float *ks = reinterpret_cast<const float *>(sgen + C::kScale) + (i & 1) * kTile;
            const float *vs = ks + kStages * kTile;
            const int first = z.lo - pos, end = z.hi - pos;   // columns [first, end) are seen
            if (I8 && !__all_sync(~0u, wait(v_full(i & 1), (i >> 1) & 1))) break;   // the tile's scales
            uint32_t p[kTile / 2];
            while (true) {
                const float ref = m == -INFINITY ? 0.0f : m;
                float top = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t v[32];
                    tmem_ld32(t_s(h) + lanes + 32 * q, v);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        float t = __uint_as_float(v[e]) * (I8 ? ks[32 * q + e] : L.scale_log2);
                        if (partial && (32 * q + e < first || 32 * q + e >= end)) t = -INFINITY;
                        top = fmaxf(top, t);
                        float x = frag::ex2(t - ref);
                        sum += x;
                        if (I8) x = partial && t == -INFINITY ? 0.0f : x * vs[32 * q + e];
                        v[e] = __float_as_uint(x);
                    }
                    // Rounded to bf16 for the second product: at most 2^-8 of
                    // each term, of either sign, as small as the output's own rounding.
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        p[16 * q + e] = frag::pack_bf16(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
                }
                const bool grow = top > m + kLazy;   // also from m = -inf
                if (!__any_sync(~0u, grow)) {
                    l += sum;
                    break;
                }
                // Raise the maxima and read the scores again.
                const float nm = fmaxf(m, top);
                const float fac = nm == -INFINITY ? 1.0f : frag::ex2(m - nm);
                if (i > 0) {
                    if (!__all_sync(~0u, wait(pv_done(h), (i - 1) & 1))) break;
                    ptx::tc_fence_after();
#pragma unroll
                    for (int q = 0; q < D / 32; ++q) {
                        uint32_t v[32];
                        tmem_ld32(t_o(h) + lanes + 32 * q, v);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * fac);
                        tmem_st32(t_o(h) + lanes + 32 * q, v);
                    }
                    tmem_st_wait();
                }
                l *= fac;
                m = nm;
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                uint32_t v[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = p[32 * q + e];
                tmem_st32(t_s(h) + lanes + 32 * q, v);
            }
            tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(p_ready(h));
        }
        if (n > 0) wait(pv_done(h), (n - 1) & 1);
        ptx::tc_fence_after();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();

    // ---------------------------------------------------------- output
    const int tile = (b * c.kv_heads + head) * L.row_tiles + rt;
    if (softmax && !lost()) {
        const size_t at = ((size_t)tile * L.split + sp) * kRows + (r - r0);
        if (!I8 && words[2]) {
            constexpr int kE = D / 32;
            for (int x = 0; x < 32; ++x) {
                const int row = r - lane + x;
                if (row >= rs.R) break;
                float acc[kE], mm, ll;
                slow_row<D>(L, rs, b, row, key0, key0 + n * kTile, lane, acc, mm, ll);
                if (active == 1) {
                    const Seen z = rs.seen(L, row);
                    const float inv = __fdiv_rn(1.0f, ll);
#pragma unroll
                    for (int e = 0; e < kE; ++e)
                        rs.out(L, row, D)[lane * kE + e] = __float2bfloat16_rn(z.hi > z.lo ? acc[e] * inv : 0.0f);
                } else {
#pragma unroll
                    for (int e = 0; e < kE; ++e) L.partial[(at - lane + x) * D + lane * kE + e] = acc[e];
                    if (lane == 0) L.stats[at - lane + x] = make_float2(mm, ll);
                }
            }
        } else {
            const Seen z = rs.seen(L, min(r, rs.R - 1));
            const float inv = __fdiv_rn(1.0f, l);
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
                uint32_t v[32];
                if (n > 0) {
                    tmem_ld32(t_o(h) + lanes + 32 * q, v);
                    ptx::tmem_ld_wait();
                }
                if (r < rs.R && active == 1) {
                    const bool any = z.hi > z.lo && n > 0;
                    uint4 *dst = reinterpret_cast<uint4 *>(rs.out(L, r, D) + 32 * q);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t w[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            w[y] = any ? frag::pack_bf16(__uint_as_float(v[8 * e + 2 * y]) * inv,
                                                         __uint_as_float(v[8 * e + 2 * y + 1]) * inv)
                                       : 0u;
                        dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else if (r < rs.R) {
                    uint4 *dst = reinterpret_cast<uint4 *>(L.partial + at * D + 32 * q);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dst[e] = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                    if (q == 0) L.stats[at] = make_float2(m, l);
                }
                __syncwarp();
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc(tmem, 512);
    if (active > 1) join_ranges<D, kRows, C::kThreads>(L, rs, tile, r0, active, tid, reinterpret_cast<int *>(const_cast<uint32_t *>(words + 3)));
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        cudaDriverEntryPointQueryResult q;
        void *p = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// The pool's rows [pages * heads * page][D], boxes of a page (at most a tile)
// by 64 dimensions, 128-byte swizzle.
cbs_status pool_map(CUtensorMap *tm, const CacheArgs &c, void *pool) {
    EncodeTiledFn fn = encode_tiled();
    if (!fn) return fail(CBS_ERR_CUDA, "cannot resolve cuTensorMapEncodeTiled from the driver");
    const cuuint64_t dims[2] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.num_pages * c.kv_heads << c.page_shift};
    const cuuint64_t strides[1] = {(cuuint64_t)c.head_dim * 2};
    const int page = 1 << c.page_shift;
    const cuuint32_t box[2] = {64u, (cuuint32_t)(page < kTile ? page : kTile)}, es[2] = {1u, 1u};
    const CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, pool, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(CBS_ERR_CUDA, "cuTensorMapEncodeTiled (cache) failed (%d)", (int)r);
    return CBS_OK;
}

template <int D, bool I8>
cbs_status launch_chunk(const AttnLaunch &L, cudaStream_t s) {
    alignas(64) CUtensorMap tk = {}, tv = {};
    if (!I8) {
        CBS_TRY(pool_map(&tk, L.c, L.c.k));
        CBS_TRY(pool_map(&tv, L.c, L.c.v));
    }
    using C = Chunk<D, I8>;
    auto kern = attn_chunk_kernel<D, I8>;
    CBS_TRY(cuda_check(set_max_dyn_smem(kern, C::kSmem), "attention shared memory"));
    const dim3 grid(L.split, L.c.kv_heads * L.row_tiles, L.c.batch);
    return cuda_check(launch_kernel(kern, grid, C::kThreads, C::kSmem, s, tk, tv, L), "attention launch");
}

}  // namespace

cbs_status launch_attn_chunk(const AttnLaunch &L, cudaStream_t s) {
    if (L.c.head_dim == 64) return L.c.int8 ? launch_chunk<64, true>(L, s) : launch_chunk<64, false>(L, s);
    return L.c.int8 ? launch_chunk<128, true>(L, s) : launch_chunk<128, false>(L, s);
}

}  // namespace cbs
