// k_attn_chunk.cuh -- attention of chunks over a paged cache on the tensor cores:
// one pass over keys and values with the running maximum and sum of a softmax,
//
//   S = Q K^T,   P = 2^(scale log2(e) S - m),   O += P V
//
// with S, P and O in tensor memory.  A CTA takes 256 (token, query head) rows of
// one key/value head as two halves of 128, and a range of keys in tiles of
// 128.  One warp issues the MMAs; while a half's eight softmax warps (two threads
// a row) turn its scores into probabilities, the tensor cores work on the other
// half, and K and V tiles are shared by both.  P replaces S in place as bf16
// and is the A operand of the second product straight from tensor memory.
//
// bf16 cache: TMA brings each page's rows (a box a page and 64 dimensions);
// positions past the sequence's pages are boxes outside the tensor, which read
// as zeros.  int8 cache: bulk copies bring the codes, four converter warps widen
// them to bf16 (exact) and write the operands' swizzled rows; the scales of a
// tile's keys lie beside it.
//
// The maximum is raised only when a score passes it by 2^8, so one pass over
// the scores usually does: no second read, no rescaling of O.
//
// Ranges of keys are the CTAs of a cluster; each joins its part of the rows from
// the others' shared memory, in the ranges' order.
//
// The softmax bounds it: a tile of 128 keys takes 1.6 us (head dimension 128; 1.4
// at 64), the products alone 1.1 us, a CTA's start and end 7 to 10 us.  2048 tokens
// of 32 heads over 32768 keys of 8 key heads: 797 us, 1.34 PFLOP/s.  8 bits: 2.7 us
// a tile alone and 3.5 with every SM busy (2.2 and 2.7 at 64), where widening the
// codes takes as many issue slots again.
//
// The modes (AttnMode) differ in what the join stores, which they all go through;
// a weighed call also sums up the probabilities before they are rounded.
#pragma once

#include <cuda.h>

#include "attn_common.cuh"
#include "tc_ptx.cuh"
#include "tc_warp.cuh"

namespace cbs {

namespace {

constexpr int kHalf = 128, kRows = kAttnChunkRows, kTile = kAttnChunkKeys;   // rows of a half and of a CTA; keys of a tile
static_assert(kRows == 2 * kHalf, "two halves");
constexpr int kMostRanges = kAttnChunkSplitMost;
constexpr int kCols = kTile / 2;              // keys of a tile a softmax thread takes
constexpr uint64_t kWaitNs = 2000000000ull;   // 2 s per wait

template <int D, bool I8>
struct Chunk {
    // Warp 0: MMA issue; 1: loads; 2, 3: check values (bf16), or converters (int8,
    // with 20 and 21); 4-19: softmax, eight warps a half (two
    // threads a row, 64 keys of the tile each).
    static constexpr int kThreads = I8 ? 704 : 640;
    static constexpr int kConverters = 4;
    static constexpr int kPanel = kTile * 128;                 // 64 dimensions of 128 rows
    static constexpr int kOperand = (D / 64) * kPanel;         // one Q half, K tile or V tile
    // A ring of K and V tiles in turn (K of tile i is its item 2 i, V 2 i + 1): as
    // deep as shared memory allows, since a tile takes about a microsecond to
    // arrive and as long to use.
    static constexpr int kSlots = D == 64 ? 8 : I8 ? 4 : 5;
    static constexpr int kQ = 0, kRing = 2 * kOperand;
    // int8: codes on their way, 64 keys' rows of K or V a piece, four pieces a tile.
    static constexpr int kPieceKeys = kTile / 2, kPiece = kPieceKeys * D, kPieces = I8 ? (D == 64 ? 8 : 3) : 0;
    static constexpr int kRaw = kRing + kSlots * kOperand;
    // int8: the scales of four tiles' keys, [K, V][tile % 4][128] floats.  Tile i's
    // are written once its V tile's slot is free, when V of tile i - kSlots / 2 (at
    // least i - 4) has been used, and so have that tile's scales.
    static constexpr int kScaleTiles = 4;
    static constexpr int kScale = kRaw + kPieces * kPiece;
    static constexpr int kShare = kScale + (I8 ? 2 * kScaleTiles * kTile * 4 : 0);   // a row's threads exchange here
    static constexpr int kBars = kShare + 2 * kRows * 4;
    // V tiles checked but not yet waited for: while the MMAs of tile i wait, items
    // up to 2 i + kSlots have had their slots, V of tile i + (kSlots - 1) / 2 the last.
    static constexpr int kReady = 4;
    static_assert((kSlots - 1) / 2 < kReady, "a check's turn comes after the last one's was seen");
    // q_full[2], s_full[2], p_ready[2], pv_done[2], drain, ready[], full[K, V][], empty[], raw_full[], raw_empty[];
    // then the TMEM address and flags.
    // The join's places in Q's: each row's maximum and sum, then the ranges' factors.
    // (kAttnWeighed: behind them a range's sums before rounding.)
    static constexpr int kJoinStats = 0, kJoinFacs = kRows * 8, kJoinSums = kJoinFacs + (kMostRanges + 1) * kRows * 4;
    static_assert(kJoinSums + kRows * 4 <= 2 * kOperand && 2 * kHalf * D * 4 <= kSlots * kOperand, "join");
    static constexpr int kNumBars = 9 + kReady + 3 * kSlots + 2 * kPieces;
    static constexpr int kSmem = kBars + kNumBars * 8 + 16;
    static_assert(kSmem <= kMaxDynSmem, "ring");
    static_assert(!I8 || (kSlots % 2 == 0 && kSlots / 2 <= kScaleTiles), "scales are free when V's slot is");
};

// An item's slot in the ring, and the parity of its turn there.
template <int kSlots>
struct Turn {
    int slot;
    uint32_t parity;
    __device__ __forceinline__ explicit Turn(int item) : slot(item % kSlots), parity((item / kSlots) & 1) {}
};

// The rows the halves of a CTA hold and the keys they see.
struct Span { int lo, hi, all_lo, all_hi; };   // seen by some row; seen by every row
__device__ __forceinline__ Span span_of(const AttnLaunch &L, const Rows &s, int r0, int r1) {
    const Seen a = s.seen(L, r0), b = s.seen(L, r1 - 1);
    return Span{a.lo, b.hi, b.lo, a.hi};
}

// A thread's pass over its kCols of a row's scores: t = s * scale - ref (ks: a scale a key,
// for 8-bit keys), p = 2^t (times vs, for 8-bit values) as bf16 pairs, the
// largest t and, in 8 bits, the sum of 2^t (p has the value's scale in it; in
// bf16 the sum is of p as rounded, below).  MASK: columns outside [first, end) are
// not seen.  Rounding p to bf16 moves each term by at most 2^-8 of itself, either
// way, as the output's own rounding does.
template <bool I8, bool MASK, bool EXACT>
__device__ __forceinline__ void tile_pass(uint32_t taddr, float scale, float ref, const float *ks, const float *vs, int first,
                                          int end, uint32_t (&p)[kCols / 2], float &top, float &sum) {
    constexpr int kPart = I8 ? 8 : 16;   // columns at a time: of more, registers spilled
    const F2 scale2 = pair(scale, scale), ref2 = pair(-ref, -ref);
    F2 acc[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
    float tops[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int q = 0; q < kCols / kPart; ++q) {
        uint32_t v[kPart];
        if constexpr (I8) ptx::tmem_ld8(taddr + kPart * q, v);
        else ptx::tmem_ld16(taddr + kPart * q, v);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < kPart; e += 4) {
            F2 k2[2] = {scale2, scale2}, w2[2];
            if constexpr (I8) {
                const float4 k4 = *reinterpret_cast<const float4 *>(ks + kPart * q + e), v4 = *reinterpret_cast<const float4 *>(vs + kPart * q + e);
                k2[0] = pair(k4.x, k4.y); k2[1] = pair(k4.z, k4.w);
                w2[0] = pair(v4.x, v4.y); w2[1] = pair(v4.z, v4.w);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float2 t = split(fma2(pair(__uint_as_float(v[e + 2 * x]), __uint_as_float(v[e + 2 * x + 1])), k2[x], ref2));
                if constexpr (MASK) {
                    const int col = kPart * q + e + 2 * x;
                    if (col < first || col >= end) t.x = -INFINITY;
                    if (col + 1 < first || col + 1 >= end) t.y = -INFINITY;
                }
                tops[x] = fmaxf(tops[x], fmaxf(t.x, t.y));
                F2 pr = pair(frag::ex2(t.x), frag::ex2(t.y));
                if constexpr (I8 || EXACT) acc[x] = add2(acc[x], pr);
                if constexpr (I8) pr = mul2(pr, w2[x]);
                float2 y = split(pr);
                if constexpr (I8 && MASK) {   // a hidden key's scale may be anything
                    if (t.x == -INFINITY) y.x = 0.0f;
                    if (t.y == -INFINITY) y.y = 0.0f;
                }
                p[kPart / 2 * q + (e >> 1) + x] = frag::pack_bf16(y.x, y.y);
            }
        }
    }
    top = fmaxf(tops[0], tops[1]);
    const float2 a = split(add2(acc[0], acc[1]));
    sum = a.x + a.y;   // (bf16: none, unless EXACT)
}

// The sum of a thread's probabilities as they were rounded, taken while their
// store to tensor memory is under way (16 maps of 20x20 23.3 us, in the pass
// itself 24.0; the chunk of 2048 797 and 809).
__device__ __forceinline__ float sum_rounded(const uint32_t (&p)[kCols / 2]) {
    float sums[4] = {};
#pragma unroll
    for (int e = 0; e < kCols / 2; ++e) {
        sums[2 * (e & 1)] = frag::add_bf16(sums[2 * (e & 1)], p[e]);
        sums[2 * (e & 1) + 1] = frag::add_bf16(sums[2 * (e & 1) + 1], p[e] >> 16);
    }
    return (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// The largest of a thread's scores, in base 2.
template <bool I8, bool MASK>
__device__ __forceinline__ float tile_top(uint32_t taddr, float scale, const float *ks, int first, int end) {
    float tops[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int q = 0; q < kCols / 16; ++q) {
        uint32_t v[16];
        ptx::tmem_ld16(taddr + 16 * q, v);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            float t = __uint_as_float(v[e]) * (I8 ? ks[16 * q + e] : scale);
            if (MASK && (16 * q + e < first || 16 * q + e >= end)) t = -INFINITY;
            tops[e & 1] = fmaxf(tops[e & 1], t);
        }
    }
    return fmaxf(tops[0], tops[1]);
}

template <int D, bool I8, int MODE>
__global__ void __launch_bounds__(Chunk<D, I8>::kThreads, 1)
attn_chunk_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const AttnLaunch L) {
    using C = Chunk<D, I8>;
    using T = Turn<C::kSlots>;
    extern __shared__ __align__(1024) unsigned char sgen[];   // the only shared memory: it starts at a multiple of 1 KB
    const uint32_t sbase = ptx::smem_u32(sgen);
    const CacheArgs &c = L.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // Before the kernel ahead has ended: barriers, tensor memory, the tensor maps.
    if (!I8 && warp == 1 && lane < 2) ptx::prefetch_tmap(lane ? &tm_v : &tm_k);
    const auto bar = [&](int i) { return sbase + C::kBars + 8u * i; };
    const auto q_full = [&](int h) { return bar(h); };
    const auto s_full = [&](int h) { return bar(2 + h); };
    const auto p_ready = [&](int h) { return bar(4 + h); };
    const auto pv_done = [&](int h) { return bar(6 + h); };
    const uint32_t drain = bar(8);
    // bf16: tile i's V has been checked.  Its own turns, by tile: a slot of the
    // ring holds K and V alternately, so the ring's parities do not count V's.
    const auto ready = [&](int i) { return bar(9 + i % C::kReady); };
    // Tile i's K or V has arrived: barriers of each side's own, so that whoever
    // waits for one side's tiles in order sees every turn of its barriers (loads
    // end out of order, and of a slot's turns K's or V's alone are every other).
    const auto full = [&](int i, int side) { return bar(9 + C::kReady + side * C::kSlots + i % C::kSlots); };
    const auto full_turn = [&](int i) { return (uint32_t)(i / C::kSlots) & 1u; };
    const auto empty = [&](int s) { return bar(9 + C::kReady + 2 * C::kSlots + s); };   // a slot's item has been used
    const auto raw_full = [&](int s) { return bar(9 + C::kReady + 3 * C::kSlots + s); };   // int8: a piece's codes
    const auto raw_empty = [&](int s) { return bar(9 + C::kReady + 3 * C::kSlots + C::kPieces + s); };
    const auto slot_at = [&](int s) { return C::kRing + s * C::kOperand; };
    volatile uint32_t *const words = reinterpret_cast<volatile uint32_t *>(sgen + C::kBars + 8 * C::kNumBars);
    // words[0]: TMEM address; [1]: a wait ran out; [2]: the rows go the slow path (a
    // value that some must not see is not finite, or a row's scores are far from zero)

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(q_full(i), 8);
            ptx::mbar_init(s_full(i), 1);
            ptx::mbar_init(p_ready(i), 8);
            ptx::mbar_init(pv_done(i), 1);
        }
        for (int i = 0; i < C::kReady; ++i) ptx::mbar_init(ready(i), 2);
        for (int s = 0; s < C::kSlots; ++s) {
            ptx::mbar_init(full(s, 0), I8 ? C::kConverters : 1);
            ptx::mbar_init(full(s, 1), I8 ? C::kConverters : 1);
            ptx::mbar_init(empty(s), 1);
        }
        for (int s = 0; s < C::kPieces; ++s) {
            ptx::mbar_init(raw_full(s), 1);
            ptx::mbar_init(raw_empty(s), C::kConverters);
        }
        ptx::mbar_init(drain, 1);
        ptx::fence_mbar_init();
        words[1] = words[2] = 0;
    }
    if (warp == 1) {
        ptx::tmem_alloc(sbase + C::kBars + 8 * C::kNumBars, 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    begin_attention<MODE>();
    ptx::griddep_launch_dependents();
    const int b = blockIdx.z, head = blockIdx.y % c.kv_heads;
    const int rt = L.row_tiles - 1 - blockIdx.y / c.kv_heads;   // later rows see more keys: they start first
    const Rows rs = rows_of<MODE>(L, b, head, D);
    const int r0 = rt * kRows;
    // CTAs of one cluster meet twice at the end, and none leaves before: whatever
    // is read there is still some CTA's, even if the lengths change meanwhile.
    const auto leave = [&] {
        end_attention<MODE>();
        if (warp == 1) ptx::tmem_dealloc(words[0], 512);
        if (L.split == 1) return;
        cluster_sync();
        cluster_sync();
    };
    if (r0 >= rs.R) return leave();
    const int halves = r0 + kHalf < rs.R ? 2 : 1, r1 = min(rs.R, r0 + kRows);
    const Span all = span_of(L, rs, r0, r1);
    const int lo = all.lo & ~(kTile - 1);
    const int tiles = all.hi > all.lo ? (all.hi - lo + kTile - 1) / kTile : 0;
    const int per = (tiles + L.split - 1) / L.split;
    const int active = per ? (tiles + per - 1) / per : 1;
    const int sp = blockIdx.x;
    if (sp >= active) return leave();
    const int i0 = sp * per, n = min(tiles, i0 + per) - i0;   // this CTA's key tiles
    const int key0 = lo + i0 * kTile;

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
        if (n > 0) {
            constexpr uint32_t idesc0 = (1u << 4) | (1u << 7) | (1u << 10) | ((kHalf >> 4) << 24);
            constexpr uint32_t idesc_s = idesc0 | ((kTile >> 3) << 17);
            constexpr uint32_t idesc_o = idesc0 | ((D >> 3) << 17) | (1u << 16);   // V: dimensions contiguous
            const uint32_t lead = elect_one();
            // Operand descriptors: everything but the slot and the step along k.
            const uint64_t d_q = ptx::smem_desc(sbase + C::kQ, 16, 1024, 2), d_k = ptx::smem_desc(sbase + C::kRing, 16, 1024, 2);
            const uint64_t d_v = ptx::smem_desc(sbase + C::kRing, C::kPanel, 1024, 2);
            constexpr uint32_t kStep = C::kOperand >> 4;   // descriptors count 16 bytes
            const auto scores = [&](int h, int slot) {
                const uint64_t q = d_q + h * kStep, k = d_k + (uint32_t)slot * kStep;
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    constexpr uint32_t kPanelStep = C::kPanel >> 4;
                    const uint32_t off = (x >> 2) * kPanelStep + (x & 3) * 2;
                    mma_ss(lead, t_s(h), q + off, k + off, idesc_s, x > 0);
                }
                mma_commit(lead, s_full(h));
            };
            const auto output = [&](int h, int slot, bool more) {
                const uint64_t v = d_v + (uint32_t)slot * kStep;
#pragma unroll
                for (int x = 0; x < kTile / 16; ++x) mma_ts(lead, t_o(h), t_s(h) + 8 * x, v + 128u * x, idesc_o, more || x > 0);
                mma_commit(lead, pv_done(h));
            };
            bool ok = wait(full(0, 0), 0);
            for (int h = 0; ok && h < halves; ++h) {
                ok = wait(q_full(h), 0);
                if (!ok) break;
                ptx::tc_fence_after();
                scores(h, 0);
            }
            if (ok) mma_commit(lead, empty(0));
            int v_slot = 1, k_slot = 2 % C::kSlots;   // items 2 i + 1 and 2 i + 2
            const auto advance = [](int &slot) {
                slot += 2;
                if (slot >= C::kSlots) slot -= C::kSlots;
            };
            for (int i = 0; ok && i < n; ++i) {
                ok = (I8 ? wait(full(i, 1), full_turn(i)) : wait(ready(i), (i / C::kReady) & 1)) && !lost();
                ok = __all_sync(~0u, ok);
                for (int h = 0; ok && h < halves; ++h) {
                    ok = wait(p_ready(h), i & 1);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    output(h, v_slot, i > 0);
                    if (h == halves - 1) mma_commit(lead, empty(v_slot));
                    if (i + 1 < n) {
                        if (h == 0) ok = wait(full(i + 1, 0), full_turn(i + 1));
                        if (!ok) break;
                        ptx::tc_fence_after();
                        scores(h, k_slot);
                        if (h == halves - 1) mma_commit(lead, empty(k_slot));
                    }
                }
                advance(v_slot);
                advance(k_slot);
            }
            __syncwarp();
            mma_commit(lead, drain);   // nothing leaves while an MMA reads shared memory
            if (!ptx::mbar_wait_bounded(drain, 0, kWaitNs)) atomicOr(c.status, kStatusTimeout);
        }
    } else if (warp == 1 && !I8) {
        // ------------------------------------------------------- TMA
        const int page = 1 << c.page_shift, box = min(page, kTile), boxes = kTile / box;
        const int none = c.num_pages * c.kv_heads << c.page_shift;   // a row past the pool: reads as zeros
        // Lane x < boxes: the page of tile i's position x * box as loaded (two
        // tiles ahead), and from it the pool's row.
        const auto needed = [&](int i) {   // (pages that no row sees may be gone)
            const int pos = key0 + i * kTile + lane * box;
            return i < n && lane < boxes && pos + box > all.lo && pos < all.hi;
        };
        const auto page_entry = [&](int i) -> int {
            return needed(i) ? __ldg(c.page_table + (size_t)b * c.max_pages + ((key0 + i * kTile + lane * box) >> c.page_shift)) : 0;
        };
        int entry = page_entry(0), entry_next = page_entry(1), done = 0;
        for (int i = 0; i < n; ++i) {
            int row = none;
            if (needed(i)) {
                if ((unsigned)entry < (unsigned)c.num_pages)
                    row = ((entry * c.kv_heads + head) << c.page_shift) + ((key0 + i * kTile + lane * box) & (page - 1));
                else
                    atomicOr(c.status, kStatusBadIndex);
            }
            entry = entry_next;
            entry_next = page_entry(i + 2);
            bool ok = true;
#pragma unroll
            for (int side = 0; side < 2 && ok; ++side) {
                const T x(2 * i + side);
                if (lane == 0) {
                    ok = wait(empty(x.slot), x.parity ^ 1) && !lost();
                    if (ok) ptx::mbar_arrive_expect_tx(full(i, side), C::kOperand);
                }
                ok = __shfl_sync(~0u, (int)ok, 0) != 0;
                if (ok && lane < boxes) {
                    const uint32_t dst = sbase + slot_at(x.slot) + lane * box * 128;
#pragma unroll
                    for (int p = 0; p < D / 64; ++p)
                        ptx::tma_load_2d(dst + p * C::kPanel, side ? &tm_v : &tm_k, full(i, side), p * 64, row);
                }
                if (ok) ++done;
            }
            if (!ok) break;
        }
        // The copies in flight land before the CTA leaves, whoever gives up.
        if (lane == 0)
            for (int x = max(0, done - C::kSlots); x < done; ++x) wait(full(x >> 1, x & 1), full_turn(x >> 1));
    } else if (!I8 && warp < 4) {
        // ------------------------- values some row must not see (bf16 cache)
        for (int i = 0; i < n; ++i) {
            const T x(2 * i + 1);
            const int pos = key0 + i * kTile;
            if (!wait(full(i, 1), full_turn(i))) break;
            if (pos < all.all_lo || pos + kTile > all.all_hi) {
                // Rows that nobody sees become zeros (a page's slots past the
                // length may hold anything, and 0 x NaN is NaN); a value that is
                // not finite among the others sends the CTA down the slow path.
                unsigned char *v = sgen + slot_at(x.slot);
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
            if (lane == 0) ptx::mbar_arrive(ready(i));
        }
    } else if (I8 && warp == 1) {
        // ------------------------------------------------------- codes' loads
        if constexpr (I8) {
            using P = Turn<C::kPieces>;
            const int run = min(1 << c.page_shift, C::kPieceKeys), runs = C::kPieceKeys / run;   // of a page's consecutive rows
            // Lane x < 2 runs: the page of tile i's position x * run as loaded (two
            // tiles ahead), and from it the pool's row (-1: no row that anybody sees).
            const auto needed = [&](int i) {
                const int pos = key0 + i * kTile + lane * run;
                return i < n && lane < 2 * runs && pos + run > all.lo && pos < all.hi;
            };
            const auto page_entry = [&](int i) -> int {
                return needed(i) ? __ldg(c.page_table + (size_t)b * c.max_pages + ((key0 + i * kTile + lane * run) >> c.page_shift)) : 0;
            };
            int entry = page_entry(0), entry_next = page_entry(1), done = 0;
            bool ok = true;
            for (int i = 0; i < n && ok; ++i) {
                long long row = -1;
                if (needed(i)) {
                    if ((unsigned)entry < (unsigned)c.num_pages)
                        row = ((entry * c.kv_heads + head) << c.page_shift) + ((key0 + i * kTile + lane * run) & ((1 << c.page_shift) - 1));
                    else
                        atomicOr(c.status, kStatusBadIndex);
                }
                entry = entry_next;
                entry_next = page_entry(i + 2);
                const unsigned with = __ballot_sync(~0u, row >= 0);
#pragma unroll
                for (int piece = 0; piece < 4 && ok; ++piece) {
                    const P x(4 * i + piece);
                    const int first = (piece & 1) * runs;
                    if (lane == 0) {
                        ok = wait(raw_empty(x.slot), x.parity ^ 1) && !lost();
                        if (ok) ptx::mbar_arrive_expect_tx(raw_full(x.slot), __popc(with >> first & ((1u << runs) - 1u)) * run * D);
                    }
                    ok = __shfl_sync(~0u, (int)ok, 0) != 0;
                    if (ok && row >= 0 && lane >= first && lane < first + runs)
                        bulk_load(sbase + C::kRaw + x.slot * C::kPiece + (lane - first) * run * D,
                                  static_cast<const char *>(piece >> 1 ? c.v : c.k) + row * D, run * D, raw_full(x.slot));
                    if (ok) ++done;
                }
            }
            // The copies in flight land before the CTA leaves, whoever gives up.
            if (lane == 0)
                for (int x = max(0, done - C::kPieces); x < done; ++x) wait(raw_full(P(x).slot), P(x).parity);
        }
    } else if (I8 && (warp < 4 || warp >= 20)) {
        // ------------------------------------------------------- converters
        if constexpr (I8) {
            using P = Turn<C::kPieces>;
            constexpr int kU = D / 16;                                  // 16-code units of a row
            constexpr int kLanes = C::kConverters * 32, kRowsOnce = kLanes / kU, kPer = C::kPieceKeys / kRowsOnce;
            static_assert(kRowsOnce % 8 == 0 && kPer * kRowsOnce == C::kPieceKeys && kLanes == kTile, "a thread's rows are alike in the swizzle");
            const int t = (warp < 4 ? warp - 2 : warp - 18) * 32 + lane, u = t % kU, row0 = t / kU;
            // Where a unit's first 16 bytes go in an operand.  Lanes of the second 64
            // dimensions write their upper 8 first: the eight lanes of a row are then
            // in eight different banks' sixteen bytes.
            const uint32_t second = D == 128 ? u >> 2 : 0;
            const uint32_t place = C::kRing + (u >> 2) * C::kPanel + row0 * 128 + ((((u & 3) * 2 + second) ^ (row0 & 7)) << 4);
            // Thread t takes the scales of tile i's key t: the page two tiles ahead, the scales one.
            const auto sees = [&](int i) {
                const int pos = key0 + i * kTile + t;
                return i < n && pos >= all.lo && pos < all.hi;
            };
            const auto page_entry = [&](int i) -> int {
                return sees(i) ? __ldg(c.page_table + (size_t)b * c.max_pages + ((key0 + i * kTile + t) >> c.page_shift)) : -1;
            };
            const auto scales = [&](int i, int entry) -> float2 {
                if (!sees(i) || (unsigned)entry >= (unsigned)c.num_pages) return make_float2(0.0f, 0.0f);
                const int at = ((entry * c.kv_heads + head) << c.page_shift) + ((key0 + i * kTile + t) & ((1 << c.page_shift) - 1));
                return make_float2(__ldg(c.k_scale + at), __ldg(c.v_scale + at));
            };
            float2 sc_next = scales(0, page_entry(0));
            int entry = page_entry(1);
            bool ok = true;
            for (int i = 0; i < n && ok; ++i) {
                const float2 sc = sc_next;
                sc_next = scales(i + 1, entry);
                entry = page_entry(i + 2);
#pragma unroll
                for (int piece = 0; piece < 4; ++piece) {
                    const int side = piece >> 1, half = piece & 1;
                    const T item(2 * i + side);
                    const P x(4 * i + piece);
                    ok = wait(raw_full(x.slot), x.parity) && !lost();
                    ok = __all_sync(~0u, ok);
                    if (!ok) break;
                    uint4 raw[kPer];
#pragma unroll
                    for (int r = 0; r < kPer; ++r)
                        raw[r] = *reinterpret_cast<const uint4 *>(sgen + C::kRaw + x.slot * C::kPiece + r * (kLanes * 16) + t * 16);
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(raw_empty(x.slot));
                    // Zeros for positions that nobody sees.
                    const int pos = key0 + i * kTile + half * C::kPieceKeys;
                    if (pos < all.lo || pos + C::kPieceKeys > all.hi) {
#pragma unroll
                        for (int r = 0; r < kPer; ++r) {
                            const int key = pos + r * kRowsOnce + row0;
                            if (key < all.lo || key >= all.hi) raw[r] = make_uint4(0, 0, 0, 0);
                        }
                    }
                    if (half == 0) {
                        ok = wait(empty(item.slot), item.parity ^ 1) && !lost();
                        ok = __all_sync(~0u, ok);
                        if (!ok) break;
                    }
                    unsigned char *const to = sgen + item.slot * C::kOperand + half * (C::kPieceKeys * 128);
#pragma unroll
                    for (int r = 0; r < kPer; ++r) {
                        const uint4 a = raw[r];
                        const uint32_t w[4] = {second ? a.z : a.x, second ? a.w : a.y, second ? a.x : a.z, second ? a.y : a.w};
                        uint32_t o[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            o[2 * e] = frag::i8_pair(__byte_perm(w[e], 0, 0x4140));
                            o[2 * e + 1] = frag::i8_pair(__byte_perm(w[e], 0, 0x4342));
                        }
                        *reinterpret_cast<uint4 *>(to + place + r * (kRowsOnce * 128)) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4 *>(to + (place ^ 16) + r * (kRowsOnce * 128)) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                    if (piece == 3) {   // both sides' scales go with the values
                        float *at = reinterpret_cast<float *>(sgen + C::kScale) + (i % C::kScaleTiles) * kTile;
                        at[t] = sc.x * L.scale_log2;
                        at[C::kScaleTiles * kTile + t] = sc.y;
                    }
                    if (half == 1) {
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(full(i, side));
                    }
                }
            }
        }
    }
    __syncwarp();

    constexpr bool kExact = MODE == kAttnWeighed;
    float m = -INFINITY, l = 0.0f, lx = 0.0f;   // lx: of the probabilities before they are rounded (kExact)
    // A softmax warp's half, its part of each tile's keys (and of O's
    // dimensions), and its thread's row.
    const int h = ((warp - 4) >> 2) & 1, part = (warp - 4) >> 3;
    const int hr = (warp & 3) * 32 + lane, r = r0 + h * kHalf + hr;
    const uint32_t lanes = (uint32_t)(warp & 3) * 32u << 16;
    const bool softmax = warp >= 4 && warp < 20 && h < halves;
    constexpr int kDims = D / 2;                      // of O a thread rescales and writes
    float *const share = reinterpret_cast<float *>(sgen + C::kShare);
    const int pair_bar = 1 + h * 4 + (warp & 3);      // the two warps of 32 rows
    if (softmax) {
        // ------------------------------------------------------- softmax
        {   // the half's rows of Q, in the operand's swizzled rows: consecutive lanes
            // take consecutive 16 bytes of a row
            const int at = part * 128 + hr;
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
                const int unit = x * 256 + at, row = unit / (D / 8), u = unit % (D / 8);
                const int qr = r0 + h * kHalf + row;
                const uint4 w = qr < rs.R ? __ldg(reinterpret_cast<const uint4 *>(rs.query(L, qr, D)) + u) : make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4 *>(sgen + C::kQ + h * C::kOperand + (u >> 3) * C::kPanel + row * 128 + (((u & 7) ^ (row & 7)) << 4)) = w;
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(q_full(h));
        }
        const int last = min(r1, r0 + (h + 1) * kHalf);
        const Span mine = span_of(L, rs, r0 + h * kHalf, last);
        const Seen z = rs.seen(L, min(r, rs.R - 1));
        const uint32_t t_mine = t_s(h) + lanes;
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            ok = wait(s_full(h), i & 1) && !lost();
            if (I8 && ok) ok = wait(full(i, 1), full_turn(i));   // the tile's scales
            __syncwarp();
            // The two warps leave together, whatever ran out.
            if (ptx::bar_red_or(pair_bar, 64, !ok)) break;
            ptx::tc_fence_after();
            const int pos = key0 + i * kTile;
            const bool partial = pos < mine.all_lo || pos + kTile > mine.all_hi;
            const int col0 = part * kCols;
            const float *ks = reinterpret_cast<const float *>(sgen + C::kScale) + (i % C::kScaleTiles) * kTile + col0;
            const float *vs = ks + C::kScaleTiles * kTile;
            const int first = z.lo - pos - col0, end = z.hi - pos - col0;   // of my columns, [first, end) are seen
            uint32_t p[kCols / 2];
            if (i == 0) {
                // The first tile's largest score is the first reference.
                float top;
                if (partial) top = tile_top<I8, true>(t_mine + col0, L.scale_log2, ks, first, end);
                else top = tile_top<I8, false>(t_mine + col0, L.scale_log2, ks, first, end);
                share[part * kRows + h * kHalf + hr] = top;
                ptx::bar_red_or(pair_bar, 64, false);
                m = fmaxf(top, share[(part ^ 1) * kRows + h * kHalf + hr]);
                ptx::bar_red_or(pair_bar, 64, false);   // `share` may be written again
            }
            while (true) {
                // Scores in base 2 above the reference maximum, their largest, the
                // probabilities and their sum.
                const float ref = m == -INFINITY ? 0.0f : m;
                float top, sum;
                if (partial) tile_pass<I8, true, kExact>(t_mine + col0, L.scale_log2, ref, ks, vs, first, end, p, top, sum);
                else tile_pass<I8, false, kExact>(t_mine + col0, L.scale_log2, ref, ks, vs, first, end, p, top, sum);
                top += ref;
                const bool grow = top > m + kLazy;   // also from m = -inf
                // Both warps have read their scores here: P may replace them.
                if (!ptx::bar_red_or(pair_bar, 64, grow)) {
                    if constexpr (kExact) lx += sum;
                    if constexpr (I8 || !kExact) l += sum;
                    break;
                }
                // Raise the maxima to what both threads of a row saw, and read
                // the scores again.
                share[part * kRows + h * kHalf + hr] = top;
                ptx::bar_red_or(pair_bar, 64, false);
                const float nm = fmaxf(m, fmaxf(top, share[(part ^ 1) * kRows + h * kHalf + hr]));
                const float fac = nm == -INFINITY ? 1.0f : frag::ex2(m - nm);
                if (i > 0) {
                    ok = wait(pv_done(h), (i - 1) & 1);
                    __syncwarp();
                    ptx::tc_fence_after();
                    if (__all_sync(~0u, ok)) {
#pragma unroll
                        for (int q = 0; q < kDims / 32; ++q) {
                            uint32_t v[32];
                            const uint32_t at = t_o(h) + lanes + part * kDims + 32 * q;
                            tmem_ld32(at, v);
                            ptx::tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * fac);
                            tmem_st32(at, v);
                        }
                        tmem_st_wait();
                    }
                }
                l *= fac;
                if constexpr (kExact) lx *= fac;
                m = nm;
                ptx::bar_red_or(pair_bar, 64, false);   // `share` may be written again
            }
            if (is_far(m)) words[2] = 1;
            tmem_st32(t_mine + part * (kCols / 2), p);
            if constexpr (!I8) l += sum_rounded(p);
            tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(p_ready(h));
        }
        if (n > 0 && ok) wait(pv_done(h), (n - 1) & 1);
        __syncwarp();
        ptx::tc_fence_after();
        share[part * kRows + h * kHalf + hr] = l;
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();

    // ---------------------------------------------------------- output
    end_attention<MODE>();   // the prefix's shares
    const bool join = MODE != kAttnPlain || active > 1;
    if (softmax && !lost()) {
        // Float rows of a range and their (maximum, sum), for the join: where the
        // ring and Q were.
        unsigned char *const f_rows = sgen + C::kRing + h * (kHalf * D * 4);
        float2 *const stats = reinterpret_cast<float2 *>(sgen + C::kQ + C::kJoinStats);
        if (words[2]) {
            constexpr int kE = D / 32;
            float lx_row = 0.0f;
            if constexpr (kExact) {
                share[part * kRows + h * kHalf + hr] = lx;
                ptx::bar_red_or(pair_bar, 64, false);
                lx_row = lx + share[(part ^ 1) * kRows + h * kHalf + hr];
            }
            for (int x = part; x < 32; x += 2) {
                const int row = r - lane + x;
                if (row >= rs.R) break;
                float acc[kE], mm, ll;
                slow_row<D, I8>(L, rs, b, row, key0, key0 + n * kTile, lane, acc, mm, ll);
                // What the weights are divided by is of the scores that they are taken from:
                // this pass's own but for far rows (k_attn_weights.cu).
                float exact = ll;
                if constexpr (kExact) {
                    const float m_row = __shfl_sync(~0u, m, x), sum_row = __shfl_sync(~0u, lx_row, x);
                    if (mm != -INFINITY && !is_far(m_row)) exact = sum_row * frag::ex2(m_row - mm);
                }
                if (!join) {
                    const Seen z = rs.seen(L, row);
                    const float inv = __fdiv_rn(1.0f, ll);
#pragma unroll
                    for (int e = 0; e < kE; ++e)
                        rs.out(L, row, D)[lane * kE + e] = __float2bfloat16_rn(z.hi > z.lo ? acc[e] * inv : 0.0f);
                } else {
#pragma unroll
                    for (int e = 0; e < kE; ++e) {
                        const int d = lane * kE + e, hrow = hr - lane + x;
                        *reinterpret_cast<float *>(f_rows + hrow * (D * 4) + (((d >> 2) ^ (hrow & 7)) << 4) + (d & 3) * 4) = acc[e];
                    }
                    if (lane == 0) {
                        stats[row - r0] = make_float2(mm, ll);
                        if constexpr (kExact) reinterpret_cast<float *>(sgen + C::kQ + C::kJoinSums)[row - r0] = exact;
                    }
                }
            }
        } else {
            // Through shared memory (the ring, and Q, are free), so that stores
            // are of whole rows: bf16 rows in Q's place, or float rows in the ring's.
            const Seen z = rs.seen(L, min(r, rs.R - 1));
            l += share[(part ^ 1) * kRows + h * kHalf + hr];
            const bool any = z.hi > z.lo && n > 0;
            const float inv = __fdiv_rn(1.0f, l);
            unsigned char *const b_rows = sgen + C::kQ + h * C::kOperand;
#pragma unroll
            for (int q = 0; q < kDims / 32; ++q) {
                uint32_t v[32];
                if (n > 0) {
                    tmem_ld32(t_o(h) + lanes + part * kDims + 32 * q, v);
                    ptx::tmem_ld_wait();
                }
                const int dim = part * kDims + 32 * q;
                if (!join) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t w[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            w[y] = any ? frag::pack_bf16(__uint_as_float(v[8 * e + 2 * y]) * inv,
                                                         __uint_as_float(v[8 * e + 2 * y + 1]) * inv)
                                       : 0u;
                        const int u = dim / 8 + e;
                        *reinterpret_cast<uint4 *>(b_rows + hr * (D * 2) + ((u ^ (hr & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int u = dim / 4 + e;
                        *reinterpret_cast<uint4 *>(f_rows + hr * (D * 4) + ((u ^ (hr & 7)) << 4)) =
                            make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                    }
                }
            }
            if (join && part == 0) stats[r - r0] = make_float2(m, l);
            if constexpr (kExact) {
                ptx::bar_red_or(pair_bar, 64, false);   // both have read `share`
                share[part * kRows + h * kHalf + hr] = lx;
                ptx::bar_red_or(pair_bar, 64, false);
                if (part == 0) reinterpret_cast<float *>(sgen + C::kQ + C::kJoinSums)[r - r0] = lx + share[kRows + h * kHalf + hr];
            }
            if (!join) {
                ptx::bar_red_or(9 + h, 256, false);   // the half's rows are in place
                const int mine = part * 128 + hr;
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    const int unit = x * 256 + mine, row = unit / (D / 8), u = unit % (D / 8);
                    const int qr = r0 + h * kHalf + row;
                    if (qr < rs.R)
                        reinterpret_cast<uint4 *>(rs.out(L, qr, D))[u] =
                            *reinterpret_cast<const uint4 *>(b_rows + row * (D * 2) + ((u ^ (row & 7)) << 4));
                }
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc(tmem, 512);
    if (!join) {
        if (L.split > 1) cluster_sync(), cluster_sync();
        return;
    }

    // ------------------------------------------------------------ join
    // Each CTA of the cluster finishes its part of the rows: the ranges in their
    // order, read from the CTAs' shared memory.
    cluster_sync();
    const int all_rows = min(kRows, rs.R - r0), rows_each = (all_rows + active - 1) / active;
    const int j0 = sp * rows_each, rows_mine = max(min(all_rows - j0, rows_each), 0);
    float *const facs = reinterpret_cast<float *>(sgen + C::kQ + C::kJoinFacs);   // [range][row], then the sums
    // The rows' maxima and exact sums, where the threads of a row exchanged theirs.
    float2 *const own_top = reinterpret_cast<float2 *>(sgen + C::kShare);
    for (int j = tid; j < rows_mine; j += C::kThreads) {
        const uint32_t at = sbase + C::kQ + C::kJoinStats + (j0 + j) * 8;
        float2 st[kMostRanges];
        float top = -INFINITY, sum = 0.0f, exact = 0.0f;
#pragma unroll
        for (int x = 0; x < kMostRanges; ++x) {
            if (x < active) st[x] = ld_cluster2(at, x), top = fmaxf(top, st[x].x);
        }
#pragma unroll
        for (int x = 0; x < kMostRanges; ++x) {
            if (x >= active) break;
            const float fac = share_factor(st[x].x, st[x].y, top);
            const bool skip = st[x].x == -INFINITY && fac == 0.0f;   // a range that saw nothing
            facs[x * kRows + j] = skip ? -1.0f : fac;
            if (!skip) sum = fmaf(st[x].y, fac, sum);
            if constexpr (kExact)
                if (!skip) exact = fmaf(ld_cluster1(sbase + C::kQ + C::kJoinSums + (j0 + j) * 4, x), fac, exact);
        }
        facs[kMostRanges * kRows + j] = sum;
        if constexpr (MODE != kAttnPlain) own_top[j] = make_float2(top, exact);
    }
    __syncthreads();
    constexpr int kU = D / 4;   // units of four dimensions
    for (int i = tid; i < rows_mine * kU; i += C::kThreads) {
        const int j = i / kU, u = i % kU, row = j0 + j;
        const uint32_t at = sbase + C::kRing + row * (D * 4) + ((u ^ (row & 7)) << 4);
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int x = 0; x < active; ++x) {
            const float4 v = ld_cluster4(at, x);
            const float fac = facs[x * kRows + j];
            if (fac < 0.0f) continue;
            acc.x = fmaf(v.x, fac, acc.x); acc.y = fmaf(v.y, fac, acc.y);
            acc.z = fmaf(v.z, fac, acc.z); acc.w = fmaf(v.w, fac, acc.w);
        }
        float2 own = make_float2(0.0f, 0.0f);
        if constexpr (MODE != kAttnPlain) own = own_top[j];
        store_out4<MODE>(L, rs, r0 + row, D, 4 * u, acc, facs[kMostRanges * kRows + j], own.x, own.y);
    }
    __syncthreads();
    cluster_sync();   // nobody's rows go while another CTA reads them
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

template <int D, bool I8, int MODE>
cbs_status launch_chunk(const AttnLaunch &L, cudaStream_t s) {
    alignas(64) CUtensorMap tk = {}, tv = {};
    if (!I8) {
        CBS_TRY(pool_map(&tk, L.c, L.c.k));
        CBS_TRY(pool_map(&tv, L.c, L.c.v));
    }
    using C = Chunk<D, I8>;
    auto kern = attn_chunk_kernel<D, I8, MODE>;
    static ContextOfDevice set;
    CBS_TRY(cuda_check(set_max_dyn_smem_once(kern, C::kSmem, set), "attention shared memory"));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(L.split, L.c.kv_heads * L.row_tiles, L.c.batch);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = (launch_options() & CBS_LAUNCH_PDL) ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = L.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = L.split > 1 ? 2 : 1;
    return cuda_check(cudaLaunchKernelEx(&cfg, kern, tk, tv, L), "attention launch");
}

template <int MODE>
cbs_status launch_attn_chunk_as(const AttnLaunch &L, cudaStream_t s) {
    if (L.c.head_dim == 64) return L.c.int8 ? launch_chunk<64, true, MODE>(L, s) : launch_chunk<64, false, MODE>(L, s);
    return L.c.int8 ? launch_chunk<128, true, MODE>(L, s) : launch_chunk<128, false, MODE>(L, s);
}

}  // namespace

}  // namespace cbs
