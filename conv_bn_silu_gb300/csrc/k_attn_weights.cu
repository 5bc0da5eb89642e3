// k_attn_weights.cu -- the weight that each position of a paged cache received from
// a call's new tokens: over the rows (token, query head) of its key head
//
//   mass[key] = decay mass[key] + sum_r p[r, key],   p = 2^(score - m_r) / l_r
//
// (a key that is new in the call starts at zero), with the rows' maxima m_r and sums
// l_r from the attention that ran before.  Every key has one owner, so nothing is
// added atomically and equal calls give equal results.
//
// Few rows: the attention left its scores, 4 bytes a row and key where the key itself
// has 64 to 256.  Where one tile holds a head's rows it sums them up itself, in the CTAs
// that know the rows' sums; else the first kernel here does.  Chunks would leave too many: the
// second kernel takes the first product again, S^T = K Q^T on tcgen05 with 128 keys as
// the lanes of tensor memory.  A key tile stays where it is while the rows' tiles
// pass, and a thread's sum over them never leaves its registers.  The exponentials,
// one a score and sixteen a clock and SM, bound it from below: 1024 tokens over 16384
// keys, 32 heads, 107 us of them; it takes 155, for a buffer of scores goes from hand to
// hand in some 3000 cycles.  (32 streams of one token, 8192 keys, 8 bits: the first
// kernel 15 us after an attention of 98.)
#include "attn_common.cuh"
#include "tc_ptx.cuh"
#include "tc_warp.cuh"

namespace cbs {

namespace {

// A sequence's rows as the attention took them (which has reported what is wrong with them).
__device__ __forceinline__ Rows rows_again(const AttnLaunch &L, int b, int head) {
    const CacheArgs &c = L.c;
    Rows s;
    s.len = seq_len(c, b);
    s.start = max(0, min(c.new_start[b], c.total));
    s.fresh = min(max(s.start, min(c.new_start[b + 1], c.total)) - s.start, L.max_new);
    s.R = s.fresh * L.group;
    s.head = head;
    s.base = s.len - s.fresh;
    return s;
}

// A warp's lanes take four keys each; a CTA's warps lie along the keys or, `along` of
// them, along the rows, whose shares are then added in the warps' order (64 rows of 100,
// 400 and 1500 keys, with the attention: 19.4, 20.0 and 22.7 us when every warp took all
// rows, now 9.5, 10.2 and 12.4).
constexpr int kSumWarps = 8, kSumThreads = 32 * kSumWarps, kWarpKeys = 128;

__global__ void __launch_bounds__(kSumThreads) weights_of_scores_kernel(const AttnLaunch L, int along) {
    __shared__ float4 s_sum[kSumWarps][32];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const CacheArgs &c = L.c;
    const int head = blockIdx.y, b = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Rows rs = rows_again(L, b, head);
    if (rs.fresh == 0) return;
    if (rs.len > L.len_pad && threadIdx.x == 0) atomicOr(c.status, kStatusBadIndex);
    const int part = warp % along, end = min(rs.len, L.len_pad);
    const int key = (blockIdx.x * (kSumWarps / along) + warp / along) * kWarpKeys + 4 * lane;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (key < end) sum = weigh_four(L, rs, b, key, 4 * part, 4 * along, [&](int r) { return __ldg(&L.row_stats[rs.number(L, r)]); });
    if (along > 1) {
        s_sum[warp][lane] = sum;
        __syncthreads();
        for (int x = 1; x < along && part == 0; ++x) {
            const float4 v = s_sum[warp + x][lane];
            sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
        }
    }
    if (part == 0 && key < end) store_four(L, rs, b, key, end, sum);
}

// ------------------------------------------------------------------- chunks
// A tile of rows is kRowTile of them at most: T tokens' S query heads each, where S is
// all of a key head's (or, of more than 128, its largest divisor that fits) and T as
// many as fit, so that one box of TMA brings them.  Two warpgroups take tiles in turn,
// a thread a key; two CTAs an SM, so that one's start runs beside the other's sums.
constexpr int kKeys = 128, kRowTile = 128, kBufs = 2;
constexpr int kStatWarps = 4, kWarpMma = 4 * kBufs + kStatWarps, kWarpTma = kWarpMma + 1, kThreads = (kWarpTma + 1) * 32;
constexpr uint64_t kWaitNs = 2000000000ull;   // 2 s per wait

template <int D>
struct Weigh {
    static constexpr int kOperand = (D / 64) * kKeys * 128;   // panels of 64 dimensions
    static constexpr int kQ = kOperand, kStats = kQ + kBufs * kOperand;
    // each buffer's rows: -m[128], 1 / l[128], lo[128], hi[128]; after them whether one is far
    static constexpr int kStat = 4 * kRowTile * 4, kFar = kStats + kBufs * kStat, kBars = kFar + kBufs * 8;
    static constexpr int kNumBars = 4 * kBufs;   // q_full[], stat_full[], s_full[], s_free[]
    static constexpr int kSum = kBars + kNumBars * 8, kSmem = kSum + (kBufs - 1) * kKeys * 4 + 16;
    static_assert(kSmem <= 113 * 1024, "two CTAs an SM");
};

// As slow_row takes a row's score of a key, to the bit.
template <int D, bool I8>
__device__ __noinline__ float slow_score(const AttnLaunch &L, const Rows &s, int r, size_t row, int lane) {
    constexpr int kE = D / 32;
    const __nv_bfloat16 *q = s.query(L, r, D) + lane * kE;
    const size_t at = row * D + lane * kE;
    float dot = 0.0f;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        const float k = I8 ? (float)static_cast<const int8_t *>(L.c.k)[at + e] : __bfloat162float(static_cast<const __nv_bfloat16 *>(L.c.k)[at + e]);
        dot = fmaf(__bfloat162float(q[e]), k, dot);
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) dot += __shfl_xor_sync(~0u, dot, x);
    return __fmul_rn(dot, I8 ? L.c.k_scale[row] * L.scale_log2 : L.scale_log2);
}

// Whether a row of the keys' operand holds an infinity or a NaN.
template <int D>
__device__ __noinline__ bool odd_key(const unsigned char *keys, int row) {
    const auto not_finite = [](uint32_t x) { return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u; };
    bool odd = false;
    for (int u = 0; u < D / 8; ++u) {
        const uint4 w = *reinterpret_cast<const uint4 *>(keys + (u >> 3) * (kKeys * 128) + row * 128 + (((u & 7) ^ (row & 7)) << 4));
        odd |= not_finite(w.x) || not_finite(w.y) || not_finite(w.z) || not_finite(w.w);
    }
    return odd;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *tmap, uint32_t bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// A thread's sum over a tile's rows: scores, as they come from tensor memory, to
// exponentials times what belongs to each row.  Two lanes of an instruction at a time,
// and the next sixteen scores on their way.
// MASK: rows that do not see `key` are left out.
template <bool MASK>
__device__ __forceinline__ void tile_sum(uint32_t taddr, const float *stat, float scale, int key, F2 (&sums)[2]) {
    const int *lo = reinterpret_cast<const int *>(stat) + 2 * kRowTile, *hi = lo + kRowTile;
    const F2 scale2 = pair(scale, scale);
    const auto part = [&](const uint32_t (&v)[16], int q) {
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
            const float4 m = *reinterpret_cast<const float4 *>(stat + 16 * q + e), inv = *reinterpret_cast<const float4 *>(stat + kRowTile + 16 * q + e);
            const float2 a = split(fma2(pair(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), scale2, pair(m.x, m.y)));
            const float2 b = split(fma2(pair(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])), scale2, pair(m.z, m.w)));
            float x[4] = {frag::ex2(a.x), frag::ex2(a.y), frag::ex2(b.x), frag::ex2(b.y)};
            if constexpr (MASK) {
                const int4 l4 = *reinterpret_cast<const int4 *>(lo + 16 * q + e), h4 = *reinterpret_cast<const int4 *>(hi + 16 * q + e);
                x[0] = key >= l4.x && key < h4.x ? x[0] * inv.x : 0.0f;
                x[1] = key >= l4.y && key < h4.y ? x[1] * inv.y : 0.0f;
                x[2] = key >= l4.z && key < h4.z ? x[2] * inv.z : 0.0f;
                x[3] = key >= l4.w && key < h4.w ? x[3] * inv.w : 0.0f;
                const F2 one = pair(1.0f, 1.0f);
                sums[0] = fma2(pair(x[0], x[1]), one, sums[0]);
                sums[1] = fma2(pair(x[2], x[3]), one, sums[1]);
            } else {
                sums[0] = fma2(pair(x[0], x[1]), pair(inv.x, inv.y), sums[0]);
                sums[1] = fma2(pair(x[2], x[3]), pair(inv.z, inv.w), sums[1]);
            }
        }
    };
    uint32_t u[16], v[16];
    ptx::tmem_ld16(taddr, u);
#pragma unroll
    for (int q = 0; q < kRowTile / 16; q += 2) {
        ptx::tmem_ld_wait();
        ptx::tmem_ld16(taddr + 16 * (q + 1), v);
        part(u, q);
        ptx::tmem_ld_wait();
        if (q + 2 < kRowTile / 16) ptx::tmem_ld16(taddr + 16 * (q + 2), u);
        part(v, q + 1);
    }
}

// Tiles of a call: S heads, T tokens, and how many tiles a token's heads make.
struct RowTiles {
    int heads, tokens, parts;
    static RowTiles of(int group) {
        RowTiles t = {group, 1, 1};
        if (group <= kRowTile) t.tokens = kRowTile / group;
        else
            for (t.heads = kRowTile; group % t.heads; --t.heads) {}
        t.parts = group / t.heads;
        return t;
    }
};

template <int D, bool I8>
__global__ void __launch_bounds__(kThreads, 2) weights_of_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const AttnLaunch L, const RowTiles rt) {
    using C = Weigh<D>;
    extern __shared__ __align__(1024) unsigned char smem[];   // the only shared memory: starts at a multiple of 1 KB
    const uint32_t sbase = ptx::smem_u32(smem);
    const CacheArgs &c = L.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp == kWarpTma && lane == 0) ptx::prefetch_tmap(&tm_q);
    ptx::griddep_wait();
    const int head = blockIdx.y, b = blockIdx.z, key0 = blockIdx.x * kKeys;
    const Rows rs = rows_again(L, b, head);
    if (rs.len > L.len_pad && tid == 0) atomicOr(c.status, kStatusBadIndex);
    const int end = min(min(rs.len, L.len_pad), key0 + kKeys);
    if (rs.fresh == 0 || key0 >= end) return;
    // The tokens that see one of the keys, and the tiles of their rows.
    const int t0 = (int)min((long long)rs.fresh, L.causal ? max(0ll, (long long)key0 - rs.base) : 0ll);
    const int t1 = (int)max((long long)t0, L.window ? min((long long)rs.fresh, (long long)end - 1 + L.window - rs.base) : (long long)rs.fresh);
    const int tiles = (t1 - t0 + rt.tokens - 1) / rt.tokens * rt.parts;
    struct Tile { int token, head, tokens; };   // of the sequence and of the key head; of them within t1
    const auto tile_of = [&](int i) {
        const int group = rt.parts == 1 ? i : i / rt.parts;
        return Tile{t0 + group * rt.tokens, (i - group * rt.parts) * rt.heads, min(rt.tokens, t1 - t0 - group * rt.tokens)};
    };

    const auto bar = [&](int i) { return sbase + C::kBars + 8u * i; };
    const auto q_full = [&](int s) { return bar(s); };                // a tile's rows have arrived
    const auto stat_full = [&](int s) { return bar(kBufs + s); };     // and what the attention left of them
    const auto s_full = [&](int s) { return bar(2 * kBufs + s); };    // its scores are there (and its rows have been used)
    const auto s_free = [&](int s) { return bar(3 * kBufs + s); };    // and have been summed up
    volatile uint32_t *const words = reinterpret_cast<volatile uint32_t *>(smem + C::kSum + (kBufs - 1) * kKeys * 4);
    // words[0]: TMEM address; [1]: a wait ran out
    if (tid == 0) {
        for (int s = 0; s < kBufs; ++s) {
            ptx::mbar_init(q_full(s), 1);
            ptx::mbar_init(stat_full(s), kStatWarps);
            ptx::mbar_init(s_full(s), 1);
            ptx::mbar_init(s_free(s), 4);
        }
        ptx::fence_mbar_init();
        words[1] = 0;
    }
    if (warp == kWarpMma) {
        ptx::tmem_alloc(sbase + C::kSum + (kBufs - 1) * kKeys * 4, kBufs * kRowTile);
        ptx::tmem_relinquish();
    }
    // The keys, widened, in the operand's swizzled rows; zeros past the end.
    constexpr int kU = D / (I8 ? 16 : 8);   // units of 16 bytes of the cache
    for (int i = tid; i < kKeys * kU; i += kThreads) {
        const int row = i / kU, u = i % kU, key = key0 + row;
        const int p = key < end ? page_of(c, b, key) : -1;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (p >= 0) {
            const size_t at = (((size_t)p * c.kv_heads + head) << c.page_shift) + (key & ((1 << c.page_shift) - 1));
            w = __ldg(reinterpret_cast<const uint4 *>(static_cast<const char *>(c.k) + at * (D * (I8 ? 1 : 2))) + u);
        }
        if constexpr (I8) {
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                o[2 * e] = frag::i8_pair(__byte_perm(x[e], 0, 0x4140));
                o[2 * e + 1] = frag::i8_pair(__byte_perm(x[e], 0, 0x4342));
            }
            unsigned char *to = smem + (u >> 2) * (kKeys * 128) + row * 128;
            const int ch = (u & 3) * 2;
            *reinterpret_cast<uint4 *>(to + ((ch ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4 *>(to + (((ch + 1) ^ (row & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
        } else {
            *reinterpret_cast<uint4 *>(smem + (u >> 3) * (kKeys * 128) + row * 128 + (((u & 7) ^ (row & 7)) << 4)) = w;
        }
    }
    // Rows that no box brings: zeros, whose exponentials then count for nothing (but with
    // a key that is not finite: its summing warp leaves them out).
    const int boxed = rt.heads * rt.tokens, rest = (kRowTile - boxed) * 8;
    for (int i = tid; i < kBufs * (D / 64) * rest; i += kThreads)
        *reinterpret_cast<uint4 *>(smem + C::kQ + (i / rest) * (kKeys * 128) + boxed * 128 + i % rest * 16) = make_uint4(0, 0, 0, 0);
    ptx::fence_proxy_async_smem();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    ptx::griddep_launch_dependents();
    const uint32_t tmem = words[0];

    const auto wait = [&](uint32_t bar_, uint32_t parity) -> bool {
        if (ptx::mbar_wait_bounded(bar_, parity, kWaitNs)) return true;
        words[1] = 1;
        atomicOr(c.status, kStatusTimeout);
        return false;
    };
    const auto lost = [&] { return words[1] != 0; };

    const int key = key0 + (warp & 3) * 32 + lane;   // a summing thread's
    float acc = 0.0f;
    if (warp == kWarpMma) {
        // ------------------------------------------------------- MMA issue
        constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((kRowTile >> 3) << 17) | ((kKeys >> 4) << 24);
        const uint32_t lead = elect_one();
        const uint64_t d_k = ptx::smem_desc(sbase, 16, 1024, 2), d_q = ptx::smem_desc(sbase + C::kQ, 16, 1024, 2);
        int issued = 0;
        for (int i = 0; i < tiles; ++i) {
            const int s = i % kBufs;
            const uint32_t turn = (i / kBufs) & 1;
            if (!__all_sync(~0u, wait(q_full(s), turn) && wait(s_free(s), turn ^ 1) && !lost())) break;
            ptx::tc_fence_after();
            const uint64_t q = d_q + (uint32_t)(s * C::kOperand) / 16;
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
                const uint32_t off = (x >> 2) * (kKeys * 128 / 16) + (x & 3) * 2;
                mma_ss(lead, tmem + (uint32_t)(s * kRowTile), d_k + off, q + off, idesc, x > 0);
            }
            mma_commit(lead, s_full(s));
            ++issued;
        }
        // Nothing leaves while an MMA reads shared memory.
        for (int i = max(0, issued - kBufs); i < issued; ++i)
            if (!ptx::mbar_wait_bounded(s_full(i % kBufs), (i / kBufs) & 1, kWaitNs)) atomicOr(c.status, kStatusTimeout);
    } else if (warp == kWarpTma) {
        // ------------------------------------------------------- rows
        if (lane == 0) {
            int loaded = 0;
            for (int i = 0; i < tiles; ++i) {
                const int s = i % kBufs;
                if (!wait(s_full(s), (i / kBufs + 1) & 1) || lost()) break;   // (used: their scores are there)
                const Tile t = tile_of(i);
                ptx::mbar_arrive_expect_tx(q_full(s), (uint32_t)(boxed * D * 2));
#pragma unroll
                for (int p = 0; p < D / 64; ++p)
                    tma_load_3d(sbase + C::kQ + s * C::kOperand + p * (kKeys * 128), &tm_q, q_full(s), p * 64, head * L.group + t.head, rs.start + t.token);
                ++loaded;
            }
            // The copies in flight land before the CTA leaves, whoever gives up.
            for (int i = max(0, loaded - kBufs); i < loaded; ++i) ptx::mbar_wait_bounded(q_full(i % kBufs), (i / kBufs) & 1, kWaitNs);
        }
    } else if (warp >= 4 * kBufs) {
        // ------------------------------------------- what the attention left
        // A row a thread, a tile ahead.
        const int t = tid - 4 * kBufs * 32, my_token = t / rt.heads, my_head = t - my_token * rt.heads;
        const auto row_of = [&](int i) {   // of the key head's, or -1
            if (i >= tiles) return -1;
            const Tile x = tile_of(i);
            return my_token < x.tokens ? (x.token + my_token) * L.group + x.head + my_head : -1;
        };
        const auto statistics = [&](int r) { return r >= 0 ? __ldg(&L.row_stats[rs.number(L, r)]) : make_float2(0.0f, 0.0f); };
        int row_next = row_of(0);
        float2 next = statistics(row_next);
        for (int i = 0; i < tiles; ++i) {
            const int s = i % kBufs, r = row_next;
            const float2 st = next;
            row_next = row_of(i + 1);
            next = statistics(row_next);
            const bool ok = wait(s_free(s), (i / kBufs + 1) & 1) && !lost();
            // A far row: by itself, from its own loads; here every exponential of it is zero.
            const bool far = is_far(st.x), any_far = ptx::bar_red_or(1, kStatWarps * 32, far);
            if (ptx::bar_red_or(1, kStatWarps * 32, !ok)) break;   // (together, whatever ran out)
            float *const stat = reinterpret_cast<float *>(smem + C::kStats + s * C::kStat);
            const Seen z = r >= 0 ? rs.seen(L, r) : Seen{0, 0};
            stat[t] = far ? -INFINITY : -st.x;
            stat[kRowTile + t] = far ? 0.0f : st.y;
            reinterpret_cast<int *>(stat)[2 * kRowTile + t] = z.lo;
            reinterpret_cast<int *>(stat)[3 * kRowTile + t] = z.hi;
            if (t == 0) *reinterpret_cast<volatile int *>(smem + C::kFar + 8 * s) = any_far;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(stat_full(s));
        }
    } else {
        // ------------------------------------------------------- sums
        const int wg = warp >> 2;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const int p = key < end ? page_of(c, b, key) : -1;
        const size_t at = p < 0 ? 0 : (((size_t)p * c.kv_heads + head) << c.page_shift) + (key & ((1 << c.page_shift) - 1));
        const float scale = I8 ? (p < 0 ? 0.0f : c.k_scale[at] * L.scale_log2) : L.scale_log2;
        // A box's tokens, where all of its rows may count (-1: rows that no box brings are left
        // out, beside a key that is not finite).
        int box_tokens = rt.tokens;
        if (rest > 0 && __any_sync(~0u, I8 ? !(fabsf(scale) < INFINITY) : odd_key<D>(smem, key - key0))) box_tokens = -1;
        F2 sums[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
        float slow = 0.0f;
        for (int i = wg; i < tiles; i += kBufs) {
            const Tile t = tile_of(i);
            const uint32_t turn = (i / kBufs) & 1;
            if (!__all_sync(~0u, wait(s_full(wg), turn) && wait(stat_full(wg), turn) && !lost())) break;
            ptx::tc_fence_after();
            const float *stat = reinterpret_cast<const float *>(smem + C::kStats + wg * C::kStat);
            // Every row of the box is the sequence's, and sees every key.
            const bool whole = t.tokens == box_tokens && seen_by(rs.base + t.token + t.tokens - 1, rs.len, L.causal, L.window).lo <= key0 &&
                               seen_by(rs.base + t.token, rs.len, L.causal, L.window).hi >= end;
            const uint32_t taddr = tmem + (uint32_t)(wg * kRowTile) + lanes;
            if (whole) tile_sum<false>(taddr, stat, scale, key, sums);
            else tile_sum<true>(taddr, stat, scale, key, sums);
            const bool far = *reinterpret_cast<volatile int *>(smem + C::kFar + 8 * wg) != 0;
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(s_free(wg));
            if (far) {   // seldom met
                for (int x = 0; x < t.tokens * rt.heads; ++x) {
                    const int r = (t.token + x / rt.heads) * L.group + t.head + x % rt.heads;
                    const float2 st = __ldg(&L.row_stats[rs.number(L, r)]);
                    if (!is_far(st.x)) continue;
                    const Seen z = rs.seen(L, r);
                    for (int y = 0; y < 32; ++y) {
                        const int k = __shfl_sync(~0u, key, y), kp = __shfl_sync(~0u, p, y);
                        const size_t row = (size_t)__shfl_sync(~0u, (unsigned long long)at, y);
                        if (kp < 0 || k < z.lo || k >= z.hi) continue;
                        const float w = frag::ex2(slow_score<D, I8>(L, rs, r, row, lane) - st.x) * st.y;
                        if (lane == y) slow += w;
                    }
                }
            }
        }
        const float2 a = split(sums[0]), d = split(sums[1]);
        acc = ((a.x + a.y) + (d.x + d.y)) + slow;
        if (wg > 0) reinterpret_cast<float *>(smem + C::kSum)[(wg - 1) * kKeys + key - key0] = acc;
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kWarpMma) ptx::tmem_dealloc(tmem, kBufs * kRowTile);
    if (warp < 4 && key < end && !lost()) {
#pragma unroll
        for (int g = 0; g < kBufs - 1; ++g) acc += reinterpret_cast<const float *>(smem + C::kSum)[g * kKeys + key - key0];
        const int p = page_of(c, b, key);
        if (p >= 0) {
            float *mass = L.mass + (((size_t)p * c.kv_heads + head) << c.page_shift) + (key & ((1 << c.page_shift) - 1));
            *mass = weight_after(L, rs, key, *mass, acc);
        }
    }
}

template <int D, bool I8>
cbs_status launch_chunk_weights(const AttnLaunch &L, cudaStream_t s) {
    EncodeTiledFn fn = encode_tiled();
    if (!fn) return fail(CBS_ERR_CUDA, "cannot resolve cuTensorMapEncodeTiled from the driver");
    // The call's rows [total][heads][D], boxes of T tokens, S heads and 64 dimensions.
    const RowTiles rt = RowTiles::of(L.group);
    alignas(64) CUtensorMap tq;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)L.heads, (cuuint64_t)L.c.total};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)L.q_stride * 2};
    const cuuint32_t box[3] = {64u, (cuuint32_t)rt.heads, (cuuint32_t)rt.tokens}, es[3] = {1u, 1u, 1u};
    const CUresult r = fn(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(L.q), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(CBS_ERR_CUDA, "cuTensorMapEncodeTiled (queries) failed (%d)", (int)r);
    static ContextOfDevice set;
    CBS_TRY(cuda_check(set_max_dyn_smem_once(weights_of_chunk_kernel<D, I8>, Weigh<D>::kSmem, set), "weights' shared memory"));
    return cuda_check(launch_kernel(weights_of_chunk_kernel<D, I8>, dim3((L.len_pad + kKeys - 1) / kKeys, L.c.kv_heads, L.c.batch), kThreads,
                                    Weigh<D>::kSmem, s, tq, L, rt), "weights launch");
}

}  // namespace

cbs_status launch_attn_weights(const AttnLaunch &L, cudaStream_t s) {
    if (L.scores) {
        int along = 1;   // a warp four rows at least
        while (along < kSumWarps && 8 * along <= L.rows_pad) along *= 2;
        const int keys = kSumWarps / along * kWarpKeys;
        return cuda_check(launch_kernel(weights_of_scores_kernel, dim3((L.len_pad + keys - 1) / keys, L.c.kv_heads, L.c.batch), kSumThreads, 0, s, L, along),
                          "weights launch");
    }
    if (L.c.head_dim == 64) return L.c.int8 ? launch_chunk_weights<64, true>(L, s) : launch_chunk_weights<64, false>(L, s);
    return L.c.int8 ? launch_chunk_weights<128, true>(L, s) : launch_chunk_weights<128, false>(L, s);
}

}  // namespace cbs
