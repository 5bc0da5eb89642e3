// k_attn_rows.cuh -- attention of few query rows over a paged cache (the single-token
// form, and short chunks): one pass over keys and values with the running
// maximum and sum of the softmax.
//
//   out[t, h] = sum_j p_j v_j / sum_j p_j,   p_j = 2^(scale log2(e) q.k_j - m)
//
// A key/value head's G query heads and the chunk's tokens make the rows of one
// product (row = t G + g), so K and V are read once for all of them.  HBM (or
// L2) bandwidth bounds it: each CTA takes 8 or 16 rows and a range of keys, its
// warps blocks of 16 keys in turn, through a ring of three blocks a warp (or two:
// takes_second) in shared memory.
// The products are S^T = K Q^T and O^T = V^T P^T: keys, then head dimensions,
// fill the 16 rows of the MMA and the few query rows its 8 columns, so no lane
// of a single-token call's MMA is spent on rows that do not exist twice over.
// The contraction order is free, so a lane's share of a key is 16-byte loads of
// consecutive elements, and 8-bit codes are widened exactly in registers, keys to
// f16 and values to bf16 (their scales multiply the scores and the probabilities).
//
// One token of 32 heads, 8 key heads of 128: 1000 keys 5.3 us on the GPU (latency: 8
// ranges in clusters); 64 sequences of 4000 to 8000 keys 226 us in bf16, of up to 8192 155
// us in 8 bits, 5.4 TB/s.  With the next block in registers in place of the ring: 239 and
// 205; 64 of 1000 45 us in bf16, now 34, in 8 bits 40 and 29; one of 4000 in bf16 9.7
// and 7.7; heads of 64 in bf16, 64 of 1000, 24.0 and 19.5.
//
// Up to eight ranges of keys are the CTAs of a cluster, which join them from each
// other's shared memory; more are joined through the workspace by the CTA that
// finishes last (a counter per row tile).  Both in the order of the ranges: the
// result does not depend on which CTA that is.
//
// What the modes add (AttnMode): a group's prefix gives the rows' unnormalised
// shares, the sequences' own keys are joined with them, and a weighed call also
// writes every score, from which whoever knows the rows' maxima and sums at the end
// has the weights of a key without reading it again.
#pragma once

#include <type_traits>

#include "attn_common.cuh"
#include "mma_frag.cuh"
#include "tc_ptx.cuh"
#include "tc_warp.cuh"
#include "tokens.cuh"

namespace cbs {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps, kBlock = 16;   // keys a warp takes at a time

__device__ __forceinline__ bool not_finite_pair(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// CTAs an SM and blocks of a warp's ring.  The first form has three blocks and as many
// CTAs as then fit (attn_rows_ctas); the second one, where there is one, these.
constexpr int kRingStages = 3;
struct Fit { int ctas, stages; };
template <int D, bool I8, int NR>
constexpr Fit kSecond = I8 ? (D == 64 ? Fit{0, 0} : Fit{NR == 1 ? 3 : 2, 3}) : D == 128 ? Fit{3, 2} : Fit{5, 2};

// Which form a call takes (the results are the same).  bf16: one CTA more an SM, where that
// saves a round of them.  One token of 32 heads, 8 key heads, first / second form in us: heads
// of 128, 48 sequences (384 CTAs, two rounds and one) of 30 keys 5.9/3.8, of 500 18.3/15.4, 80
// (640, three and two) 8.3/6.3 and 33.5/30.5, but 64 (512, two and two) of 500 25.4/28.4; heads
// of 64, 80 of 30 and 500 (two and one) 5.2/3.7 and 14.1/10.9.  8 bits, heads of 128: one CTA
// fewer with more registers, where both have one round of them and that many an SM: 48 of 500
// 16.4/13.3, but 32 10.9/13.0 and 64 16.7/18.4; tiles of 16 rows, four tokens a sequence, 30
// (240 CTAs) of 1000 28.8/21.1.
template <int D, bool I8, int NR>
bool takes_second(long long ctas) {
    const long long sms = current_device_sms();
    if (I8) return ctas <= kSecond<D, I8, NR>.ctas * sms && (NR == 2 || ctas > 2 * sms);
    const auto rounds = [&](int per_sm) { return (ctas + per_sm * sms - 1) / (per_sm * sms); };
    return rounds(kSecond<D, I8, NR>.ctas) < rounds(attn_rows_ctas(D, I8, 8));
}

template <int D, bool I8>
struct KvFrag {
    // K: chunks of 16 bytes a lane and key (32 dimensions of bf16 or 64 of int8
    // across the four lanes of a key); two keys (g, g + 8) a lane.
    static constexpr int kKC = D * (I8 ? 1 : 2) / 64;
    // V: words a lane and key; four keys (2j, 2j+1, 2j+8, 2j+9) a lane.
    static constexpr int kVW = D * (I8 ? 1 : 2) / 32;
    uint4 k[2][kKC];
    uint32_t v[4][kVW];
    float ks[2], vs[2];
};

// A warp's ring of blocks in shared memory, filled by its lanes' asynchronous copies.  A
// block's 16 rows of K, of V, then the scales of both; rows of 256 bytes as two panels
// of 128; 16-byte units are permuted within 128 bytes, so that V's reads of eight lanes
// meet all banks.
template <int D, bool I8, int STAGES>
struct KvRing {
    static constexpr int kRow = D * (I8 ? 1 : 2), kStages = STAGES, kRows = kBlock * kRow, kStage = 2 * kRows + (I8 ? 128 : 0), kWarp = kStages * kStage;
    static constexpr int kPart = kRow == 256 ? 128 : kRow, kPanel = kBlock * 128;   // of a row; of a block
    using F = KvFrag<D, I8>;
    int put[4], k_at, v_at[2];   // of a lane
    __device__ __forceinline__ explicit KvRing(int lane) {
        const int g = lane >> 2, j = lane & 3;
        if constexpr (kRow == 256) {
            #pragma unroll
            for (int i = 0; i < 4; ++i) put[i] = ((lane >> 3) & 1) * kPanel + (lane >> 4) * 128 + (((lane & 7) ^ ((2 * i + (lane >> 4)) & 7)) * 16);
        } else if constexpr (kRow == 128) {
            put[0] = put[2] = (lane >> 3) * 128 + (((lane & 7) ^ (lane >> 3)) * 16);
            put[1] = put[3] = put[0] ^ 64;
        }
        if constexpr (kRow >= 128) {
            k_at = g * 128 + ((j ^ g) * 16);
            v_at[0] = 2 * j * 128 + ((g ^ (2 * j)) * 16);
            v_at[1] = (2 * j + 1) * 128 + ((g ^ (2 * j + 1)) * 16);
        } else {
            put[0] = put[1] = put[2] = put[3] = (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) * 16);
            k_at = g * 64 + ((j ^ (g >> 1)) * 16);
            v_at[0] = 2 * j * 64 + (((g >> 1) ^ j) * 16) + (g & 1) * 8;
            v_at[1] = v_at[0] + 64;
        }
    }
    // A block whose first row is row0 (a block lies within a page): in 8 bits all of it,
    // whose codes are numbers whatever they are; in bf16 what is not live is zeros.
    __device__ __forceinline__ void copy(const CacheArgs &c, size_t row0, unsigned live, uint32_t to, int lane) const {
        const char *k = static_cast<const char *>(c.k) + row0 * kRow + lane * 16, *v = static_cast<const char *>(c.v) + row0 * kRow + lane * 16;
#pragma unroll
        for (int i = 0; i < kRows / 512; ++i) {
            const uint32_t bytes = I8 || (live >> (i * (512 / kRow) + lane / (kRow / 16)) & 1) ? 16 : 0;
            ptx::cp_async_16(to + i * (512 * kPart / kRow) + put[i & 3], k + i * 512, bytes);
            ptx::cp_async_16(to + kRows + i * (512 * kPart / kRow) + put[i & 3], v + i * 512, bytes);
        }
        if constexpr (I8) {
            const float *sc = (lane < 16 ? c.k_scale : c.v_scale) + row0 + (lane & 15);
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + 2 * kRows + lane * 4), "l"(sc) : "memory");
        }
    }
    __device__ __forceinline__ void read_k(F &f, const unsigned char *at, int lane) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int q = 0; q < F::kKC; ++q)
                f.k[i][q] = *reinterpret_cast<const uint4 *>(at + i * 8 * kPart + (q >> 1) * kPanel + (k_at ^ ((q & 1) * 64)));
            if constexpr (I8) f.ks[i] = *reinterpret_cast<const float *>(at + 2 * kRows + ((lane >> 2) + 8 * i) * 4);
        }
    }
    __device__ __forceinline__ void read_v(F &f, const unsigned char *at, int lane) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned char *p = at + kRows + (i >> 1) * 8 * kPart + v_at[i & 1];
            if constexpr (kRow == 64) {
                const uint2 w = *reinterpret_cast<const uint2 *>(p);
                f.v[i][0] = w.x; f.v[i][1] = w.y;
            } else {
#pragma unroll
                for (int q = 0; q < F::kVW / 4; ++q) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(p + q * kPanel);
                    f.v[i][4 * q] = w.x; f.v[i][4 * q + 1] = w.y; f.v[i][4 * q + 2] = w.z; f.v[i][4 * q + 3] = w.w;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < (I8 ? 2 : 0); ++i) f.vs[i] = *reinterpret_cast<const float *>(at + 2 * kRows + 64 + ((lane >> 2) + 8 * i) * 4);
    }
};

template <int D, bool I8, int NR, int MODE, bool SECOND>
__global__ void __launch_bounds__(kThreads, SECOND ? kSecond<D, I8, NR>.ctas : attn_rows_ctas(D, I8, 8 * NR)) attn_rows_kernel(const AttnLaunch L) {
    constexpr int kRows = 8 * NR;
    constexpr int kMT = D / 16;              // 16-dimension tiles of O^T
    using F = KvFrag<D, I8>;
    // The warps' shares at the end, each where the warp's ring was.
    using Ring = KvRing<D, I8, SECOND ? kSecond<D, I8, NR>.stages : kRingStages>;
    constexpr int kPitch = D + 4, kShare = Ring::kWarp / 4;
    static_assert(kShare >= kRows * kPitch, "a share fits where the ring was");
    extern __shared__ __align__(128) unsigned char s_ring[];
    float *const s_o = reinterpret_cast<float *>(s_ring);
    const auto share = [&](int w, int r, int dim) { return s_o + w * kShare + r * kPitch + dim; };
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
    __shared__ float2 s_stat[kRows];   // a range's (maximum, sum), for the other CTAs of a cluster
    // kAttnWeighed: sums of the probabilities before they are rounded (in 8 bits s_l has those).
    constexpr bool kExact = MODE == kAttnWeighed;
    __shared__ float s_x[kExact ? kWarps : 1][kRows], s_statx[kExact ? kRows : 1];
    __shared__ float2 s_fin[kExact ? kRows : 1];   // the rows' maxima and 1 / sums over all ranges
    __shared__ int s_flag;
    begin_attention<MODE>();
    ptx::griddep_launch_dependents();

    const CacheArgs &c = L.c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, j = lane & 3;
    const int b = blockIdx.z, head = blockIdx.y % c.kv_heads, rt = blockIdx.y / c.kv_heads;
    const Rows rs = rows_of<MODE>(L, b, head, D);
    const int R = rs.R, r0 = rt * kRows, len = rs.len, base = rs.base;
    // CTAs of one cluster meet twice at the end, and none leaves before: what is read
    // there is still some CTA's, even if the lengths change meanwhile.
    const auto leave = [&] {
        end_attention<MODE>();
        if (L.cluster) {
            cluster_sync();
            cluster_sync();
        }
    };
    if (r0 >= R) return leave();
    const int t_lo = Rows::token(L, r0), t_hi = Rows::token(L, min(R, r0 + kRows) - 1);
    // Keys that some row of the tile sees, in blocks of 16 from a multiple of 16.
    const int lo = seen_by(base + t_lo, len, L.causal, L.window).lo;
    const int hi = seen_by(base + t_hi, len, L.causal, L.window).hi;
    const int lo16 = lo & ~(kBlock - 1);
    const int blocks = hi > lo ? (hi - lo16 + kBlock - 1) / kBlock : 0;
    const int per = (blocks + L.split - 1) / L.split;
    const int active = per ? (blocks + per - 1) / per : 1;   // ranges that hold keys (one for none)
    const int sp = blockIdx.x;
    if (sp >= active) return leave();
    const int b0 = sp * per, b1 = min(blocks, b0 + per);
    // From here on every key below is seen by every row: no masks.
    const int all_lo = seen_by(base + t_hi, len, L.causal, L.window).lo;
    const int all_hi = seen_by(base + t_lo, len, L.causal, L.window).hi;

    if (tid == 0) s_flag = 0;
    __syncthreads();

    // Q: column g of each 8-row tile, this lane's dimensions (those of its K loads).
    uint32_t q[NR][D / 8];
    float q_back[NR][2];   // 8 bits: what rows 2 j and 2 j + 1 were multiplied with, taken back
    Seen seen[NR][2];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const int r = r0 + n * 8 + g;
        const __nv_bfloat16 *p = rs.query(L, r, D);
#pragma unroll
        for (int u = 0; u < D / 32; ++u) {   // 16-byte units of this lane
            const int dim = I8 ? (u >> 1) * 64 + j * 16 + (u & 1) * 8 : u * 32 + j * 8;
            const uint4 w = r < R ? __ldg(reinterpret_cast<const uint4 *>(p + dim)) : make_uint4(0, 0, 0, 0);
            q[n][4 * u] = w.x; q[n][4 * u + 1] = w.y; q[n][4 * u + 2] = w.z; q[n][4 * u + 3] = w.w;
        }
        if constexpr (I8) {
            // Codes widen to f16 with fewer instructions than to bf16, so the queries
            // are f16 here, a row's largest moved to 2^14 by a power of two: exact but
            // for values below 2^-28 of it, which keep an error of 2^-39 of it.  (By
            // 2^126 at most, whose reciprocal is a normal float.)
            float top = 0.0f;
#pragma unroll
            for (int u = 0; u < D / 8; ++u)
                top = fmaxf(top, fmaxf(fabsf(__uint_as_float(q[n][u] << 16)), fabsf(__uint_as_float(q[n][u] & 0xffff0000u))));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
            const int up = top > 0.0f ? min(268 - (int)(__float_as_uint(top) >> 23), 253) : 127;   // exponents with their bias
            const float by = __int_as_float(up << 23), back = __int_as_float((254 - up) << 23);
#pragma unroll
            for (int u = 0; u < D / 8; ++u)
                q[n][u] = frag::pack_half(__uint_as_float(q[n][u] << 16) * by, __uint_as_float(q[n][u] & 0xffff0000u) * by);
#pragma unroll
            for (int i = 0; i < 2; ++i) q_back[n][i] = __shfl_sync(~0u, back, (2 * j + i) * 4);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) seen[n][i] = rs.seen(L, r0 + n * 8 + 2 * j + i);
    }

    float o[NR][kMT][4], m[NR][2], l[NR][2], lx[kExact ? NR : 1][2] = {};
#pragma unroll
    for (int n = 0; n < NR; ++n) {
#pragma unroll
        for (int t = 0; t < kMT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][t][i] = 0.0f;
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.0f;
    }

    // A block's first row in the pool, and which of its 16 keys are live.
    auto place_of = [&](int blk, unsigned &live) -> size_t {
        live = 0;
        if (blk >= b1) return 0;
        const int pos = lo16 + blk * kBlock;
        const int p = page_of(c, b, pos);
        if (p < 0) return 0;
        const int first = max(lo - pos, 0), last = min(hi - pos, kBlock);
        live = ((1u << last) - 1u) & ~((1u << first) - 1u);
        return (((size_t)p * c.kv_heads + head) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
    };

    float *scores[kExact ? NR : 1][2];   // of this lane's rows
    if constexpr (kExact) {
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                scores[n][i] = L.scores + (((size_t)b * c.kv_heads + head) * L.rows_pad + r0 + n * 8 + 2 * j + i) * L.len_pad;
    }

    F f;
    int blk = b0 + warp;
    unsigned live_next;   // of the next block to load; `coming`: of those on their way, the first one's first
    constexpr int kAhead = Ring::kStages - 1;
    const Ring ring(lane);
    const unsigned char *const ring_at = s_ring + warp * Ring::kWarp;
    const uint32_t ring_to = ptx::smem_u32(ring_at);
    unsigned coming[kAhead];
    int stage = 0;   // bytes
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const size_t row = place_of(blk + i * kWarps, coming[i]);
        if (I8 ? coming[i] != 0 : blk + i * kWarps < b1) ring.copy(c, row, coming[i], ring_to + i * Ring::kStage, lane);
        ptx::cp_async_commit();
    }
    size_t row_next = place_of(blk + kAhead * kWarps, live_next);
    bool poison = false;
    while (blk < b1) {
        const int pos = lo16 + blk * kBlock;
        // This block has arrived, and every lane is done with the one before.
        ptx::cp_async_wait<kAhead - 1>();
        __syncwarp();
        if (I8 ? live_next != 0 : blk + kAhead * kWarps < b1)
            ring.copy(c, row_next, live_next, ring_to + (stage ? stage - Ring::kStage : kAhead * Ring::kStage), lane);
        ptx::cp_async_commit();
        const unsigned now = coming[0];
#pragma unroll
        for (int i = 0; i + 1 < kAhead; ++i) coming[i] = coming[i + 1];
        coming[kAhead - 1] = live_next;
        row_next = place_of(blk + (kAhead + 1) * kWarps, live_next);
        ring.read_k(f, ring_at + stage, lane);
        // ---- S^T = K Q^T
        float s[NR][4];
#pragma unroll
        for (int n = 0; n < NR; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
        for (int u = 0; u < F::kKC; ++u) {
            const uint32_t ka[4] = {f.k[0][u].x, f.k[0][u].y, f.k[0][u].z, f.k[0][u].w};
            const uint32_t kb[4] = {f.k[1][u].x, f.k[1][u].y, f.k[1][u].z, f.k[1][u].w};
            if constexpr (I8) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t a0, a1, a2, a3;
                    frag::i8_halves(ka[w], a0, a2);
                    frag::i8_halves(kb[w], a1, a3);
#pragma unroll
                    for (int n = 0; n < NR; ++n)
                        frag::mma_half(s[n], a0, a1, a2, a3, q[n][u * 8 + w * 2], q[n][u * 8 + w * 2 + 1]);
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int n = 0; n < NR; ++n)
                        frag::mma(s[n], ka[2 * h], kb[2 * h], ka[2 * h + 1], kb[2 * h + 1], q[n][u * 4 + 2 * h],
                                  q[n][u * 4 + 2 * h + 1]);
            }
        }
        const float ks0 = I8 ? f.ks[0] * L.scale_log2 : L.scale_log2, ks1 = I8 ? f.ks[1] * L.scale_log2 : L.scale_log2;

        // ---- scores, in base 2; keys a row does not see become -inf
        const bool partial = now != 0xffffu || pos < all_lo || pos + kBlock > all_hi;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            // (A key's scale and the row's power of two first: their product is of
            // ordinary size where the score is, the sum with one of them may not be.)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float ks = i < 2 ? ks0 : ks1;
                s[n][i] = __fmul_rn(s[n][i], I8 ? ks * q_back[n][i & 1] : ks);   // rounded, as the maximum is
            }
        }
        if (partial) {
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int off = g + 8 * (i >> 1), key = pos + off;
                    const Seen &z = seen[n][i & 1];
                    if (!((now >> off) & 1) || key < z.lo || key >= z.hi) s[n][i] = -INFINITY;
                }
        }
        if constexpr (kExact) {
            // Every score that some row sees, as it is: eight lanes' consecutive keys of a row.
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = r0 + n * 8 + 2 * j + (i & 1), key = pos + g + 8 * (i >> 1);
                    if (r < R && key < L.len_pad) scores[n][i & 1][key] = s[n][i];
                }
        }
        ring.read_v(f, ring_at + stage, lane);
        // ---- running maximum
        float top[NR][2];
        bool grow = false;
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                top[n][i] = fmaxf(s[n][i], s[n][2 + i]);
                grow |= top[n][i] > m[n][i] + kLazy;   // also from m = -inf
            }
        if (__any_sync(~0u, grow)) {
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float t = fmaxf(top[n][i], m[n][i]);
                    t = fmaxf(t, __shfl_xor_sync(~0u, t, 4));
                    t = fmaxf(t, __shfl_xor_sync(~0u, t, 8));
                    t = fmaxf(t, __shfl_xor_sync(~0u, t, 16));
                    const float fac = t == -INFINITY ? 1.0f : frag::ex2(m[n][i] - t);
                    m[n][i] = t;
                    l[n][i] *= fac;
                    if constexpr (kExact) lx[n][i] *= fac;
#pragma unroll
                    for (int d = 0; d < kMT; ++d) {
                        o[n][d][i] *= fac;
                        o[n][d][2 + i] *= fac;
                    }
                }
        }
        // ---- probabilities, as the columns of P^T
        uint32_t p0[NR], p1[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            float p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float mm = m[n][i & 1] == -INFINITY ? 0.0f : m[n][i & 1];
                p[i] = frag::ex2(s[n][i] - mm);
                if constexpr (kExact) lx[n][i & 1] += p[i];
                if (I8) {
                    l[n][i & 1] += p[i];
                    // a masked key's scale may be anything
                    p[i] = s[n][i] == -INFINITY ? 0.0f : p[i] * f.vs[i >> 1];
                }
            }
            // Rounded to bf16 for the second product: half a unit in 2^-8 of
            // each term, of either sign, below the output's own rounding.  The sum
            // that divides is of the rounded ones, so that the weights add up to one;
            // in 8 bits they carry the values' scales, so it is of the probabilities
            // before them, and the weights add up to one within 2^-8.
            const uint32_t w0 = frag::pack_bf16(p[0], p[1]), w1 = frag::pack_bf16(p[2], p[3]);
            if (!I8) {
                l[n][0] = frag::add_bf16(frag::add_bf16(l[n][0], w0), w1);
                l[n][1] = frag::add_bf16(frag::add_bf16(l[n][1], w0 >> 16), w1 >> 16);
            }
            p0[n] = frag::transpose8x8(w0);
            p1[n] = frag::transpose8x8(w1);
        }
        // ---- O^T += V^T P^T
        if (!I8 && partial) {
            // A value that some rows must not see would reach them as 0 x inf.
            bool bad = false;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int w = 0; w < F::kVW; ++w) bad |= not_finite_pair(f.v[i][w]);
            poison |= bad;
        }
#pragma unroll
        for (int w = 0; w < F::kVW; ++w) {
            if constexpr (I8) {
                // a word holds four dimensions: two tiles of O^T
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t s0 = h ? 0x6622u : 0x4400u, s1 = h ? 0x7733u : 0x5511u;
                    const uint32_t a0 = frag::i8_pair(__byte_perm(f.v[0][w], f.v[1][w], s0));
                    const uint32_t a1 = frag::i8_pair(__byte_perm(f.v[0][w], f.v[1][w], s1));
                    const uint32_t a2 = frag::i8_pair(__byte_perm(f.v[2][w], f.v[3][w], s0));
                    const uint32_t a3 = frag::i8_pair(__byte_perm(f.v[2][w], f.v[3][w], s1));
#pragma unroll
                    for (int n = 0; n < NR; ++n) frag::mma(o[n][2 * w + h], a0, a1, a2, a3, p0[n], p1[n]);
                }
            } else {
                const uint32_t a0 = __byte_perm(f.v[0][w], f.v[1][w], 0x5410), a1 = __byte_perm(f.v[0][w], f.v[1][w], 0x7632);
                const uint32_t a2 = __byte_perm(f.v[2][w], f.v[3][w], 0x5410), a3 = __byte_perm(f.v[2][w], f.v[3][w], 0x7632);
#pragma unroll
                for (int n = 0; n < NR; ++n) frag::mma(o[n][w], a0, a1, a2, a3, p0[n], p1[n]);
            }
        }
        stage = stage == kAhead * Ring::kStage ? 0 : stage + Ring::kStage;
        blk += kWarps;
    }
    if (poison) s_flag = 1;
    __syncwarp();   // the ring's place becomes the share's

    // ---- the warps' shares, joined in shared memory
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float t = l[n][i];
            t += __shfl_xor_sync(~0u, t, 4);
            t += __shfl_xor_sync(~0u, t, 8);
            t += __shfl_xor_sync(~0u, t, 16);
            const int r = n * 8 + 2 * j + i;
            if (g == 0) {
                s_m[warp][r] = m[n][i];
                s_l[warp][r] = t;
            }
            if constexpr (kExact) {
                float x = lx[n][i];
                x += __shfl_xor_sync(~0u, x, 4);
                x += __shfl_xor_sync(~0u, x, 8);
                x += __shfl_xor_sync(~0u, x, 16);
                if (g == 0) s_x[warp][r] = x;
            }
            // dimension of tile t2's rows g and g + 8: see the V loads
#pragma unroll
            for (int d = 0; d < kMT; ++d) {
                const int dim = I8 ? g * (D / 8) + 2 * d : (d >> 2) * 64 + g * 8 + 2 * (d & 3);
                share(warp, r, dim)[0] = o[n][d][i];
                share(warp, r, dim)[1] = o[n][d][2 + i];
            }
        }
    __syncthreads();

    if (!I8 && s_flag) {
        // Slow and sure: a masked block of this range holds a value that is not
        // finite.  Each row by itself, over the keys it sees.
        constexpr int kE = D / 32;   // dimensions a lane
        for (int r = warp; r < kRows && r0 + r < R; r += kWarps) {
            float acc[kE], mm, ll;
            slow_row<D, false, kExact>(L, rs, b, r0 + r, lo16 + b0 * kBlock, lo16 + b1 * kBlock, lane, acc, mm, ll);
#pragma unroll
            for (int e = 0; e < kE; ++e) *share(0, r, lane * kE + e) = acc[e];
            if (lane < kWarps) {
                s_m[lane][r] = lane == 0 ? mm : -INFINITY;
                s_l[lane][r] = lane == 0 ? ll : 0.0f;
                if constexpr (kExact) s_x[lane][r] = lane == 0 ? ll : 0.0f;
            }
        }
        __syncthreads();
    }

    end_attention<MODE>();   // the prefix's shares
    const int tile = (b * c.kv_heads + head) * L.row_tiles + rt;
    constexpr int kU = D / 4;   // units of four dimensions
    for (int i = tid; i < kRows * kU; i += kThreads) {
        const int r = i / kU, u = i % kU;
        if (r0 + r >= R) break;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float sum = 0.0f, exact = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float fac = share_factor(s_m[w][r], s_l[w][r], top);
            if (s_m[w][r] == -INFINITY && fac == 0.0f) continue;
            const float4 v = *reinterpret_cast<const float4 *>(share(w, r, 4 * u));
            acc.x = fmaf(v.x, fac, acc.x); acc.y = fmaf(v.y, fac, acc.y);
            acc.z = fmaf(v.z, fac, acc.z); acc.w = fmaf(v.w, fac, acc.w);
            sum = fmaf(s_l[w][r], fac, sum);
            if constexpr (kExact) exact = fmaf(s_x[w][r], fac, exact);
        }
        if (active == 1) {
            store_out4<MODE>(L, rs, r0 + r, D, 4 * u, acc, sum, top, exact);
            if constexpr (kExact) {
                const Seen z = rs.seen(L, r0 + r);
                if (u == 0) s_fin[r] = row_stats(z.hi > z.lo, top, exact);
            }
        } else if (L.cluster) {   // (a unit's own place, which nobody else has read)
            *reinterpret_cast<float4 *>(share(0, r, 4 * u)) = acc;
            if (u == 0) s_stat[r] = make_float2(top, sum);
            if constexpr (kExact)
                if (u == 0) s_statx[r] = exact;
        } else {
            const size_t at = ((size_t)tile * L.split + sp) * kRows + r;
            *reinterpret_cast<float4 *>(L.partial + at * D + 4 * u) = acc;
            if (u == 0) L.stats[at] = make_float2(top, sum);
            if constexpr (kExact)
                if (u == 0) L.sums[at] = exact;
        }
    }
    // A weighed call's keys [from, to): the rows' statistics are in s_fin.
    const auto weigh = [&](int from, int to) {
        __syncthreads();
        for (int key = from + 4 * tid; key < to; key += 4 * kThreads)
            store_four(L, rs, b, key, to, weigh_four(L, rs, b, key, 0, 4, [&](int r) { return s_fin[r]; }));
    };
    const int end = min(len, L.len_pad);   // (of a weighed call)
    if (kExact && L.fused && sp == 0 && tid == 0 && len > L.len_pad) atomicOr(c.status, kStatusBadIndex);
    if (!L.cluster) {
        const bool mine = active == 1 || join_ranges<D, kRows, kThreads, MODE>(L, rs, tile, r0, active, tid, &s_flag, s_fin);
        if constexpr (kExact)
            if (L.fused && mine) weigh(0, end);
        return;
    }
    // The ranges of a cluster, in their order, from the CTAs' shared memory: each
    // CTA finishes some of the units.
    __syncthreads();
    cluster_sync();
    if constexpr (kExact) {
        if (L.fused && active > 1 && tid < R) {   // (one tile of rows)
            const uint32_t at = ptx::smem_u32(&s_stat[tid]), x_at = ptx::smem_u32(&s_statx[tid]);
            float2 st[kAttnClusterMost];
            float sx[kAttnClusterMost], top = -INFINITY, exact = 0.0f;
#pragma unroll
            for (int x = 0; x < kAttnClusterMost; ++x)
                if (x < active) st[x] = ld_cluster2(at, x), sx[x] = ld_cluster1(x_at, x);
#pragma unroll
            for (int x = 0; x < kAttnClusterMost; ++x)
                if (x < active) top = fmaxf(top, st[x].x);
#pragma unroll
            for (int x = 0; x < kAttnClusterMost; ++x) {
                if (x >= active) break;
                const float fac = share_factor(st[x].x, st[x].y, top);
                if (!(st[x].x == -INFINITY && fac == 0.0f)) exact = fmaf(sx[x], fac, exact);
            }
            const Seen z = rs.seen(L, tid);
            s_fin[tid] = row_stats(z.hi > z.lo, top, exact);
        }
    }
    if (active > 1) {
        for (int i = sp * kThreads + tid; i < kRows * kU; i += active * kThreads) {
            const int r = i / kU, u = i % kU;
            if (r0 + r >= R) break;
            const uint32_t o_at = ptx::smem_u32(share(0, r, 4 * u)), s_at = ptx::smem_u32(&s_stat[r]);
            float2 st[kAttnClusterMost];
            float4 v[kAttnClusterMost];
            float top = -INFINITY, sum = 0.0f, exact = 0.0f;
#pragma unroll
            for (int x = 0; x < kAttnClusterMost; ++x)
                if (x < active) st[x] = ld_cluster2(s_at, x), v[x] = ld_cluster4(o_at, x);
#pragma unroll
            for (int x = 0; x < kAttnClusterMost; ++x)
                if (x < active) top = fmaxf(top, st[x].x);
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int x = 0; x < kAttnClusterMost; ++x) {
                if (x >= active) break;
                const float fac = share_factor(st[x].x, st[x].y, top);
                if (st[x].x == -INFINITY && fac == 0.0f) continue;   // a range that saw nothing
                acc.x = fmaf(v[x].x, fac, acc.x); acc.y = fmaf(v[x].y, fac, acc.y);
                acc.z = fmaf(v[x].z, fac, acc.z); acc.w = fmaf(v[x].w, fac, acc.w);
                sum = fmaf(st[x].y, fac, sum);
                if constexpr (kExact)   // (a few-row call's own weights have it already)
                    if (!L.fused) exact = fmaf(ld_cluster1(ptx::smem_u32(&s_statx[r]), x), fac, exact);
            }
            store_out4<MODE>(L, rs, r0 + r, D, 4 * u, acc, sum, top, exact);
        }
    }
    __syncthreads();
    if constexpr (kExact) {   // each range's CTA its own keys, the first and the last also what nobody sees
        if (L.fused) weigh(sp == 0 ? 0 : lo16 + b0 * kBlock, sp == active - 1 ? end : min(end, lo16 + b1 * kBlock));
    }
    cluster_sync();   // nobody's rows go while another CTA reads them
}

template <int D, bool I8, int MODE>
cudaError_t launch_rows(const AttnLaunch &L, int row_tile, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(L.split, L.c.kv_heads * L.row_tiles, L.c.batch);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = (launch_options() & CBS_LAUNCH_PDL) ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = L.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = L.cluster ? 2 : 1;
    const auto launch = [&](auto kern, int smem, ContextOfDevice &set) {
        cfg.dynamicSmemBytes = smem;
        const cudaError_t e = set_max_dyn_smem_once(kern, smem, set);
        return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, kern, L);
    };
    const auto either = [&](auto tiles) {
        constexpr int NR = decltype(tiles)::value;
        constexpr Fit second = kSecond<D, I8, NR>;
        static ContextOfDevice set1, set2;
        if constexpr (MODE == kAttnPlain && second.ctas > 0)
            if (takes_second<D, I8, NR>((long long)cfg.gridDim.x * cfg.gridDim.y * cfg.gridDim.z))
                return launch(attn_rows_kernel<D, I8, NR, MODE, true>, kWarps * KvRing<D, I8, second.stages>::kWarp, set2);
        return launch(attn_rows_kernel<D, I8, NR, MODE, false>, kWarps * KvRing<D, I8, kRingStages>::kWarp, set1);
    };
    if constexpr (I8)
        if (row_tile == 16) return either(std::integral_constant<int, 2>{});
    return either(std::integral_constant<int, 1>{});
}

template <int MODE>
cudaError_t launch_attn_rows_as(const AttnLaunch &L, int row_tile, cudaStream_t s) {
    if (L.c.head_dim == 64) return L.c.int8 ? launch_rows<64, true, MODE>(L, row_tile, s) : launch_rows<64, false, MODE>(L, row_tile, s);
    return L.c.int8 ? launch_rows<128, true, MODE>(L, row_tile, s) : launch_rows<128, false, MODE>(L, row_tile, s);
}

}  // namespace

}  // namespace cbs
