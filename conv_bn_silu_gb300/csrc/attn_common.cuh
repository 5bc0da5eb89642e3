// attn_common.cuh -- what the attention kernels share: which keys a row sees,
// where its query and output lie, the slow path for values that are not
// finite, and the joining of ranges of keys.
#pragma once

#include "mma_frag.cuh"
#include "tc_ptx.cuh"
#include "tokens.cuh"

namespace cbs {

// The running maximum is raised only when a score passes it by more than this
// (base 2): p stays below 2^8, far inside float and bf16, and most blocks need
// neither an exchange between lanes nor a rescaling of the output.
constexpr float kLazy = 8.0f;

// What becomes of a row's softmax beside or in place of its output.
enum AttnMode {
    kAttnPlain = 0,
    kAttnPrefix = 1,   // a group's prefix: the rows' shares go to L.share, unnormalised
    kAttnOwn = 2,      // the sequences' own keys: joined with those shares
    kAttnBeside = 4,   // the sequences' own keys, their shares left for a kernel that joins both
    kAttnWeighed = 3   // the output, and each row's (maximum, 1 / sum) to L.row_stats
};

// Until what a call reads is there.  The sequences' own part begins while their
// prefixes' part, the kernel before it, still runs.  All that it reads and writes but
// the shares is older: it is launched once every CTA of the prefixes' part has let it,
// which they do after their own wait for the kernels before.  The fence drops what this
// SM's L1 held until then.  (A kernel's own griddepcontrol.wait is all that the programming
// model names as making older writes visible.  That the fence does it here rests on the
// chip: those kernels have ended, so their writes are in L2, and loads after the fence come
// from there.  With the wait at the start the two parts would not overlap.)
constexpr bool runs_beside(int mode) { return mode == kAttnOwn || mode == kAttnBeside; }
template <int MODE>
__device__ __forceinline__ void begin_attention() {
    if constexpr (runs_beside(MODE)) __threadfence();
    else ptx::griddep_wait();
}
// Before the shares are read (kAttnOwn), and before a CTA ends: what comes after this
// kernel has to come after both parts.  One waiting CTA is enough for that; with
// kAttnBeside the others make room for the next.
template <int MODE>
__device__ __forceinline__ void end_attention() {
    if constexpr (MODE == kAttnOwn) ptx::griddep_wait();
    if constexpr (MODE == kAttnBeside)
        if (blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1 && blockIdx.z == gridDim.z - 1) ptx::griddep_wait();
}

// Keys [lo, hi) are what a row at `place` sees of a sequence.
struct Seen { int lo, hi; };
__device__ __forceinline__ Seen seen_by(int place, int len, int causal, int window) {
    Seen s;
    s.hi = causal ? min(len, place + 1) : len;
    s.lo = window && window <= place ? place - window + 1 : 0;
    return s;
}

// One sequence's rows of one key/value head: row r is token r / G of the
// chunk, query head head * G + r % G.
struct Rows {
    int start, fresh, R, len, base, head;   // first new token, how many, rows; length, first place
    static __device__ __forceinline__ int token(const AttnLaunch &L, int r) {
        return L.group > 1 ? (int)__umulhi((unsigned)r, L.group_magic) : r;
    }
    __device__ __forceinline__ Seen seen(const AttnLaunch &L, int r) const {
        return seen_by(base + token(L, r), len, L.causal, L.window);
    }
    __device__ __forceinline__ const __nv_bfloat16 *query(const AttnLaunch &L, int r, int D) const {
        const int t = token(L, r);
        return static_cast<const __nv_bfloat16 *>(L.q) + (size_t)(start + t) * L.q_stride + (size_t)(head * L.group + r - t * L.group) * D;
    }
    // Of all (token, query head) rows of the call, this one's number.
    __device__ __forceinline__ size_t number(const AttnLaunch &L, int r) const {
        const int t = token(L, r);
        return (size_t)(start + t) * L.heads + head * L.group + r - t * L.group;
    }
    __device__ __forceinline__ __nv_bfloat16 *out(const AttnLaunch &L, int r, int D) const {
        const int t = token(L, r);
        return static_cast<__nv_bfloat16 *>(L.out) + (size_t)(start + t) * L.out_stride + (size_t)(head * L.group + r - t * L.group) * D;
    }
};

// Tokens from `end` on belong to no sequence: zeros, from the CTAs of the last
// sequence together.
__device__ __forceinline__ void zero_padding(const AttnLaunch &L, int end, int D) {
    const int units = L.heads * D / 8;   // of 16 bytes, a token
    const long long all = (long long)(L.c.total - end) * units, step = (long long)gridDim.x * gridDim.y * blockDim.x;
    for (long long i = ((long long)blockIdx.y * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x; i < all; i += step) {
        const int t = (int)(i / units);
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(L.out) + (size_t)(end + t) * L.out_stride + (size_t)(i - (long long)t * units) * 8) =
            make_uint4(0, 0, 0, 0);
    }
}

// The rows of sequence b, its starts within the call's tokens and its chunk
// within the plan's (the status bit otherwise).  Behind the last sequence's
// tokens, the padding.
// (kAttnPrefix: b is a group, its rows those of all its sequences.)
template <int MODE>
__device__ __forceinline__ Rows rows_of(const AttnLaunch &L, int b, int head, int D) {
    const CacheArgs &c = L.c;
    Rows s;
    int i0 = b, i1 = b + 1;
    if constexpr (MODE == kAttnPrefix) {
        const int g0 = L.group_start[b], g1 = L.group_start[b + 1];
        i0 = max(0, min(g0, L.sequences));
        i1 = max(i0, min(g1, L.sequences));
        if ((i0 != g0 || i1 != g1 || (b == 0 && g0 != 0) || (b == c.batch - 1 && g1 != L.sequences)) && threadIdx.x == 0)
            atomicOr(c.status, kStatusBadIndex);
    }
    const int s0 = c.new_start[i0], s1 = c.new_start[i1];
    s.len = seq_len(c, b);
    s.start = max(0, min(s0, c.total));
    const int end = max(s.start, min(s1, c.total));
    s.fresh = end - s.start;
    if (s.start != s0 || end != s1 || s.fresh > L.max_new || (i0 == 0 && s0 != 0)) {
        if (threadIdx.x == 0) atomicOr(c.status, kStatusBadIndex);
        s.fresh = min(s.fresh, L.max_new);
    }
    if (MODE != kAttnPrefix && b == c.batch - 1 && end < c.total) zero_padding(L, end, D);
    s.R = s.fresh * L.group;
    s.head = head;
    s.base = s.len - s.fresh;
    return s;
}

// A share of a row's softmax: (maximum, sum) and the unnormalised output.  A
// share without a visible key has maximum -inf and sum zero, and adds nothing
// (its output may hold anything); a NaN score leaves the sum NaN, which stays.
__device__ __forceinline__ float share_factor(float m, float l, float top) {
    if (m == -INFINITY) return l == 0.0f ? 0.0f : 1.0f;
    return frag::ex2(m - top);
}

// A prefix's share and a row's own of the same dimensions, joined into acc and sum;
// false where neither saw a key.
__device__ __forceinline__ bool join_shares(float2 pre, float4 pre_acc, float2 own, float4 &acc, float &sum) {
    const float both = fmaxf(own.x, pre.x), mine = share_factor(own.x, own.y, both), theirs = share_factor(pre.x, pre.y, both);
    const bool no_own = own.x == -INFINITY && mine == 0.0f, no_pre = pre.x == -INFINITY && theirs == 0.0f;
    acc = no_own ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : make_float4(acc.x * mine, acc.y * mine, acc.z * mine, acc.w * mine);
    sum = no_own ? 0.0f : own.y * mine;
    if (!no_pre) {
        acc.x = fmaf(pre_acc.x, theirs, acc.x); acc.y = fmaf(pre_acc.y, theirs, acc.y);
        acc.z = fmaf(pre_acc.z, theirs, acc.z); acc.w = fmaf(pre_acc.w, theirs, acc.w);
        sum = fmaf(pre.y, theirs, sum);
    }
    return !(no_own && no_pre);
}

// A weighed row's maximum and 1 / sum; zeros for a row that sees nothing.
__device__ __forceinline__ float2 row_stats(bool any, float top, float exact) {
    return any ? make_float2(top == -INFINITY ? 0.0f : top, __fdiv_rn(1.0f, exact)) : make_float2(0.0f, 0.0f);
}

// A key's weight: what it was (nothing, if the key is new or decay is 0), and what came.
__device__ __forceinline__ float weight_after(const AttnLaunch &L, const Rows &s, int key, float before, float came) {
    return (key < s.base && L.decay != 0.0f ? L.decay * before : 0.0f) + came;
}

// What the four keys from `key` on (a multiple of four) receive from rows first,
// first + 1, ... four at a time, every `step` after them, from the scores that the
// attention left.
template <typename Stats>
__device__ __forceinline__ float4 weigh_four(const AttnLaunch &L, const Rows &s, int b, int key, int first, int step, Stats stats_of) {
    const float *scores = L.scores + ((size_t)b * L.c.kv_heads + s.head) * L.rows_pad * L.len_pad + key;
    float sum[4] = {};
    constexpr int kOnce = 4;   // rows on their way together
    for (int r0 = first; r0 < s.R; r0 += step) {
        float4 v[kOnce];
        float2 st[kOnce];
        Seen z[kOnce];
#pragma unroll
        for (int x = 0; x < kOnce; ++x) {
            z[x] = r0 + x < s.R ? s.seen(L, r0 + x) : Seen{0, 0};
            if (z[x].hi <= key || z[x].lo >= key + 4) continue;
            st[x] = stats_of(r0 + x);
            v[x] = __ldcg(reinterpret_cast<const float4 *>(scores + (size_t)(r0 + x) * L.len_pad));
        }
#pragma unroll
        for (int x = 0; x < kOnce; ++x) {
            if (z[x].hi <= key || z[x].lo >= key + 4) continue;
            const float y[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (key + i >= z[x].lo && key + i < z[x].hi) sum[i] = fmaf(frag::ex2(y[i] - st[x].x), st[x].y, sum[i]);
        }
    }
    return make_float4(sum[0], sum[1], sum[2], sum[3]);
}

// What they weigh then, those before `end`.  (All four are on one page: pages hold
// multiples of sixteen.)
__device__ __forceinline__ void store_four(const AttnLaunch &L, const Rows &s, int b, int key, int end, float4 came) {
    const CacheArgs &c = L.c;
    const int p = page_of(c, b, key);
    if (p < 0) return;
    float *mass = L.mass + (((size_t)p * c.kv_heads + s.head) << c.page_shift) + (key & ((1 << c.page_shift) - 1));
    float4 before = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (L.decay != 0.0f) before = *reinterpret_cast<const float4 *>(mass);
    const float4 after = make_float4(weight_after(L, s, key, before.x, came.x), weight_after(L, s, key + 1, before.y, came.y),
                                     weight_after(L, s, key + 2, before.z, came.z), weight_after(L, s, key + 3, before.w, came.w));
    if (key + 4 <= end) {
        *reinterpret_cast<float4 *>(mass) = after;
    } else {
        mass[0] = after.x;
        if (key + 1 < end) mass[1] = after.y;
        if (key + 2 < end) mass[2] = after.z;
    }
}

// Four dimensions of a row's output: acc / sum, zeros for a row that sees nothing.
// `top`: the maximum that acc and sum are above; `exact`: kAttnWeighed, the sum of
// the probabilities before any rounding.
template <int MODE>
__device__ __forceinline__ void store_out4(const AttnLaunch &L, const Rows &s, int r, int D, int dim, float4 acc, float sum, float top,
                                           float exact) {
    if constexpr (MODE == kAttnPrefix || MODE == kAttnBeside) {
        const size_t row = s.number(L, r);
        if (dim == 0) L.share_stats[row] = make_float2(top, sum);
        *reinterpret_cast<float4 *>(L.share + row * D + dim) = acc;
        return;
    }
    const Seen z = s.seen(L, r);
    uint2 w = make_uint2(0u, 0u);
    bool any = z.hi > z.lo;
    if constexpr (MODE == kAttnOwn) {
        const size_t row = s.number(L, r);
        any = join_shares(__ldcg(&L.share_stats[row]), __ldcg(reinterpret_cast<const float4 *>(L.share + row * D + dim)),
                          any ? make_float2(top, sum) : make_float2(-INFINITY, 0.0f), acc, sum);
    }
    if constexpr (MODE == kAttnWeighed)
        if (dim == 0 && !L.fused) L.row_stats[s.number(L, r)] = row_stats(any, top, exact);
    if (any) {
        const float inv = __fdiv_rn(1.0f, sum);
        w.x = frag::pack_bf16(acc.x * inv, acc.y * inv);
        w.y = frag::pack_bf16(acc.z * inv, acc.w * inv);
    }
    *reinterpret_cast<uint2 *>(s.out(L, r, D) + dim) = w;
}

// Pairs of floats in one register pair (two lanes of one instruction).
struct F2 { unsigned long long v; };
__device__ __forceinline__ F2 pair(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ float2 split(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}

// Beyond 2^22 a float's last place is more than a quarter: a score's product with
// the scale, which the chunk kernels' passes do not round, may then lie far from the
// reference, which is rounded (from 2^31 on by 2^128 and more).  Such rows, seldom met,
// go the slow path.
__device__ __forceinline__ bool is_far(float m) { return fabsf(m) > 4194304.0f && fabsf(m) < INFINITY; }

// A row by itself over keys [k0, k1): what the kernels fall back to when a block
// that some rows must not see in full holds a value that is not finite (0 x inf
// would reach them; a bf16 cache), or when scores are too large for the fast
// pass.  A warp; lane holds D / 32 dimensions.  KEEP: its scores, which are summed up in
// another order than the fast pass does, to L.scores.
template <int D, bool I8, bool KEEP = false>
__device__ __noinline__ void slow_row(const AttnLaunch &L, const Rows &s, int b, int r, int k0, int k1, int lane,
                                      float (&acc)[D / 32], float &mm, float &ll) {
    constexpr int kE = D / 32;
    const CacheArgs &c = L.c;
    const __nv_bfloat16 *qp = s.query(L, r, D) + lane * kE;
    const Seen z = s.seen(L, r);
    float qv[kE];
    mm = -INFINITY;
    ll = 0.0f;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
        qv[e] = __bfloat162float(qp[e]);
        acc[e] = 0.0f;
    }
    const auto value = [&](const void *pool, size_t at) {
        if constexpr (I8) return (float)static_cast<const int8_t *>(pool)[at];
        else return __bfloat162float(static_cast<const __nv_bfloat16 *>(pool)[at]);
    };
    for (int key = max(z.lo, k0); key < min(z.hi, k1); ++key) {
        const int p = page_of(c, b, key);
        if (p < 0) continue;
        const size_t row = (((size_t)p * c.kv_heads + s.head) << c.page_shift) + (key & ((1 << c.page_shift) - 1));
        const size_t at = row * D + lane * kE;
        float dot = 0.0f;
#pragma unroll
        for (int e = 0; e < kE; ++e) dot = fmaf(qv[e], value(c.k, at + e), dot);
#pragma unroll
        for (int x = 16; x; x >>= 1) dot += __shfl_xor_sync(~0u, dot, x);
        dot = __fmul_rn(dot, I8 ? c.k_scale[row] * L.scale_log2 : L.scale_log2);   // rounded, as the maximum is
        if (KEEP && lane == 0 && key < L.len_pad)
            L.scores[(((size_t)b * c.kv_heads + s.head) * L.rows_pad + r) * L.len_pad + key] = dot;
        const float nm = fmaxf(mm, dot);
        const float use = nm == -INFINITY ? 0.0f : nm;
        const float fac = mm == -INFINITY ? 0.0f : frag::ex2(mm - use), pr = frag::ex2(dot - use);
        const float pv = I8 ? pr * c.v_scale[row] : pr;
        ll = ll * fac + pr;
#pragma unroll
        for (int e = 0; e < kE; ++e) acc[e] = acc[e] * fac + pv * value(c.v, at + e);
        mm = nm;
    }
}

// After a CTA has written its range's share of a tile (L.partial, L.stats):
// the CTA that comes last joins the ranges, in their order, so that the result
// does not depend on which one that is.  `flag`: a word of shared memory; `fin`: the
// rows' statistics there (kAttnWeighed).  Returns whether this CTA was the last.
template <int D, int kRows, int kThreads, int MODE>
__device__ __forceinline__ bool join_ranges(const AttnLaunch &L, const Rows &s, int tile, int r0, int active, int tid, int *flag,
                                            float2 *fin) {
    __threadfence();
    __syncthreads();
    if (tid == 0) {
        const unsigned before = atomicAdd(L.counters + tile, 1u);
        *flag = before == (unsigned)active - 1u;
        if (*flag) L.counters[tile] = 0u;   // ready for the next call
    }
    __syncthreads();
    if (!*flag) return false;
    __threadfence();
    constexpr int kU = D / 4;   // units of four dimensions
    for (int i = tid; i < kRows * kU; i += kThreads) {
        const int r = i / kU, u = i % kU;
        if (r0 + r >= s.R) break;
        const size_t at = (size_t)tile * L.split * kRows + r;
        float top = -INFINITY;
        for (int x = 0; x < active; ++x) top = fmaxf(top, __ldcg(&L.stats[at + (size_t)x * kRows]).x);
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float sum = 0.0f, exact = 0.0f;
        for (int x = 0; x < active; ++x) {
            const float2 st = __ldcg(&L.stats[at + (size_t)x * kRows]);
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(L.partial + (at + (size_t)x * kRows) * D + 4 * u));
            const float fac = share_factor(st.x, st.y, top);
            if (st.x == -INFINITY && fac == 0.0f) continue;
            acc.x = fmaf(v.x, fac, acc.x); acc.y = fmaf(v.y, fac, acc.y);
            acc.z = fmaf(v.z, fac, acc.z); acc.w = fmaf(v.w, fac, acc.w);
            sum = fmaf(st.y, fac, sum);
            if constexpr (MODE == kAttnWeighed) exact = fmaf(__ldcg(&L.sums[at + (size_t)x * kRows]), fac, exact);
        }
        store_out4<MODE>(L, s, r0 + r, D, 4 * u, acc, sum, top, exact);
        if constexpr (MODE == kAttnWeighed) {
            const Seen z = s.seen(L, r0 + r);
            if (u == 0) fin[r] = row_stats(z.hi > z.lo, top, exact);
        }
    }
    return true;
}

}  // namespace cbs
