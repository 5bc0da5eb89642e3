// attn_common.cuh -- what the attention kernels share: which keys a row sees,
// where its query and output lie, the slow path for values that are not
// finite, and the joining of ranges of keys.
#pragma once

#include "mma_frag.cuh"
#include "tokens.cuh"

namespace cbs {

// The running maximum is raised only when a score passes it by more than this
// (base 2): p stays below 2^8, far inside float and bf16, and most blocks need
// neither an exchange between lanes nor a rescaling of the output.
constexpr float kLazy = 8.0f;

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
__device__ __forceinline__ Rows rows_of(const AttnLaunch &L, int b, int head, int D) {
    const CacheArgs &c = L.c;
    Rows s;
    const int s0 = c.new_start[b], s1 = c.new_start[b + 1];
    s.len = seq_len(c, b);
    s.start = max(0, min(s0, c.total));
    const int end = max(s.start, min(s1, c.total));
    s.fresh = end - s.start;
    if (s.start != s0 || end != s1 || s.fresh > L.max_new || (b == 0 && s0 != 0)) {
        if (threadIdx.x == 0) atomicOr(c.status, kStatusBadIndex);
        s.fresh = min(s.fresh, L.max_new);
    }
    if (b == c.batch - 1 && end < c.total) zero_padding(L, end, D);
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

// Four dimensions of a row's output: acc / sum, zeros for a row that sees nothing.
__device__ __forceinline__ void store_out4(const AttnLaunch &L, const Rows &s, int r, int D, int dim, float4 acc, float sum) {
    const Seen z = s.seen(L, r);
    uint2 w = make_uint2(0u, 0u);
    if (z.hi > z.lo) {
        const float inv = __fdiv_rn(1.0f, sum);
        w.x = frag::pack_bf16(acc.x * inv, acc.y * inv);
        w.y = frag::pack_bf16(acc.z * inv, acc.w * inv);
    }
    *reinterpret_cast<uint2 *>(s.out(L, r, D) + dim) = w;
}

// A row by itself over keys [k0, k1): what the kernels fall back to when a block
// that some rows must not see in full holds a value that is not finite (0 x inf
// would reach them; a bf16 cache), or when scores are too large for the fast
// pass.  A warp; lane holds D / 32 dimensions.
template <int D, bool I8>
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
// does not depend on which one that is.  `flag`: a word of shared memory.
template <int D, int kRows, int kThreads>
__device__ __forceinline__ void join_ranges(const AttnLaunch &L, const Rows &s, int tile, int r0, int active, int tid, int *flag) {
    __threadfence();
    __syncthreads();
    if (tid == 0) {
        const unsigned before = atomicAdd(L.counters + tile, 1u);
        *flag = before == (unsigned)active - 1u;
        if (*flag) L.counters[tile] = 0u;   // ready for the next call
    }
    __syncthreads();
    if (!*flag) return;
    __threadfence();
    constexpr int kU = D / 4;   // units of four dimensions
    for (int i = tid; i < kRows * kU; i += kThreads) {
        const int r = i / kU, u = i % kU;
        if (r0 + r >= s.R) break;
        const size_t at = (size_t)tile * L.split * kRows + r;
        float top = -INFINITY;
        for (int x = 0; x < active; ++x) top = fmaxf(top, __ldcg(&L.stats[at + (size_t)x * kRows]).x);
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float sum = 0.0f;
        for (int x = 0; x < active; ++x) {
            const float2 st = __ldcg(&L.stats[at + (size_t)x * kRows]);
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(L.partial + (at + (size_t)x * kRows) * D + 4 * u));
            const float fac = share_factor(st.x, st.y, top);
            if (st.x == -INFINITY && fac == 0.0f) continue;
            acc.x = fmaf(v.x, fac, acc.x); acc.y = fmaf(v.y, fac, acc.y);
            acc.z = fmaf(v.z, fac, acc.z); acc.w = fmaf(v.w, fac, acc.w);
            sum = fmaf(st.y, fac, sum);
        }
        store_out4(L, s, r0 + r, D, 4 * u, acc, sum);
    }
}

}  // namespace cbs
