// k_tokens.cu -- RMS normalisation with the residual's addition and an 8-bit
// output, the seam back from rows in 8 bits, and the paged cache's write and
// read.  All of them move data once; HBM bandwidth bounds them.
#include <cuda_bf16.h>

#include "tc_ptx.cuh"
#include "tokens.cuh"

namespace cbs {

namespace {

// Code of x in a row of scale s: clamp(rne(x / s)), IEEE division as in the
// library's other quantisers.  A zero scale (a row of zeros, or one so small
// that max / 127 is zero) gives code 0, and so does a NaN.
//
// x times the reciprocal (within an ulp) is within 2^-15 of the quotient (|q| <=
// 127), so away from the halves between whole numbers both round to the same
// code; only a product that close to a half (or a scale whose reciprocal is
// infinite) pays for the division.  Adding 1.5 * 2^23 rounds to
// the nearest even whole number and leaves it in the sum's low byte.
struct RowScale {
    float s, inv;
    static __device__ __forceinline__ RowScale of(float scale) { return RowScale{scale, reciprocal(scale)}; }
    // (Infinite where it is too large or the scale subnormal: then no product is
    // near a whole number.)
    static __device__ __forceinline__ float reciprocal(float x) {
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
        return r;
    }
    __device__ __forceinline__ static uint32_t divided(float x, float s) {
        if (!(s > 0.0f)) return 0u;
        const float q = rintf(__fdiv_rn(x, s));
        return q != q ? 0u : (uint32_t)(int)fminf(fmaxf(q, -127.0f), 127.0f);
    }
    __device__ __forceinline__ uint2 codes(const float (&x)[8]) const {
        uint32_t c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float y = __fmul_rn(x[i], inv), t = __fadd_rn(y, 12582912.0f);
            c[i] = __float_as_uint(t);
            if (!(fabsf(__fsub_rn(y, __fsub_rn(t, 12582912.0f))) < 0.5f - 6.2e-5f)) c[i] = divided(x[i], s);
        }
        return make_uint2(pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7]));
    }
    static __device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
        return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
    }
};

template <typename T>
struct Vec8;   // eight consecutive elements as loaded and stored
template <>
struct Vec8<__nv_bfloat16> {
    uint4 w;
    __device__ void load(const __nv_bfloat16 *p) { w = *reinterpret_cast<const uint4 *>(p); }
    __device__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint4 *>(p) = w; }
    __device__ void get(float (&f)[8]) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    __device__ void set(const float (&f)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        w = make_uint4(u[0], u[1], u[2], u[3]);
    }
    // The largest magnitude's bits as a float (an infinity's or a NaN's if there is one).
    __device__ uint32_t top() const {
        constexpr uint32_t m = 0x7fff7fffu;
        const uint32_t a = __vmaxu2(__vmaxu2(w.x & m, w.y & m), __vmaxu2(w.z & m, w.w & m));
        return max(a << 16, a & 0xffff0000u);
    }
};
template <>
struct Vec8<float> {
    float4 a, b;
    __device__ void load(const float *p) {
        a = *reinterpret_cast<const float4 *>(p);
        b = *reinterpret_cast<const float4 *>(p + 4);
    }
    __device__ void store(float *p) const {
        *reinterpret_cast<float4 *>(p) = a;
        *reinterpret_cast<float4 *>(p + 4) = b;
    }
    __device__ void get(float (&f)[8]) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    __device__ void set(const float (&f)[8]) {
        a = make_float4(f[0], f[1], f[2], f[3]);
        b = make_float4(f[4], f[5], f[6], f[7]);
    }
    __device__ uint32_t top() const {
        const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
        return m;
    }
};

// Sixteen values as T: 32 or 64 bytes of one thread, so that a warp's store fills
// whole sectors where two of eight each would fill halves.  wide: `p` is at a
// multiple of 32 bytes.
__device__ __forceinline__ void store32(void *p, const uint4 &a, const uint4 &b) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
                 "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}
__device__ __forceinline__ uint4 bits(const float4 &v) {
    return make_uint4(__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w));
}
__device__ __forceinline__ void store16(__nv_bfloat16 *p, const Vec8<__nv_bfloat16> &a, const Vec8<__nv_bfloat16> &b, bool wide) {
    if (wide) {
        store32(p, a.w, b.w);
    } else {
        a.store(p);
        b.store(p + 8);
    }
}
__device__ __forceinline__ void store16(float *p, const Vec8<float> &a, const Vec8<float> &b, bool wide) {
    if (wide) {
        store32(p, bits(a.a), bits(a.b));
        store32(p + 8, bits(b.a), bits(b.b));
    } else {
        a.store(p);
        b.store(p + 8);
    }
}

// A sum of squares that may pass the float range.  Below kBig it is itself;
// from there on it is negative, that of the values times 2^-80 (a float's square
// is then below 2^96).  kBig: 1024 threads' sums below it stay in range.
// (Squares below the range count as zero.)
struct Squares {
    static constexpr float kBig = 0x1p112f, kDown = 0x1p-80f;
    static __device__ __forceinline__ float scaled(float sum) { return sum < 0.0f ? -sum : sum * kDown * kDown; }
    static __device__ __forceinline__ float add(float sum, const float (&h)[8]) {
        float all = sum;
#pragma unroll
        for (int i = 0; i < 8; ++i) all = fmaf(h[i], h[i], all);
        if (sum >= 0.0f && all < kBig) return all;
        all = scaled(sum);
#pragma unroll
        for (int i = 0; i < 8; ++i) all = fmaf(h[i] * kDown, h[i] * kDown, all);
        return -all;
    }
    // Over a warp.
    static __device__ __forceinline__ float together(float sum) {
        const bool down = __any_sync(~0u, !(sum >= 0.0f));
        if (down) sum = scaled(sum);
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        return down ? -sum : sum;
    }
    // 1 / sqrt(sum / n + eps)
    static __device__ __forceinline__ float rsqrt_mean(float sum, float n, float eps) {
        const bool down = !(sum >= 0.0f);
        const float e = down ? eps * kDown * kDown : eps;
        const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(fabsf(sum), n), e)));
        return down ? r * kDown : r;
    }
};

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// ------------------------------------------------------------------ RMS norm
// h = x + r,  y = h w / sqrt(mean h^2 + eps).  With an 8-bit output the codes
// are those of u = h w in the scale max|u| / 127, and the row's scale is that
// times 1 / sqrt(..): the root cancels between a value and the row's largest,
// so no code depends on the order in which the squares are summed.
//
// One CTA per row.  The row stays in registers between the reduction (sum of
// squares and max|u| together, both in 32 bits) and the output, so x, r are
// read once and h, y written once.  A thread's unit is eight elements at a
// multiple of eight of the whole array, so rows of any width take 16-byte
// accesses; only a row's first and last unit, shared with its neighbours, go
// element by element.  8192 x 4096 bf16 with a residual to 8 bits: 44.1 us, 5.3
// TB/s of its 235 MB (a unit a thread; with two, 48 us: fewer rows in flight).
constexpr int kNormMaxThreads = 1024;

// Eight weights from column c (a multiple of eight in rows that are).  Rows of
// other widths start anywhere in a unit: three 16-byte loads around the eight,
// shifted by c mod 4, which is the same for the whole row.
template <bool WHOLE>
__device__ __forceinline__ void weights8(const float *w, long long c, int cols, float (&f)[8]) {
    if constexpr (WHOLE) {
        Vec8<float> v;
        v.load(w + c);
        v.get(f);
    } else {
        const int at = (int)c, sh = at & 3, lo = at - sh;
        if (at >= 0 && lo + 12 <= cols) {
            float g[12];
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const float4 v = __ldg(reinterpret_cast<const float4 *>(w + lo) + i);
                g[4 * i] = v.x; g[4 * i + 1] = v.y; g[4 * i + 2] = v.z; g[4 * i + 3] = v.w;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = sh < 2 ? (sh ? g[i + 1] : g[i]) : (sh == 2 ? g[i + 2] : g[i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = at + i >= 0 && at + i < cols ? __ldg(w + at + i) : 0.0f;
        }
    }
}

// WHOLE: cols is a multiple of eight, so every unit lies in one row.
template <typename T, int VPT, bool I8, bool RES, bool WHOLE>
__global__ void __launch_bounds__(kNormMaxThreads) rmsnorm_kernel(const NormLaunch L) {
    __shared__ float red[2][32];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int row = blockIdx.x, tid = threadIdx.x, nt = blockDim.x;
    const long long e0 = (long long)row * L.cols, e1 = e0 + L.cols;   // the row's elements
    const long long u0 = e0 >> 3;                                     // its first unit
    const T *x = static_cast<const T *>(L.x), *r = static_cast<const T *>(L.residual);
    T *ho = static_cast<T *>(L.h);
    const auto unit = [&](int v) { return (u0 + tid + (long long)v * nt) * 8; };
    const auto whole = [&](long long e) { return (WHOLE || e >= e0) && e + 8 <= e1; };
    const auto any = [&](long long e) { return !WHOLE && e < e1; };   // an edge's elements, one by one

    float h[VPT][8];
    {
        Vec8<T> a[VPT], b[RES ? VPT : 1];
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (whole(unit(v))) {
                a[v].load(x + unit(v));
                if constexpr (RES) b[v].load(r + unit(v));
            }
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const long long e = unit(v);
            if (whole(e)) {
                a[v].get(h[v]);
                if constexpr (RES) {
                    float f[8];
                    b[v].get(f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) h[v][i] = __fadd_rn(h[v][i], f[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const bool in = any(e) && e + i >= e0 && e + i < e1;
                    h[v][i] = in ? to_float(x[e + i]) : 0.0f;
                    if (RES && in) h[v][i] = __fadd_rn(h[v][i], to_float(r[e + i]));
                }
            }
        }
    }
    float sum = 0.0f, top = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const long long e = unit(v);
        if (RES && ho) {
            if (whole(e)) {
                Vec8<T> a;
                a.set(h[v]);
                a.store(ho + e);
            } else if (any(e)) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (e + i >= e0 && e + i < e1) put(ho + e + i, h[v][i]);
            }
        }
        if (whole(e) || any(e)) {
            float w[8];
            weights8<WHOLE>(L.weight, e - e0, L.cols, w);
            sum = Squares::add(sum, h[v]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[v][i] = __fmul_rn(h[v][i], w[i]);
                if (I8) top = most_or_nan(top, fabsf(h[v][i]));
            }
        }
    }
    // The two reductions of the block in one exchange.  (A magnitude's bits are in
    // its order, an infinity's and then a NaN's above all others.)
    uint32_t most = I8 ? __reduce_max_sync(~0u, __float_as_uint(top)) : 0u;
    sum = Squares::together(sum);
    const int nw = nt >> 5, lane = tid & 31;
    if (lane == 0) {
        red[0][tid >> 5] = sum;
        if (I8) red[1][tid >> 5] = __uint_as_float(most);
    }
    __syncthreads();
    sum = lane < nw ? red[0][lane] : 0.0f;
    if (I8) top = __uint_as_float(__reduce_max_sync(~0u, lane < nw ? __float_as_uint(red[1][lane]) : 0u));
    // With 8-bit codes only the row's scale needs the sum.
    float rstd = 0.0f;
    if (!I8 || tid < 32) {
        sum = Squares::together(sum);
        if (!I8 || tid == 0) rstd = Squares::rsqrt_mean(sum, (float)L.cols, L.eps);
    }
    // A NaN or an infinity in h makes one in u, under a weight of zero too.
    const RowScale s = RowScale::of(top < INFINITY ? __fdiv_rn(top, 127.0f) : __int_as_float(0x7fc00000));
    if (I8 && tid == 0) L.scale[row] = __fmul_rn(s.s, rstd);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const long long e = unit(v);
        if (!whole(e) && !any(e)) continue;
        if constexpr (I8) {
            int8_t *y = static_cast<int8_t *>(L.y);
            const uint2 both = s.codes(h[v]);
            if (whole(e)) {
                *reinterpret_cast<uint2 *>(y + e) = both;
            } else {
                const uint32_t w[2] = {both.x, both.y};
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (e + i >= e0 && e + i < e1) y[e + i] = (int8_t)(w[i >> 2] >> (8 * (i & 3)));
            }
        } else {
            T *y = static_cast<T *>(L.y);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[v][i] = __fmul_rn(h[v][i], rstd);
            if (whole(e)) {
                Vec8<T> a;
                a.set(h[v]);
                a.store(y + e);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (e + i >= e0 && e + i < e1) put(y + e + i, h[v][i]);
            }
        }
    }
}

template <typename T, int VPT, bool WHOLE>
cudaError_t launch_norm_vpt(const NormLaunch &L, int units, cudaStream_t s) {
    const int threads = ((units + VPT - 1) / VPT + 31) / 32 * 32;
    const bool res = L.residual != nullptr;
    if (L.out_int8) {
        if (res) return launch_kernel(rmsnorm_kernel<T, VPT, true, true, WHOLE>, L.rows, threads, 0, s, L);
        return launch_kernel(rmsnorm_kernel<T, VPT, true, false, WHOLE>, L.rows, threads, 0, s, L);
    }
    if (res) return launch_kernel(rmsnorm_kernel<T, VPT, false, true, WHOLE>, L.rows, threads, 0, s, L);
    return launch_kernel(rmsnorm_kernel<T, VPT, false, false, WHOLE>, L.rows, threads, 0, s, L);
}

template <typename T>
cudaError_t launch_norm_typed(const NormLaunch &L, cudaStream_t s) {
    // Units of eight elements a row can touch: one more where rows start off a unit's edge.
    if (L.cols % 8 == 0) {
        const int units = L.cols / 8;
        if (units <= 512) return launch_norm_vpt<T, 1, true>(L, units, s);
        if (units <= 1024) return launch_norm_vpt<T, 2, true>(L, units, s);
        return launch_norm_vpt<T, 4, true>(L, units, s);
    }
    const int units = (L.cols + 7) / 8 + 1;
    if (units <= 256) return launch_norm_vpt<T, 1, false>(L, units, s);
    if (units <= 1024) return launch_norm_vpt<T, 2, false>(L, units, s);
    return launch_norm_vpt<T, 5, false>(L, units, s);   // kNormMaxCols and an odd start: 4097 units
}

// ------------------------------------------------------- rows in 8 bits -> float
// out[r][c] = q[r][c] * scale[r]: the seam behind an operator that scales each
// row by itself.  Sixteen codes a thread, at multiples of sixteen of the whole
// array; a unit that spans rows looks each element's row up.  8192 x 4096 to
// bf16: 13.7 us, 7.3 TB/s (17.8 us with stores of 16 bytes).
template <typename T>
__global__ void dequantize_rows_kernel(const int8_t *__restrict__ q, const float *__restrict__ scale,
                                       T *__restrict__ out, size_t count, int cols) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const size_t units = (count + 15) / 16;
    const bool wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
    const bool narrow = count >> 32 == 0;   // a 64-bit division costs more than the unit's sixteen products
    for (size_t g = blockIdx.x * (size_t)blockDim.x + threadIdx.x; g < units; g += (size_t)gridDim.x * blockDim.x) {
        const size_t e = g * 16;
        const size_t row = narrow ? (uint32_t)e / (uint32_t)cols : e / cols;
        const int c = (int)(e - row * cols);
        if (e + 16 <= count && c + 16 <= cols) {
            const uint4 w = *reinterpret_cast<const uint4 *>(q + e);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            const float s = scale[row];
            Vec8<T> o[2];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    f[i] = __fmul_rn((float)(int8_t)(u[2 * v + (i >> 2)] >> (8 * (i & 3))), s);
                o[v].set(f);
            }
            store16(out + e, o[0], o[1], wide);
        } else {
            size_t r = row;
            int at = c;
            for (size_t i = e; i < e + 16 && i < count; ++i) {
                put(out + i, __fmul_rn((float)q[i], scale[r]));
                if (++at == cols) { at = 0; ++r; }
            }
        }
    }
}

int grid_for_units(size_t units, int threads, int per_sm) {
    size_t blocks = (units + threads - 1) / threads;
    const size_t cap = (size_t)current_device_sms() * per_sm;
    if (blocks > cap) blocks = cap;
    return blocks < 1 ? 1 : (int)blocks;
}

// ------------------------------------------------------------ the paged cache
// Sequence of new token i: the last b with new_start[b] <= i.  -1 when the
// starts give token i to no sequence.
__device__ __forceinline__ int sequence_of(const CacheArgs &a, int i) {
    int lo = 0, hi = a.batch;   // new_start[lo] <= i < new_start[hi], if the starts are in order
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.new_start[mid] <= i) lo = mid;
        else hi = mid;
    }
    return a.new_start[lo] <= i && i < a.new_start[lo + 1] ? lo : -1;
}

// Where a token's rows go: its page's first row of head 0 and its slot, or -1.
// (Tokens behind the last sequence's are padding and go nowhere.)
struct Place { int page, slot; };
__device__ __forceinline__ Place place_of(const CacheArgs &a, int i) {
    const int b = sequence_of(a, i);
    // (From the length as it is: from one cut to its table's end, tokens past that
    // would go to other positions' places.  page_of refuses them.)
    const int pos = b < 0 ? -1 : max(a.seq_lens[b], 0) - (a.new_start[b + 1] - i);
    if (pos < 0) {
        if (b >= 0 || i < a.new_start[a.batch]) atomicOr(a.status, kStatusBadIndex);
        return Place{-1, 0};
    }
    return Place{page_of(a, b, pos), pos & ((1 << a.page_shift) - 1)};
}

// New tokens into their pages.  A row is a token's key or value of one head;
// D / 8 lanes take it, eight elements each, and its largest magnitude comes from
// a butterfly over them.  Instructions bound it, not memory (8192 tokens, 8 heads
// of 128 to 8 bits: 17.1 us, 3.0 TB/s).  A warp takes kRowsWarp rows of one token (rows 2 head +
// side): the token's place is looked up once for all of them, behind their
// loads, which need only the token's number.
constexpr int kRowsWarp = 4;

template <typename T, int D>
__global__ void __launch_bounds__(128) cache_write_kernel(const CacheArgs a, const T *__restrict__ k, long long k_stride,
                                                          const T *__restrict__ v, long long v_stride) {
    constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kSteps = kRowsWarp / kAtOnce;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int rows = 2 * a.kv_heads, parts = (rows + kRowsWarp - 1) / kRowsWarp;
    const long long tasks = (long long)a.total * parts;
    const int lane = threadIdx.x & 31, sub = lane / kLanes, at8 = (lane % kLanes) * 8;
    const long long step = (long long)gridDim.x * (blockDim.x >> 5);
    for (long long task = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); task < tasks; task += step) {
        const int i = (int)(task / parts), part = (int)(task - (long long)i * parts);
        Vec8<T> in[kSteps];
#pragma unroll
        for (int x = 0; x < kSteps; ++x) {
            const int row = part * kRowsWarp + x * kAtOnce + sub;
            in[x] = Vec8<T>{};
            if (row < rows) in[x].load((row & 1 ? v + (size_t)i * v_stride : k + (size_t)i * k_stride) + (row >> 1) * D + at8);
        }
        const Place place = place_of(a, i);
        if (place.page < 0) continue;
#pragma unroll
        for (int x = 0; x < kSteps; ++x) {
            const int row = part * kRowsWarp + x * kAtOnce + sub, head = row >> 1;
            const size_t at = (((size_t)place.page * a.kv_heads + head) << a.page_shift) + place.slot;
            float f[8];
            in[x].get(f);
            if (a.int8) {
                // The largest magnitude as bits, above which only infinities and NaN lie.
                uint32_t top = in[x].top();
#pragma unroll
                for (int o = kLanes / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
                if (row >= rows) continue;
                // A row that holds a NaN or an infinity reads back as NaN.
                const RowScale s = RowScale::of(top < 0x7f800000u ? __fdiv_rn(__uint_as_float(top), 127.0f) : __int_as_float(0x7fc00000));
                *reinterpret_cast<uint2 *>(static_cast<int8_t *>(row & 1 ? a.v : a.k) + at * D + at8) = s.codes(f);
                if (at8 == 0) (row & 1 ? a.v_scale : a.k_scale)[at] = s.s;
            } else if (row < rows) {
                Vec8<__nv_bfloat16> o;
                o.set(f);
                o.store(static_cast<__nv_bfloat16 *>(row & 1 ? a.v : a.k) + at * D + at8);
            }
        }
    }
}

// The sequences' rows in order: out[b][pos][head][:], zero past a length.  A
// CTA takes consecutive positions of one sequence and some of its heads
// (blockIdx.z and every gridDim.z after it); a thread 16 bytes of the cache a
// row, of K and V, so the pages' rows are read as they lie and every index but
// the page is a shift.  4 x 16384 positions, 8 heads of 128, 8 bits to bf16: 65.1
// us, 6.3 TB/s of its 407 MB (80 us with stores of 16 bytes).
constexpr int kReadThreads = 256;
template <int D, bool I8>
constexpr int read_positions() { return kReadThreads / (D * (I8 ? 1 : 2) / 16); }

template <typename T, int D, bool I8>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const CacheArgs a, int max_len, T *__restrict__ k_out,
                                                                  T *__restrict__ v_out) {
    constexpr int kE = I8 ? 16 : 8, kUnits = D / kE;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int u = threadIdx.x % kUnits, b = blockIdx.y;
    const bool wide = ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31) == 0;
    const int pos = blockIdx.x * read_positions<D, I8>() + threadIdx.x / kUnits;
    if (pos >= max_len) return;
    const int p = pos < seq_len(a, b) ? page_of(a, b, pos) : -1;
    const size_t from = (((size_t)(p < 0 ? 0 : p) * a.kv_heads) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
    const size_t to = ((size_t)b * max_len + pos) * a.kv_heads;
#pragma unroll 2
    for (int head = blockIdx.z; head < a.kv_heads; head += gridDim.z) {
        const size_t at = from + ((size_t)head << a.page_shift);
        uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        float s[2] = {0.0f, 0.0f};
        if (p >= 0) {
            w[0] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const char *>(a.k) + at * (D * (I8 ? 1 : 2))) + u);
            w[1] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const char *>(a.v) + at * (D * (I8 ? 1 : 2))) + u);
            if (I8) {
                s[0] = a.k_scale[at];
                s[1] = a.v_scale[at];
            }
        }
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            T *out = (side ? v_out : k_out) + (to + head) * D + u * kE;
            if constexpr (I8) {
                const uint32_t c[4] = {w[side].x, w[side].y, w[side].z, w[side].w};
                Vec8<T> o[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float f[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = __fmul_rn((float)(int8_t)(c[2 * q + (i >> 2)] >> (8 * (i & 3))), s[side]);
                    o[q].set(f);
                }
                store16(out, o[0], o[1], wide);
            } else if constexpr (sizeof(T) == 2) {
                *reinterpret_cast<uint4 *>(out) = w[side];
            } else {
                Vec8<__nv_bfloat16> in;
                in.w = w[side];
                float f[8];
                in.get(f);
                Vec8<T> o;
                o.set(f);
                o.store(out);
            }
        }
    }
}

}  // namespace

cudaError_t launch_rmsnorm(const NormLaunch &L, cudaStream_t s) {
    return L.in_bf16 ? launch_norm_typed<__nv_bfloat16>(L, s) : launch_norm_typed<float>(L, s);
}

cudaError_t launch_dequantize_rows(const int8_t *q, const float *scale, void *out, int rows, int cols, int out_bf16,
                                   cudaStream_t s) {
    const size_t count = (size_t)rows * cols;
    const int g = grid_for_units((count + 15) / 16, 256, 16);
    if (out_bf16)
        return launch_kernel(dequantize_rows_kernel<__nv_bfloat16>, g, 256, 0, s, q, scale, (__nv_bfloat16 *)out, count, cols);
    return launch_kernel(dequantize_rows_kernel<float>, g, 256, 0, s, q, scale, (float *)out, count, cols);
}

cudaError_t launch_cache_write(const CacheArgs &a, const void *k, long long k_stride, const void *v,
                               long long v_stride, int in_bf16, cudaStream_t s) {
    const size_t threads = (size_t)a.total * ((2 * a.kv_heads + kRowsWarp - 1) / kRowsWarp) * 32;
    const int g = grid_for_units(threads, 128, 32);
    auto run = [&](auto kern, auto *kp, auto *vp) { return launch_kernel(kern, g, 128, 0, s, a, kp, k_stride, vp, v_stride); };
    auto typed = [&](auto *kp, auto *vp) {
        using T = std::remove_const_t<std::remove_pointer_t<decltype(kp)>>;
        if (a.head_dim == 64) return run(cache_write_kernel<T, 64>, kp, vp);
        return run(cache_write_kernel<T, 128>, kp, vp);
    };
    if (in_bf16) return typed(static_cast<const __nv_bfloat16 *>(k), static_cast<const __nv_bfloat16 *>(v));
    return typed(static_cast<const float *>(k), static_cast<const float *>(v));
}

cudaError_t launch_cache_read(const CacheArgs &a, int max_len, void *k_out, void *v_out, int out_bf16, cudaStream_t s) {
    const int positions = kReadThreads / (a.head_dim * (a.int8 ? 1 : 2) / 16);
    const long long ctas = (long long)((max_len + positions - 1) / positions) * a.batch;
    // Heads side by side until each SM has sixteen CTAs.
    const long long want = (current_device_sms() * 16 + ctas - 1) / ctas;
    const dim3 grid((max_len + positions - 1) / positions, a.batch, (unsigned)(want < a.kv_heads ? want : a.kv_heads));
    auto run = [&](auto kern, auto *ko, auto *vo) { return launch_kernel(kern, grid, kReadThreads, 0, s, a, max_len, ko, vo); };
    auto dims = [&](auto *ko, auto *vo) {
        using T = std::remove_pointer_t<decltype(ko)>;
        if (a.head_dim == 64)
            return a.int8 ? run(cache_read_kernel<T, 64, true>, ko, vo) : run(cache_read_kernel<T, 64, false>, ko, vo);
        return a.int8 ? run(cache_read_kernel<T, 128, true>, ko, vo) : run(cache_read_kernel<T, 128, false>, ko, vo);
    };
    if (out_bf16) return dims(static_cast<__nv_bfloat16 *>(k_out), static_cast<__nv_bfloat16 *>(v_out));
    return dims(static_cast<float *>(k_out), static_cast<float *>(v_out));
}

}  // namespace cbs
