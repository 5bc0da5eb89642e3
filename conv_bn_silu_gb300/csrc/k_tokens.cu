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
__device__ __forceinline__ int code_of(float x, float s) {
    if (!(s > 0.0f)) return 0;
    const float q = rintf(__fdiv_rn(x, s));
    return q != q ? 0 : (int)fminf(fmaxf(q, -127.0f), 127.0f);
}

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
// element by element.
constexpr int kNormMaxThreads = 1024;

template <typename T, int VPT, bool I8, bool RES>
__global__ void __launch_bounds__(kNormMaxThreads) rmsnorm_kernel(const NormLaunch L) {
    __shared__ float red[2][32];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int row = blockIdx.x, tid = threadIdx.x, nt = blockDim.x;
    const long long e0 = (long long)row * L.cols, e1 = e0 + L.cols;   // the row's elements
    const long long u0 = e0 >> 3;                                     // its first unit
    const T *x = static_cast<const T *>(L.x), *r = static_cast<const T *>(L.residual);
    T *ho = static_cast<T *>(L.h);

    float h[VPT][8];
    float sum = 0.0f, top = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const long long e = (u0 + tid + (long long)v * nt) * 8;
        if (e >= e0 && e + 8 <= e1) {
            Vec8<T> a;
            a.load(x + e);
            a.get(h[v]);
            if (RES) {
                Vec8<T> b;
                float f[8];
                b.load(r + e);
                b.get(f);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[v][i] = __fadd_rn(h[v][i], f[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool in = e + i >= e0 && e + i < e1;
                h[v][i] = in ? to_float(x[e + i]) : 0.0f;
                if (RES && in) h[v][i] = __fadd_rn(h[v][i], to_float(r[e + i]));
            }
        }
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const long long e = (u0 + tid + (long long)v * nt) * 8;
        if (RES && ho) {
            if (e >= e0 && e + 8 <= e1) {
                Vec8<T> a;
                a.set(h[v]);
                a.store(ho + e);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (e + i >= e0 && e + i < e1) put(ho + e + i, h[v][i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sum = fmaf(h[v][i], h[v][i], sum);
            const long long c = e + i - e0;
            const float w = c >= 0 && c < L.cols ? __ldg(L.weight + c) : 0.0f;
            h[v][i] = __fmul_rn(h[v][i], w);
            if (I8) top = fmaxf(top, fabsf(h[v][i]));
        }
    }
    // The two reductions of the block in one exchange.
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        sum += __shfl_xor_sync(~0u, sum, o);
        if (I8) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    }
    if ((tid & 31) == 0) {
        red[0][tid >> 5] = sum;
        if (I8) red[1][tid >> 5] = top;
    }
    __syncthreads();
    const int nw = nt >> 5, lane = tid & 31;
    sum = lane < nw ? red[0][lane] : 0.0f;
    if (I8) top = lane < nw ? red[1][lane] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        sum += __shfl_xor_sync(~0u, sum, o);
        if (I8) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    }
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sum, (float)L.cols), L.eps)));
    const float s = __fdiv_rn(top, 127.0f);
    if (I8 && tid == 0) L.scale[row] = __fmul_rn(s, rstd);
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
        const long long e = (u0 + tid + (long long)v * nt) * 8;
        const bool whole = e >= e0 && e + 8 <= e1;
        if (I8) {
            int8_t *y = static_cast<int8_t *>(L.y);
            uint32_t w[2] = {0u, 0u};
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i >> 2] |= (uint32_t)(uint8_t)code_of(h[v][i], s) << (8 * (i & 3));
            if (whole) {
                *reinterpret_cast<uint2 *>(y + e) = make_uint2(w[0], w[1]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (e + i >= e0 && e + i < e1) y[e + i] = (int8_t)(w[i >> 2] >> (8 * (i & 3)));
            }
        } else {
            T *y = static_cast<T *>(L.y);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[v][i] = __fmul_rn(h[v][i], rstd);
            if (whole) {
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

template <typename T, int VPT>
cudaError_t launch_norm_vpt(const NormLaunch &L, int units, cudaStream_t s) {
    const int threads = ((units + VPT - 1) / VPT + 31) / 32 * 32;
    const bool res = L.residual != nullptr;
    if (L.out_int8) {
        if (res) return launch_kernel(rmsnorm_kernel<T, VPT, true, true>, L.rows, threads, 0, s, L);
        return launch_kernel(rmsnorm_kernel<T, VPT, true, false>, L.rows, threads, 0, s, L);
    }
    if (res) return launch_kernel(rmsnorm_kernel<T, VPT, false, true>, L.rows, threads, 0, s, L);
    return launch_kernel(rmsnorm_kernel<T, VPT, false, false>, L.rows, threads, 0, s, L);
}

template <typename T>
cudaError_t launch_norm_typed(const NormLaunch &L, cudaStream_t s) {
    // Units of eight elements a row can touch: one more where rows start off a unit's edge.
    const int units = (L.cols + 7) / 8 + (L.cols % 8 ? 1 : 0);
    if (units <= 256) return launch_norm_vpt<T, 1>(L, units, s);
    if (units <= 1024) return launch_norm_vpt<T, 2>(L, units, s);
    return launch_norm_vpt<T, 5>(L, units, s);   // kNormMaxCols and an odd start: 4097 units
}

// ------------------------------------------------------- rows in 8 bits -> float
// out[r][c] = q[r][c] * scale[r]: the seam behind an operator that scales each
// row by itself.  Sixteen codes a thread, at multiples of sixteen of the whole
// array; a unit that spans rows looks each element's row up.
template <typename T>
__global__ void dequantize_rows_kernel(const int8_t *__restrict__ q, const float *__restrict__ scale,
                                       T *__restrict__ out, size_t count, int cols) {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const size_t units = (count + 15) / 16;
    for (size_t g = blockIdx.x * (size_t)blockDim.x + threadIdx.x; g < units; g += (size_t)gridDim.x * blockDim.x) {
        const size_t e = g * 16;
        const size_t row = e / cols;
        const int c = (int)(e - row * cols);
        if (e + 16 <= count && c + 16 <= cols) {
            const uint4 w = *reinterpret_cast<const uint4 *>(q + e);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            const float s = scale[row];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    f[i] = __fmul_rn((float)(int8_t)(u[2 * v + (i >> 2)] >> (8 * (i & 3))), s);
                Vec8<T> o;
                o.set(f);
                o.store(out + e + 8 * v);
            }
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

// New tokens into their pages.  D / 4 lanes take one row (a token's key or
// value of one head), four elements each; a row's largest magnitude comes from
// a butterfly over its lanes.
template <typename T, int D>
__global__ void cache_write_kernel(const CacheArgs a, const T *__restrict__ k, long long k_stride,
                                   const T *__restrict__ v, long long v_stride) {
    constexpr int kLanes = D / 4;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const long long rows = (long long)a.total * a.kv_heads * 2;
    const int lane = threadIdx.x % kLanes;
    const long long step = (long long)gridDim.x * (blockDim.x / kLanes);
    // Whole warps go round together: the butterfly needs every lane.
    const long long first = (long long)blockIdx.x * (blockDim.x / kLanes) + threadIdx.x / kLanes;
    const long long rounds = (rows + step - 1) / step;
    for (long long it = 0; it < rounds; ++it) {
        const long long row = first + it * step;
        bool live = row < rows;
        const int side = (int)(row & 1);   // 0: key, 1: value
        const int head = live ? (int)((row >> 1) % a.kv_heads) : 0;
        const int i = live ? (int)((row >> 1) / a.kv_heads) : 0;
        size_t at = 0;
        if (live) {
            const int b = sequence_of(a, i);
            const int n = b < 0 ? 0 : seq_len(a, b);
            const int pos = b < 0 ? -1 : n - (a.new_start[b + 1] - i);
            const int p = pos < 0 ? -1 : page_of(a, b, pos);
            if (pos < 0) atomicOr(a.status, kStatusBadIndex);
            live = p >= 0;
            if (live)
                at = (((size_t)p * a.kv_heads + head) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
        }
        float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (live) {
            const T *src = (side ? v + (size_t)i * v_stride : k + (size_t)i * k_stride) + head * D + lane * 4;
            if constexpr (sizeof(T) == 2) {
                const uint2 w = *reinterpret_cast<const uint2 *>(src);
                f[0] = __uint_as_float(w.x << 16);
                f[1] = __uint_as_float(w.x & 0xffff0000u);
                f[2] = __uint_as_float(w.y << 16);
                f[3] = __uint_as_float(w.y & 0xffff0000u);
            } else {
                const float4 w = *reinterpret_cast<const float4 *>(src);
                f[0] = w.x; f[1] = w.y; f[2] = w.z; f[3] = w.w;
            }
        }
        if (a.int8) {
            float top = fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])));
            bool nan = f[0] != f[0] || f[1] != f[1] || f[2] != f[2] || f[3] != f[3];
#pragma unroll
            for (int o = kLanes / 2; o; o >>= 1) {
                top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
                nan |= __shfl_xor_sync(~0u, (int)nan, o) != 0;
            }
            if (!live) continue;
            // A row that holds a NaN or an infinity reads back as NaN.
            const float s = nan || top > 3.402823466e38f ? __int_as_float(0x7fc00000) : __fdiv_rn(top, 127.0f);
            uint32_t w = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) w |= (uint32_t)(uint8_t)code_of(f[e], s) << (8 * e);
            int8_t *dst = static_cast<int8_t *>(side ? a.v : a.k) + at * D + lane * 4;
            *reinterpret_cast<uint32_t *>(dst) = w;
            if (lane == 0) (side ? a.v_scale : a.k_scale)[at] = s;
        } else if (live) {
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(side ? a.v : a.k) + at * D + lane * 4;
            const __nv_bfloat162 lo = __floats2bfloat162_rn(f[0], f[1]), hi = __floats2bfloat162_rn(f[2], f[3]);
            *reinterpret_cast<uint2 *>(dst) = make_uint2(*reinterpret_cast<const uint32_t *>(&lo),
                                                         *reinterpret_cast<const uint32_t *>(&hi));
        }
    }
}

// The sequences' rows in order: out[b][pos][head][:], zero past a length.
// Eight elements a thread.
template <typename T, int D, bool I8>
__global__ void cache_read_kernel(const CacheArgs a, int max_len, T *__restrict__ k_out, T *__restrict__ v_out) {
    constexpr int kUnits = D / 8;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const size_t units = (size_t)a.batch * max_len * a.kv_heads * kUnits;
    for (size_t g = blockIdx.x * (size_t)blockDim.x + threadIdx.x; g < units; g += (size_t)gridDim.x * blockDim.x) {
        const int u = (int)(g % kUnits);
        const size_t row = g / kUnits;
        const int head = (int)(row % a.kv_heads);
        const size_t bp = row / a.kv_heads;
        const int b = (int)(bp / max_len), pos = (int)(bp % max_len);
        const int p = pos < seq_len(a, b) ? page_of(a, b, pos) : -1;
        const size_t at = (((size_t)(p < 0 ? 0 : p) * a.kv_heads + head) << a.page_shift) +
                          (pos & ((1 << a.page_shift) - 1));
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            float f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            if (p >= 0) {
                if (I8) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(
                        static_cast<const int8_t *>(side ? a.v : a.k) + at * D + u * 8);
                    const float s = (side ? a.v_scale : a.k_scale)[at];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        f[i] = __fmul_rn((float)(int8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3))), s);
                } else {
                    Vec8<__nv_bfloat16> w;
                    w.load(static_cast<const __nv_bfloat16 *>(side ? a.v : a.k) + at * D + u * 8);
                    w.get(f);
                }
            }
            Vec8<T> o;
            o.set(f);
            o.store((side ? v_out : k_out) + g * 8);
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
    const size_t threads = (size_t)a.total * a.kv_heads * 2 * (a.head_dim / 4);
    const int g = grid_for_units(threads, 256, 8);
    auto run = [&](auto kern, auto *kp, auto *vp) { return launch_kernel(kern, g, 256, 0, s, a, kp, k_stride, vp, v_stride); };
    if (in_bf16) {
        auto *kp = static_cast<const __nv_bfloat16 *>(k), *vp = static_cast<const __nv_bfloat16 *>(v);
        if (a.head_dim == 64) return run(cache_write_kernel<__nv_bfloat16, 64>, kp, vp);
        return run(cache_write_kernel<__nv_bfloat16, 128>, kp, vp);
    }
    auto *kp = static_cast<const float *>(k), *vp = static_cast<const float *>(v);
    if (a.head_dim == 64) return run(cache_write_kernel<float, 64>, kp, vp);
    return run(cache_write_kernel<float, 128>, kp, vp);
}

cudaError_t launch_cache_read(const CacheArgs &a, int max_len, void *k_out, void *v_out, int out_bf16, cudaStream_t s) {
    const size_t units = (size_t)a.batch * max_len * a.kv_heads * (a.head_dim / 8);
    const int g = grid_for_units(units, 256, 16);
    auto run = [&](auto kern, auto *ko, auto *vo) { return launch_kernel(kern, g, 256, 0, s, a, max_len, ko, vo); };
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
