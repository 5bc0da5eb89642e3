// w8.cuh -- what the kernels for products of 8-bit integers share (the formula and the
// layout are in k_w8.cu).
#pragma once

#include <cuda_bf16.h>

#include "mma_frag.cuh"
#include "tc_ptx.cuh"
#include "tc_warp.cuh"
#include "tokens.cuh"

namespace cbs {
namespace w8 {

constexpr int kOut = 128;                    // outputs of a CTA: tensor memory's lanes
constexpr int kStageK = 128;                 // codes along k in a stage: a row of 128 bytes
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s per wait

// Sixteen codes of an input row (unit u of eight in a stage's row) to where the MMA
// reads them: panels of 64 f16, 128 bytes a row, swizzled.  Lanes of a row's second 64
// write their upper half first: eight lanes are then in eight different sixteen-byte
// banks.  `to`: the unit's panel.
__device__ __forceinline__ void widen_input(unsigned char *to, int row, int u, uint4 raw) {
    const uint32_t second = u >> 2;
    uint32_t o[8];
    frag::i8_halves(raw.x, o[0], o[1]);
    frag::i8_halves(raw.y, o[2], o[3]);
    frag::i8_halves(raw.z, o[4], o[5]);
    frag::i8_halves(raw.w, o[6], o[7]);
    const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
    const uint32_t at = row * 128 + ((((u & 3) * 2 + second) ^ (row & 7)) << 4);
    *reinterpret_cast<uint4 *>(to + at) = second ? hi : lo;
    *reinterpret_cast<uint4 *>(to + (at ^ 16)) = second ? lo : hi;
}

// Half h of a stage's 128 weights of an output, as 32 pairs of f16.  `from`: the row.
__device__ __forceinline__ void widen_weights(const unsigned char *from, int row, int h, uint32_t (&a)[32]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint4 w = *reinterpret_cast<const uint4 *>(from + (((4 * h + q) ^ (row & 7)) << 4));
        frag::i8_halves(w.x, a[8 * q], a[8 * q + 1]);
        frag::i8_halves(w.y, a[8 * q + 2], a[8 * q + 3]);
        frag::i8_halves(w.z, a[8 * q + 4], a[8 * q + 5]);
        frag::i8_halves(w.w, a[8 * q + 6], a[8 * q + 7]);
    }
}

// sum x_scale w_scale + bias, as (sum first) x_scale last + bias.  The scales' product may
// leave the float range where the result does not, so the sum, a whole number, is multiplied
// with one at a time: it only makes a scale larger, and one up to 1 leaves it in range; of a
// larger w_scale first, x_scale's turn comes before, and what then leaves the range would
// have.  (2048 rows of 8192 x 256 21.5 us with the scales' product, now 22.0; with the smaller
// of both first, by comparisons for every sum, 23.8.)
struct Channel {
    float first, last, bias;
    __device__ __forceinline__ Channel(float w_scale, float bias)
        : first(fabsf(w_scale) <= 1.0f ? w_scale : 1.0f), last(fabsf(w_scale) <= 1.0f ? 1.0f : w_scale), bias(bias) {}   // (a NaN is last)
    __device__ __forceinline__ float operator()(float sum, float x_scale) const { return fmaf(sum * first * x_scale, last, bias); }
};

// One output of input rows m, m + 1, ...: sums, as they come from tensor memory, to
// y + (m * n + its number).  `scales`: those rows', `left`: how many there are.
template <bool BF16, bool SILU, int COUNT>
__device__ __forceinline__ void store_rows(void *y, size_t at, int pitch, const uint32_t (&sums)[COUNT], const float *scales,
                                           const Channel &channel, int left) {
#pragma unroll
    for (int e = 0; e < COUNT; ++e) {
        float v = channel(__uint_as_float(sums[e]), scales[e]);
        if (SILU) v = silu(v);
        if (e < left) {
            if (BF16) static_cast<__nv_bfloat16 *>(y)[at] = __float2bfloat16_rn(v);
            else static_cast<float *>(y)[at] = v;
        }
        at += pitch;
    }
}
template <int COUNT>
__device__ __forceinline__ void store_rows(const W8Launch &L, int m, int n, const uint32_t (&sums)[COUNT], const float *scales,
                                           const Channel &channel) {
    const size_t at = (size_t)m * L.n + n;
    const int left = L.rows - m;
    if (L.act == CBS_ACT_SILU) {
        if (L.out_bf16) store_rows<true, true>(L.y, at, L.n, sums, scales, channel, left);
        else store_rows<false, true>(L.y, at, L.n, sums, scales, channel, left);
    } else {
        if (L.out_bf16) store_rows<true, false>(L.y, at, L.n, sums, scales, channel, left);
        else store_rows<false, false>(L.y, at, L.n, sums, scales, channel, left);
    }
}

// Rows of k codes, boxes of a stage by `box_rows`.
inline cbs_status codes_map(CUtensorMap *tm, const void *p, int k, int rows, int box_rows) {
    EncodeTiledFn fn = encode_tiled();
    if (!fn) return fail(CBS_ERR_CUDA, "cannot resolve cuTensorMapEncodeTiled from the driver");
    const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)k};
    const cuuint32_t box[2] = {(cuuint32_t)kStageK, (cuuint32_t)box_rows}, es[2] = {1u, 1u};
    const CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(CBS_ERR_CUDA, "cuTensorMapEncodeTiled (8-bit codes) failed (%d)", (int)r);
    return CBS_OK;
}

}  // namespace w8
}  // namespace cbs
