// mma_frag.cuh -- warp-level matrix fragments for the operators whose few rows
// leave the tensor cores idle and HBM busy: m16n8k16 products whose operands go
// from global memory straight to registers, with the contraction index
// permuted so that every lane's share of a row is one wide load.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

namespace cbs {
namespace frag {

// c[16 x 8] += a[16 x 16] b[16 x 8], bf16 operands, float sums.  With
// g = lane / 4 and j = lane % 4: a0 = rows g, k 2j..2j+1; a1 = rows g + 8;
// a2, a3 = the same at k + 8; b0 = column g, k 2j..2j+1; b1 at k + 8;
// c0, c1 = row g, columns 2j, 2j + 1; c2, c3 = row g + 8.
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with f16 operands.
__device__ __forceinline__ void mma_half(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four int8 codes as two pairs of f16, exactly: 1024 + (code + 128) by the byte's
// place, less 1152.
__device__ __forceinline__ void i8_halves(uint32_t codes, uint32_t &lo, uint32_t &hi) {
    const uint32_t u = codes ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
}
// Two floats as a pair of f16, the first in the low half.
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Transpose of an 8 x 8 matrix of 16-bit values held two to a lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}

// sum + the bf16 value in the low half of v.
__device__ __forceinline__ float add_bf16(float sum, uint32_t v) {
    asm("add.rn.f32.bf16 %0, %1, %0;" : "+f"(sum) : "h"((uint16_t)v));
    return sum;
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Two int8 codes, in bytes 0 and 2 of v (the other bytes hold anything), as a
// pair of bf16 values.  128 + (low seven bits) is exact in bf16's eight
// significant bits at exponent 7; taking 128 away, or 256 from a code with its
// sign bit set, leaves the code itself.
__device__ __forceinline__ uint32_t i8_pair(uint32_t v) {
    const uint32_t low = (v & 0x007f007fu) | 0x43004300u;
    const uint32_t off = (v & 0x00800080u) | 0x43004300u;
    return sub_bf16x2(low, off);
}

// Base-2 exponential, approximate (2 ulp), flushing subnormals.
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

}  // namespace frag
}  // namespace cbs
