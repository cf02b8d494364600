// What the products of a few rows share: weights as they lie in memory against a few tokens, on
// mma.m16n8k16 with bf16 operands and fp32 sums.
//
// Such a product is bound by the weights' bytes, each read once.  The contraction's order is chosen to
// fit the loads: an mma may take any 16 columns k as long as both operands agree, so each lane loads
// 16 bytes of a row (8 columns), the four lanes of a row 64 bytes, and the words go straight into the
// fragments of two mma: no shared memory, no conversion, no shuffle.  (tcgen05 would want both operands
// in shared memory and 64 or more rows of one of them: for 1 to 32 tokens the tile would be empty.)
//
// A step is 32 columns.  In a fragment's terms, with g = lane / 4 and q = lane % 4: the lane holds the
// columns 8q .. 8q + 7 of weight rows g and g + 8 and of token g, and gets the sums of rows g and g + 8
// with tokens 2q and 2q + 1.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"

namespace gb {
namespace skinny {

constexpr int kStep = 32;

// An mma cuts off what is below its sum's last bit, always towards zero: a chain of n is off by up to n 2^-23 of the sum, as
// measured by a third of that where the terms have one sign (1792 in a row: 7e-5).  So a chain ends after so many, and
// fp32 additions, rounded to nearest, join the chains.
constexpr int kChain = 64;

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A step: 16 weight rows (`lo`: row g, `hi`: row g + 8) with 8 tokens.
__device__ __forceinline__ void mma_step(float (&c)[4], const uint4& lo, const uint4& hi, const uint4& x) {
    mma(c, lo.x, hi.x, lo.y, hi.y, x.x, x.y);
    mma(c, lo.z, hi.z, lo.w, hi.w, x.z, x.w);
}

// What is read once needs no place in L1, which the tokens have.  (Not the non-coherent load: these kernels start while the
// one before still writes, perhaps what they read, and lora writes D where it read R.  It is no faster.)
__device__ __forceinline__ uint4 load_once(const uint16_t* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Eight elements of a row of `cols` at `col` (zeros from `cols` on).
__device__ __forceinline__ uint4 load_edge(const uint16_t* row, int col, int cols) {
    if (col + 8 <= cols) return *reinterpret_cast<const uint4*>(row + col);
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = col + i < cols ? row[col + i] : 0u;
    return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
}

// v as the sum of two bf16, each rounded to nearest: 17 bits of it, so that a product of v with bf16 weights loses nothing
// that fp32 sums would have kept to the output's bf16.  (hi cut off instead, as it is where it would round up to infinity,
// leaves 16: with that the experts' D was off by 5 to 8e-6 of its size before its rounding, now by 3.6e-6, where fp32
// products by a library are off by 2.5e-6.)
__device__ __forceinline__ void split(float v, uint16_t& hi, uint16_t& lo) {
    auto finite = [](uint32_t u) { return (u & 0x7f800000u) != 0x7f800000u; };
    uint32_t top = static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(v))) << 16;
    if (!finite(top)) top = __float_as_uint(v) & 0xffff0000u;
    hi = static_cast<uint16_t>(v != v ? 0x7fffu : top >> 16);
    lo = finite(top) ? __bfloat16_as_ushort(__float2bfloat16_rn(v - __uint_as_float(top))) : uint16_t(0);
}

__device__ __forceinline__ float bf16_value(uint16_t u) { return __uint_as_float(static_cast<uint32_t>(u) << 16); }
__device__ __forceinline__ uint16_t bf16_bits(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// The activations with the hardware's 2^x and 1/x (2^-22 of their value each; exact divisions took three times as long
// as all else in the adapters' epilogue).  silu(-infinity) is NaN, as -infinity / infinity is.
__device__ __forceinline__ float silu(float v) { return v * rcp_approx(1.f + ex2_approx(-1.44269504f * v)); }

__device__ __forceinline__ float activate(float v, int act) {
    if (act == 1) {
        // 0.5 (1 + tanh u) = 1 / (1 + exp(-2u)), u = sqrt(2 / pi) (v + 0.044715 v^3)
        const float u = 0.7978845608028654f * (v + 0.044715f * v * v * v);
        return v * rcp_approx(1.f + ex2_approx(-2.88539008f * u));
    }
    if (act == 2) return silu(v);
    if (act == 3) return v > 0.f ? v : (v != v ? v : 0.f);
    return v;
}

}  // namespace skinny
}  // namespace gb
