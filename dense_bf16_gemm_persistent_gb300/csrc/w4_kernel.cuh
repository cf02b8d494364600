// Device code of the products with 4-bit weights for a few tokens.
//
//   W[n,k] = (q[n,k] - z[n,k/G]) s[n,k/G]          q, z in 0..15, G = 32, 64 or 128
//   D = act(x W^T + bias) + R        or        D = silu(x W1^T) * (x W3^T)
//
// Bound by the weights' bytes: every one is read once, and at the memory's rate an SM has about
// a cycle for each 50 weights.  So the weights go from global memory to registers in the layout
// they are stored in, and the contraction's order is chosen to fit: mma.m16n8k16 may take any 16
// columns k as long as both operands agree, so a lane's share of each group is contiguous in
// memory, and x is laid out in shared memory to match.  (tcgen05 would want the widened weights
// written to shared or tensor memory first, and a read of its accumulator for each group; with
// no more than 32 tokens the warp-level instruction keeps the multiplications off the bound.)
//
// A nibble becomes a bf16 without rounding: 0x4300 | q is 128 + q, and 128 + z is taken off.  The
// products (q - z) x are summed in fp32 by the tensor cores within a group, and the group's sum is
// multiplied by its scales in fp32: no weight is ever rounded.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "ptx.cuh"

namespace gb {
namespace w4 {

constexpr int kStep = 128;           // columns of one step: four lanes x 16 bytes of weights
constexpr int kUnit = 4 * kStep;     // columns that a warp loads at a time
constexpr int kRows = 16;            // weight rows of a tile: mma's M
constexpr int kMaxWarps = 8;

enum { kXBf16 = 0, kXRowScale = 1, kXGroupScale = 2 };

struct Params {
    const void* x;
    const float* x_scale;
    int64_t ldx, ldxs;
    // the tile's rows 0..7 and 8..15 come from two sources: a linear layer's are 8 rows apart in
    // one matrix, the gated pair's are the same rows of W1 and W3
    const uint8_t* q[2];
    const uint16_t* s[2];
    const uint8_t* z[2];  // or null: 8
    int64_t ldq[2], lds[2], ldz[2];
    const uint16_t* bias;
    const uint16_t* r;
    uint16_t* d;
    int64_t ldr, ldd;
    int m, n, k;
    int act;
    int x_type;
    int tiles;        // row tiles of the whole product
    int slice_units;  // units of a cluster's CTA: its columns are slice_units * kUnit
    int k_warps;      // warps that share a row tile, along k
    int tokens;       // of a pass: blockIdx.y's
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight nibbles to four bf16 pairs (i, i + 4) of q - z; `zero` holds 128 + z in both halves.
__device__ __forceinline__ void widen(uint32_t w, uint32_t zero, uint32_t (&out)[4]) {
    const __nv_bfloat162 z = *reinterpret_cast<const __nv_bfloat162*>(&zero);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = (w >> (4 * i) & 0x000f000fu) | 0x43004300u;
        const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), z);
        out[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
}

__device__ __forceinline__ float activate(float v, int act) {
    if (act == 1) {
        const float u = 0.7978845608028654f * (v + 0.044715f * v * v * v);
        return v / (1.f + __expf(-2.f * u));  // 0.5 (1 + tanh u) = 1 / (1 + exp(-2u))
    }
    if (act == 2) return v / (1.f + __expf(-v));
    if (act == 3) return v > 0.f ? v : (v != v ? v : 0.f);
    return v;
}

// The first column of chunk `c` (8 columns) of step `step` for lane quarter `t`: a lane's part of
// a group of G columns is G/4 contiguous ones.
template <int G>
__device__ __forceinline__ int chunk_column(int step, int c, int t) {
    constexpr int kPer = G / 32;  // chunks of a lane in a group
    return step * kStep + (c / kPer) * G + t * (G / 4) + (c % kPer) * 8;
}

// G: columns of a weight's scale.  NT: tokens / 8, rounded up.  GATED: the pair.  X8: x is e4m3.
template <int G, int NT, bool GATED, bool X8>
__global__ void __launch_bounds__(32 * kMaxWarps, NT == 4 ? 1 : 2) w4_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, threads = blockDim.x, warps = threads >> 5;
    const int warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const uint32_t rank = cluster_ctarank();
    uint32_t ranks;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
    const int cluster = blockIdx.x / ranks, clusters = gridDim.x / ranks;
    const int token0 = blockIdx.y * p.tokens, tokens = min(p.tokens, p.m - token0);
    const int unit0 = rank * p.slice_units;
    const int units = max(0, min(p.slice_units, (p.k + kUnit - 1) / kUnit - unit0));
    const int col_base = unit0 * kUnit;  // the slice's first column
    const int steps = units * (kUnit / kStep);

    // shared memory: x as 16-byte chunks [step][c][token][t], its scales [step][token], and the
    // warps' sums [2][warp][token][16]
    uint4* xs = reinterpret_cast<uint4*>(smem);
    float* scales = reinterpret_cast<float*>(smem + static_cast<size_t>(p.slice_units) * 4 * 16 * p.tokens * 16);
    float* sums = scales + (X8 ? p.slice_units * 4 * p.tokens : 0);
    const int sums_of_warp = NT * 8 * kRows, sums_of_buffer = warps * sums_of_warp;

    // x: the pairs (i, i + 4) of eight columns next to each other, as widen() gives the weights'
    for (int i = tid; i < steps * 16 * tokens; i += threads) {
        const int u = i % (16 * steps), token = i / (16 * steps);
        const int step = u >> 4, c = u >> 2 & 3, lt = u & 3;
        const int col = col_base + chunk_column<G>(step, c, lt);
        uint16_t e[8];
        if (col >= p.k) {
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = 0;
        } else if (X8) {
            const __nv_fp8_e4m3* src =
                static_cast<const __nv_fp8_e4m3*>(p.x) + (token0 + token) * p.ldx + col;
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = __bfloat16_as_ushort(__float2bfloat16_rn(static_cast<float>(src[j])));
        } else {
            const uint16_t* src = static_cast<const uint16_t*>(p.x) + (token0 + token) * p.ldx + col;
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = src[j];
        }
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = e[j] | static_cast<uint32_t>(e[j + 4]) << 16;
        xs[((step * 4 + c) * tokens + token) * 4 + lt] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (X8)
        for (int i = tid; i < steps * tokens; i += threads) {
            const int step = i / tokens, token = i % tokens;
            const int group = p.x_type == kXGroupScale ? min(col_base / kStep + step, (p.k - 1) / kStep) : 0;
            scales[step * tokens + token] = p.x_scale[(token0 + token) * p.ldxs + group];
        }
    __syncthreads();

    const int k_warps = p.k_warps, row_groups = warps / k_warps;
    const int k_part = warp % k_warps, row_group = warp / k_warps;
    constexpr int kOutRows = GATED ? 8 : kRows;  // outputs of a tile
    int buffer = 0;
    for (int first = cluster * row_groups; first < p.tiles; first += clusters * row_groups, buffer ^= 1) {
        const int tile = first + row_group;
        // rows past the last one read the last one; their results are not stored
        const int64_t row_a = min(static_cast<int64_t>(tile) * kOutRows + g, static_cast<int64_t>(p.n - 1));
        const int64_t row_b = GATED ? row_a : min(static_cast<int64_t>(tile) * kOutRows + g + 8, static_cast<int64_t>(p.n - 1));
        const uint8_t* qa = p.q[0] + row_a * p.ldq[0];
        const uint8_t* qb = p.q[1] + row_b * p.ldq[1];
        float total[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) total[j][i] = 0.f;

        for (int u = k_part; u < units; u += k_warps) {
            const int col_u = col_base + u * kUnit;
            for (int s = 0; s < kUnit / kStep; ++s) {
                const int step = u * (kUnit / kStep) + s, col_s = col_u + s * kStep;
                if (col_s >= p.k) break;
                float acc[NT][4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    constexpr int kPer = G / 32;
                    const int col = chunk_column<G>(0, c, t) + col_s;
                    const int group = (col_s + (c / kPer) * G) / G;
                    const bool in = col < p.k, group_in = group * G < p.k;
                    const uint32_t wa = in ? *reinterpret_cast<const uint32_t*>(qa + col / 2) : 0u;
                    const uint32_t wb = in ? *reinterpret_cast<const uint32_t*>(qb + col / 2) : 0u;
                    const uint32_t za =
                        0x43004300u + 0x00010001u * (p.z[0] && group_in ? p.z[0][row_a * p.ldz[0] + group] : 8u);
                    const uint32_t zb =
                        0x43004300u + 0x00010001u * (p.z[1] && group_in ? p.z[1][row_b * p.ldz[1] + group] : 8u);
                    if (c % kPer == 0) {
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
                    }
                    uint32_t a[4], b[4];
                    widen(wa, za, a);
                    widen(wb, zb, b);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        uint4 x = make_uint4(0, 0, 0, 0);
                        if (g + 8 * j < tokens) x = xs[((step * 4 + c) * tokens + g + 8 * j) * 4 + t];
                        mma16816(acc[j], a[0], b[0], a[1], b[1], x.x, x.y);
                        mma16816(acc[j], a[2], b[2], a[3], b[3], x.z, x.w);
                    }
                    if (c % kPer == kPer - 1 && group_in) {
                        const float sa = __uint_as_float(p.s[0][row_a * p.lds[0] + group] << 16);
                        const float sb = __uint_as_float(p.s[1][row_b * p.lds[1] + group] << 16);
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            const int tok = min(8 * j + 2 * t, tokens - 1), tok1 = min(8 * j + 2 * t + 1, tokens - 1);
                            const float x0 = X8 ? scales[step * tokens + tok] : 1.f;
                            const float x1 = X8 ? scales[step * tokens + tok1] : 1.f;
                            total[j][0] = fmaf(acc[j][0], sa * x0, total[j][0]);
                            total[j][1] = fmaf(acc[j][1], sa * x1, total[j][1]);
                            total[j][2] = fmaf(acc[j][2], sb * x0, total[j][2]);
                            total[j][3] = fmaf(acc[j][3], sb * x1, total[j][3]);
                        }
                    }
                }
            }
        }

        float* mine = sums + buffer * sums_of_buffer + warp * sums_of_warp;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) mine[(8 * j + 2 * t + (i & 1)) * kRows + g + (i & 2 ? 8 : 0)] = total[j][i];
        // One barrier a tile: a buffer is written again two tiles later, after the barrier between,
        // which every reader of the first reaches only when it has read.
        if (ranks > 1) cluster_sync();
        else __syncthreads();

        // the cluster's threads share the tile group's outputs; the parts are added in a fixed order
        const int outputs = row_groups * kOutRows * tokens;
        for (int i = rank * threads + tid; i < outputs; i += ranks * threads) {
            const int row = i % kOutRows, rest = i / kOutRows, rg = rest % row_groups, token = rest / row_groups;
            const int64_t n = static_cast<int64_t>(first + rg) * kOutRows + row;
            if (n >= p.n) continue;
            float v = 0.f, v3 = 0.f;
            for (uint32_t r = 0; r < ranks; ++r) {
                const uint32_t from = mapa_shared(smem_addr(sums + buffer * sums_of_buffer), r);
                for (int w = 0; w < k_warps; ++w) {
                    const uint32_t at = from + 4 * ((rg * k_warps + w) * sums_of_warp + token * kRows + row);
                    float f;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(at) : "memory");
                    v += f;
                    if (GATED) {
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(at + 32) : "memory");
                        v3 += f;
                    }
                }
            }
            const int64_t out = token0 + token;
            if (GATED) {
                v = activate(v, 2) * v3;
            } else {
                if (p.bias) v += __uint_as_float(static_cast<uint32_t>(p.bias[n]) << 16);
                v = activate(v, p.act);
                if (p.r) v += __uint_as_float(static_cast<uint32_t>(p.r[out * p.ldr + n]) << 16);
            }
            p.d[out * p.ldd + n] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
        }
    }
    if (ranks > 1) cluster_sync();  // no CTA leaves while another may read its sums
}

}  // namespace w4
}  // namespace gb
