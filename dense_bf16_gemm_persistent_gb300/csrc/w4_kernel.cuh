// Device code of the products with 4-bit weights for a few tokens.
//
//   W[n,k] = (q[n,k] - z[n,k/G]) s[n,k/G]          q, z in 0..15, G = 32, 64 or 128
//   D = act(x W^T + bias) + R        or        D = silu(x W1^T) * (x W3^T)
//
// Bound by the weights' bytes: every one is read once, and at the memory's rate an SM has one
// cycle for each 50 weights, so the instructions that widen them decide how near it comes.  The
// weights are copied as they are stored, and the contraction's order is chosen to fit: an
// mma.m16n8k16 may take any 16 columns k as long as both operands agree, so a lane's share of each
// group is contiguous in memory, and x is laid out in shared memory to match.  (tcgen05 would want
// the widened weights written to shared or tensor memory first, and a read of its accumulator for
// each group.)
//
// A nibble becomes an fp16 without a conversion: masked in place it is the subnormal q 2^-24, or
// q 2^-20 for the nibble one higher; five instructions widen eight weights.  The zero point is
// taken off the group's sum instead of off each weight,
//     sum (q - z) x = sum q x - z sum x,
// with sum x from the same instructions in the same order on weights of 8, so that weights at the
// zero point 8 (all there is without zeros) leave exactly nothing; weights at another zero point leave
// 2^-24 of z s sum |x| (measured).  x becomes fp16 too: e4m3 values exactly (times 2^4), and bf16
// values are first scaled by a power of two for each 128 columns of a token, so that the largest is in
// [2^14, 2^15); what is then lost, below 2^-35 of the largest, is under fp32's own rounding of
// the sum.  Products are summed in fp32 within a group, and the group's sum is multiplied by its
// scales in fp32: no weight is ever rounded.  What x holds of infinities and NaN is added one by one,
// slowly (sum x would make NaN of an infinity).
//
// Measured on a GB300: one token x 131072 x 8192 (G = 128) 96 us, 5.8 TB/s of the bytes that the
// product cannot do without, 0.85 of the copy bandwidth; 8 tokens 104 us (0.79); 16 tokens 166 us;
// 32 tokens 304 us.  The bytes of a unit for each of an SM's sixteen warps take 1.47 us at the
// memory's rate.  A token's pair 14336 x 4096 takes 16.4 us where its bytes take 8.9: launch, x's layout
// and three rounds' joins are, by the plan's model, the rest.  Steps on the way, 8 tokens: subtracting z
// from each weight 127.5 us, off the sums 120.6; tiles of 32 rows instead of 16, with the scales by row,
// the split-phase join and the pushed sums, 108.  A pass of 32 tokens took 464 us when one of 16 took 157.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "ptx.cuh"

namespace gb {
namespace w4 {

constexpr int kStep = 128;           // columns of one step: four lanes x 16 bytes of weights
constexpr int kUnit = 2 * kStep;     // columns that a warp loads at a time
constexpr int kRows = 32;            // weight rows of a tile: two of mma's, which share x's fragments
constexpr int kUnitBytes = kRows * kUnit / 2;  // weights of a unit: 32 rows of 128 bytes
// Warps of a CTA (one CTA an SM): more tokens and groups, more registers for them.  A warp multiplies a
// unit from registers while the next is on its way to its slot in shared memory (64 KB for an SM's
// sixteen warps: at the memory's rate it takes 1.4 us to consume that, longer than a load takes).
__host__ __device__ constexpr int warps_of(int group, int nt) { return nt == 1 ? 16 : group == 128 ? 12 : 8; }
constexpr int kMaxTokens = 16;       // of a pass: two mma tiles of eight

enum { kXBf16 = 0, kXRowScale = 1, kXGroupScale = 2 };

struct Params {
    const void* x;
    const float* x_scale;
    int64_t ldx, ldxs;
    // a tile's rows 0..15 and 16..31 come from two sources: a linear layer's are 16 rows apart in
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
    int wide_scales;  // every unit's scales and zeros of a row may be loaded as one word
    int x_type;
    int tiles;        // row tiles of the whole product
    int slice_units;  // units of a cluster's CTA: its columns are slice_units * kUnit
    int k_warps;      // warps that share a row tile, along k
    int tokens;       // of a pass: blockIdx.y's
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same on a sum of zero.
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Eight nibbles to four fp16 pairs (i, i + 4) of q 2^-24 (i even) or q 2^-20 (i odd).
__device__ __forceinline__ void widen(uint32_t w, uint32_t (&out)[4]) {
    const uint32_t high = w >> 8;
    out[0] = w & 0x000f000fu;
    out[1] = w & 0x00f000f0u;
    out[2] = high & 0x000f000fu;
    out[3] = high & 0x00f000f0u;
}

// The same of q - z, exactly; `zero` holds z in both halves: z 2^-24 as fp16.
__device__ __forceinline__ void widen_less(uint32_t w, uint32_t zero, uint32_t (&out)[4]) {
    const uint32_t zero16 = zero << 4;
    widen(w, out);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&out[i]),
                                  *reinterpret_cast<const __half2*>(i & 1 ? &zero16 : &zero));
        out[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
}
// What the products are short of for that: 2^24, and 2^-4 in the odd columns of x.  Half of the 2^24 is
// in the weights' scale and half in x's, so that neither overflows; the scales of e4m3 values, which
// may be as large as 2^119, have 2^8 of theirs, and the values themselves 2^4.
constexpr float kHalfShift = 4096.f, kX8Shift = 256.f;

__device__ __forceinline__ float activate(float v, int act) {
    if (act == 1) {
        const float u = 0.7978845608028654f * (v + 0.044715f * v * v * v);
        return v / (1.f + __expf(-2.f * u));  // 0.5 (1 + tanh u) = 1 / (1 + exp(-2u))
    }
    if (act == 2) return v / (1.f + __expf(-v));
    if (act == 3) return v > 0.f ? v : (v != v ? v : 0.f);
    return v;
}

// The two halves of the barrier of a cluster's threads (a cluster of one CTA has one too), in the
// form that does not ask for converged warps.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Zeros where `in` is false: nothing is read.
__device__ __forceinline__ void copy_async_or_zero(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void load_shared(uint32_t at, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(at) : "memory");
}
__device__ __forceinline__ void load_shared(uint32_t at, uint32_t& a, uint32_t& b) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(at) : "memory");
}
__device__ __forceinline__ void load_shared(uint32_t at, uint32_t& a) {
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(a) : "r"(at) : "memory");
}
__device__ __forceinline__ void store_shared(uint32_t at, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ float load_shared_float(uint32_t at) {
    float f;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(at) : "memory");
    return f;
}
// To the shared memory of a CTA of the cluster.
__device__ __forceinline__ void store_cluster(uint32_t at, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

__device__ __forceinline__ uint32_t half_pair(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Eight columns of a token from `col` on (zeros past the end): bf16 pairs, or e4m3 quads in the
// first two words.
template <bool X8>
__device__ __forceinline__ void load_x(const Params& p, bool wide, int token, int col, bool in, uint32_t (&w)[4]) {
    w[0] = w[1] = w[2] = w[3] = 0;
    if (!in) return;
    if (X8) {
        const uint8_t* src = static_cast<const uint8_t*>(p.x) + token * p.ldx + col;
        if (wide) {
            const uint2 e = *reinterpret_cast<const uint2*>(src);
            w[0] = e.x;
            w[1] = e.y;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j / 4] |= static_cast<uint32_t>(src[j]) << (8 * (j & 3));
        }
    } else {
        const uint16_t* src = static_cast<const uint16_t*>(p.x) + token * p.ldx + col;
        if (wide) {
            const uint4 e = *reinterpret_cast<const uint4*>(src);
            w[0] = e.x;
            w[1] = e.y;
            w[2] = e.z;
            w[3] = e.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = src[2 * j] | static_cast<uint32_t>(src[2 * j + 1]) << 16;
        }
    }
}

// x of a CTA's slice to shared memory: 16-byte chunks [step][c][token][t], in each the pairs
// (i, i + 4) of eight columns as widen() gives the weights'; and what the sums are to be multiplied
// by, in `xscale` [step][token of NT eights], or with kXRowScale [token].  bf16 values that are not
// finite are left out (as zeros); returns whether the thread had none.
template <int G, int NT, int X>
__device__ __forceinline__ bool stage_x(const Params& p, uint4* xs, float* xscale, int col_base, int steps, int token0,
                                        int tokens) {
    constexpr int kPer = G / 32;
    constexpr bool X8 = X != kXBf16;
    const bool wide = (reinterpret_cast<uintptr_t>(p.x) & (X8 ? 7 : 15)) == 0 && (p.ldx & 7) == 0;
    const int at = threadIdx.x & 15, stride = blockDim.x >> 4;
    const int group = at / (4 * kPer), lt = at / kPer & 3, c = group * kPer + at % kPer;
    const int total = steps * tokens;  // a step of a token is sixteen lanes, which agree on its scale
    constexpr int kBatch = 4;          // loads that a thread has on their way
    bool finite = true;
    for (int i = threadIdx.x >> 4; (i & ~1) < total; i += kBatch * stride) {
        uint32_t w[kBatch][4];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int at_u = i + u * stride, token = at_u / steps, col = col_base + (at_u - token * steps) * kStep + at * 8;
            load_x<X8>(p, wide, token0 + token, col, at_u < total && col < p.k, w[u]);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int at_u = i + u * stride, token = at_u / steps, step = at_u - token * steps;
            if ((at_u & ~1) >= total) break;  // (of the whole warp)
            float v[8], scale = X8 ? kX8Shift : kHalfShift;
            if (X8) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    __nv_fp8x2_e4m3 pair;
                    pair.__x = static_cast<__nv_fp8x2_storage_t>(w[u][j / 2] >> (16 * (j & 1)));
                    const float2 f = static_cast<float2>(pair);
                    v[2 * j] = f.x;
                    v[2 * j + 1] = f.y;
                }
                if (at == 0 && at_u < total && (X == kXGroupScale || step == 0)) {
                    const int column = X == kXGroupScale ? min(col_base / kStep + step, (p.k - 1) / kStep) : 0;
                    scale *= p.x_scale[(token0 + token) * p.ldxs + column];
                }
            } else {
                uint32_t top = 0;  // the largest finite exponent
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t lo = w[u][j] >> 7 & 0xff, hi = w[u][j] >> 23 & 0xff;
                    finite = finite && lo != 0xff && hi != 0xff;
                    top = max(top, max(lo == 0xff ? 0u : lo, hi == 0xff ? 0u : hi));
                    v[2 * j] = lo == 0xff ? 0.f : __uint_as_float(w[u][j] << 16);
                    v[2 * j + 1] = hi == 0xff ? 0.f : __uint_as_float(w[u][j] & 0xffff0000u);
                }
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
                // 2^(14 - (top - 127)), below 2^127; its reciprocal goes to the sum
                const uint32_t up = min(268u - top, 253u);
                const float f = __uint_as_float(up << 23);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] *= f;
                scale *= __uint_as_float((254u - up) << 23);
            }
            if (at_u >= total) continue;
            constexpr float kEven = X8 ? kHalfShift / kX8Shift : 1.f, kOdd = kEven / 16.f;
            xs[((step * 4 + c) * tokens + token) * 4 + lt] =
                make_uint4(half_pair(v[0] * kEven, v[4] * kEven), half_pair(v[1] * kOdd, v[5] * kOdd),
                           half_pair(v[2] * kEven, v[6] * kEven), half_pair(v[3] * kOdd, v[7] * kOdd));
            if (at == 0 && X != kXRowScale) xscale[step * 8 * NT + token] = scale;
            if (at == 0 && X == kXRowScale && step == 0) xscale[token] = scale;
        }
    }
    return finite;
}

// Sums of x over a group, in `xsum` [group][token of NT eights]: an eighth of the group's products
// with weights of q = 8, by the instructions and in the order of the products with the weights.
template <int G, int NT>
__device__ __forceinline__ void sum_x(const uint4* xs, float* xsum, int groups, int tokens) {
    constexpr int kPer = G / 32, kStepGroups = kStep / G;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    for (int i = threadIdx.x >> 5; i < groups; i += blockDim.x >> 5) {
        __syncwarp();
        const int chunk = i / kStepGroups * 4 + i % kStepGroups * kPer;
        float acc[NT][4];
#pragma unroll
        for (int c = 0; c < kPer; ++c)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint4 x = xs[((chunk + c) * tokens + min(g + 8 * j, tokens - 1)) * 4 + t];
                const uint32_t eight = 0x00080008u, eight16 = 0x00800080u;
                if (c == 0) mma16816_first(acc[j], eight, eight, eight16, eight16, x.x, x.y);
                else mma16816(acc[j], eight, eight, eight16, eight16, x.x, x.y);
                mma16816(acc[j], eight, eight, eight16, eight16, x.z, x.w);
            }
        if (g == 0) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                xsum[i * 8 * NT + 8 * j + 2 * t] = acc[j][0] * 0.125f;
                xsum[i * 8 * NT + 8 * j + 2 * t + 1] = acc[j][1] * 0.125f;
            }
        }
    }
}

// What a token's infinities and NaN add to row n of matrix `from`: those of `units` units of columns,
// the first at `first` and the others `step` apart.
template <int G>
__device__ __noinline__ float odd_part(const Params& p, int from, int64_t n, int64_t token, int first, int units, int step) {
    float sum = 0.f;
    for (int i = 0; i < units; ++i, first += step)
        for (int col = first; col < min(first + kUnit, p.k); ++col) {
            const uint32_t x = static_cast<const uint16_t*>(p.x)[token * p.ldx + col];
            if ((x >> 7 & 0xff) != 0xff) continue;
            const int q = p.q[from][n * p.ldq[from] + col / 2] >> (4 * (col & 1)) & 15;
            const int z = p.z[from] ? p.z[from][n * p.ldz[from] + col / G] & 15 : 8;
            const float s = __uint_as_float(static_cast<uint32_t>(p.s[from][n * p.lds[from] + col / G]) << 16);
            sum += __uint_as_float(x << 16) * (static_cast<float>(q - z) * s);
        }
    return sum;
}

// A warp's place in its sequence of (row tile, unit), and the addresses that go with it.
template <bool GATED>
struct Cursor {
    int tile;           // row tile
    int unit;           // of the slice
    const uint8_t* qa;  // the lane's first row of each half of the tile, and its 16 bytes of a unit
    const uint8_t* qb;
    const uint16_t* s;  // scales and zeros of the row that the lane fetches
    const uint8_t* z;

    __device__ __forceinline__ void at_tile(const Params& p, int to, int lane) {
        tile = to;
        // (a product's last row tile may end past 2^31 - 1: unsigned)
        const uint32_t first = static_cast<uint32_t>(to) * (GATED ? 16 : 32), last = p.n - 1;
        const int64_t copied = first + (lane >> 3);
        qa = p.q[0] + copied * p.ldq[0] + (lane & 7) * 16;
        qb = p.q[1] + (GATED ? copied : copied + 16) * p.ldq[1] + (lane & 7) * 16;
        // lane l has the tile's row l: a row past the last reads the last one's
        const int from = lane >> 4;
        const int64_t at = min(first + (GATED ? lane & 15 : lane), last);
        s = p.s[from] + at * p.lds[from];
        z = p.z[from] ? p.z[from] + at * p.ldz[from] : nullptr;
    }
    // Rows of the tile's half that exist.
    __device__ __forceinline__ int rows(const Params& p, int half) const {
        const int64_t first = static_cast<int64_t>(tile) * (GATED ? 16 : 32) + (GATED ? 0 : 16 * half);
        return static_cast<int>(max(static_cast<int64_t>(0), min(p.n - first, static_cast<int64_t>(16))));
    }
};

// G: columns of a weight's scale.  NT: tokens / 8, rounded up.  GATED: the pair.  X: x's type.
//
// A CTA's warps form teams of k_warps; a team takes row tiles in turn and its warps share the
// tile's units.  Each warp streams its units through a slot of its own in shared memory with
// 16-byte cp.async, which runs ahead over the ends of tiles; no barrier but the warp's own.
//
// Which lanes may be apart at an instruction that a whole warp has to execute: none.  What decides
// whether such an instruction is reached is the same in every lane: in stage_x the loop's end and
// its break go by i & ~1, the same for a warp's two halves (its shuffles are under nothing else);
// sum_x's loop and the loops over tiles and units go by the warp's and the team's number.  Lanes part
// only between those (a token or a row past the last, the one lane of sixteen that fetches a scale, a
// matrix with zeros beside one without, the outputs that a lane adds up), and every such stretch ends
// in a __syncwarp before the next mma or barrier of the CTA's threads, or holds no wait and no
// exit, so that the lanes meet behind it.  The cluster's barriers are of the form that does not ask
// for converged warps, and every thread of every CTA comes to each of them: the loop over tiles runs
// the same number of rounds in all CTAs of a cluster (`first` and `tile_step` go by the cluster), at
// least one (there are no more clusters than groups of tiles).
template <int G, int NT, bool GATED, int X>
__global__ void __launch_bounds__(32 * warps_of(G, NT), 1) w4_kernel(const __grid_constant__ Params p) {
    constexpr bool kStepScale = X != kXRowScale;  // x has a scale for each step
    constexpr int kPer = G / 32;         // words of a lane in a group
    constexpr int kGroups = kUnit / G;   // of a unit: what a lane fetches the scales of, for one row
    constexpr int kStepGroups = kStep / G;
    constexpr int kOutRows = GATED ? 16 : 32;
    // z off each weight takes 16 G / 32 instructions a group, off the sums 8 NT
    constexpr bool kLess = 2 * G / 32 <= NT;
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, warps = blockDim.x >> 5;
    const int warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const uint32_t rank = cluster_ctarank();
    uint32_t ranks;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
    if (ranks > 1) cluster_arrive();  // (waited for before the first store to another CTA)
    allow_next_kernel();
    const int cluster = blockIdx.x / ranks, clusters = gridDim.x / ranks;
    const int token0 = blockIdx.y * p.tokens, tokens = min(p.tokens, p.m - token0);
    const int unit0 = rank * p.slice_units;
    const int units = max(0, min(p.slice_units, (p.k + kUnit - 1) / kUnit - unit0));
    const int col_base = unit0 * kUnit;  // the slice's first column
    const int steps = units * (kUnit / kStep);

    // shared memory: the slots, x, its scales and sums, the scales of
    // each warp's unit, and the sums that this CTA adds up
    const uint32_t slot = smem_addr(smem) + warp * kUnitBytes;
    uint4* xs = reinterpret_cast<uint4*>(smem + warps * kUnitBytes);
    float* xscale = reinterpret_cast<float*>(xs + static_cast<size_t>(p.slice_units) * (kUnit / 8) * p.tokens);
    float* xsum = xscale + (kStepScale ? p.slice_units * (kUnit / kStep) : 1) * 8 * NT;

    const uint32_t all_scales = smem_addr(xsum + p.slice_units * kGroups * 8 * NT);
    const uint32_t scales_of_warp = all_scales + warp * kGroups * 128, sums = all_scales + warps * kGroups * 128;

    const int k_warps = p.k_warps, teams = warps / k_warps;
    const int k_part = warp % k_warps, team = warp / k_warps;
    const int groups = (p.k + G - 1) / G;

    // A slot holds 32 rows of 128 bytes.  A row's eight 16-byte chunks are swapped by
    // swap(row), so that neither the copies (four rows a warp) nor the reads (4, 8 or 16 bytes a
    // lane of eight rows: its part of a group) meet in a bank.
    auto swap = [](uint32_t row) { return (row & 1) << 2 | (row & 2) | (row >> 2 & 1); };
    auto fetch = [&](const Cursor<GATED>& c) {
        const int col_u = col_base + c.unit * kUnit;
        const uint32_t to = slot + (lane >> 3) * 128;
        // rows lane / 8 + 4i: the swap of i odd differs in its lowest bit
        const uint32_t even = ((lane & 7) ^ swap(lane >> 3)) << 4, odd = even ^ 16;
        const uint8_t *a = c.qa + col_u / 2, *b = c.qb + col_u / 2;
        if (col_u + kUnit <= p.k && (c.tile + 1) * static_cast<int64_t>(kOutRows) <= p.n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                copy_async(to + i * 512 + (i & 1 ? odd : even), a + i * 4 * p.ldq[0]);
                copy_async(to + 2048 + i * 512 + (i & 1 ? odd : even), b + i * 4 * p.ldq[1]);
            }
        } else {
            const bool in = col_u + (lane & 7) * 32 < p.k;
            const int rows_a = in ? c.rows(p, 0) : 0, rows_b = in ? c.rows(p, 1) : 0, first = lane >> 3;
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                const bool in_a = first + 4 * i < rows_a, in_b = first + 4 * i < rows_b;
                copy_async_or_zero(to + i * 512 + (i & 1 ? odd : even), in_a ? a + i * 4 * p.ldq[0] : p.q[0], in_a);
                copy_async_or_zero(to + 2048 + i * 512 + (i & 1 ? odd : even), in_b ? b + i * 4 * p.ldq[1] : p.q[1],
                                   in_b);
            }
        }
    };
    // Scales (bf16 pairs) and zeros (bytes) of the lane's row, for the unit on its way: one load each where every row's are aligned to it, else element by element.
    constexpr int kScaleWords = kGroups / 2, kZeroWords = (kGroups + 3) / 4;
    struct Raw {
        uint32_t s[kScaleWords], z[kZeroWords];
    };
    Raw raw;
#pragma unroll
    for (int i = 0; i < kZeroWords; ++i) raw.z[i] = 0x08080808u;
    auto fetch_scales = [&](const Cursor<GATED>& c, Raw& to) {
        const int first = (col_base + c.unit * kUnit) / G;
        const uint16_t* s = c.s + first;
        const uint8_t* z = c.z ? c.z + first : nullptr;
        if (p.wide_scales && first + kGroups <= groups) {
            if constexpr (kScaleWords == 1) {
                to.s[0] = *reinterpret_cast<const uint32_t*>(s);
                if (z) to.z[0] = *reinterpret_cast<const uint16_t*>(z);
            } else if constexpr (kScaleWords == 2) {
                const uint2 v = *reinterpret_cast<const uint2*>(s);
                to.s[0] = v.x;
                to.s[1] = v.y;
                if (z) to.z[0] = *reinterpret_cast<const uint32_t*>(z);
            } else {
                const uint4 v = *reinterpret_cast<const uint4*>(s);
                to.s[0] = v.x;
                to.s[1] = v.y;
                to.s[2] = v.z;
                to.s[3] = v.w;
                if (z) {
                    const uint2 u = *reinterpret_cast<const uint2*>(z);
                    to.z[0] = u.x;
                    to.z[1] = u.y;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kScaleWords; ++i) {
                const uint32_t lo = first + 2 * i < groups ? s[2 * i] : 0u;
                to.s[i] = lo | (first + 2 * i + 1 < groups ? static_cast<uint32_t>(s[2 * i + 1]) << 16 : 0u);
            }
            if (z) {
#pragma unroll
                for (int i = 0; i < kZeroWords; ++i) to.z[i] = 0;
#pragma unroll
                for (int i = 0; i < kGroups; ++i)
                    to.z[i / 4] |= first + i < groups ? static_cast<uint32_t>(z[i]) << (8 * (i & 3)) : 0u;
            }
        }
    };

    const int mine = units > k_part ? (units - k_part + k_warps - 1) / k_warps : 0;  // units of a tile
    const int tile_step = clusters * teams;
    Cursor<GATED> ahead;  // the unit whose copies are started next
    ahead.at_tile(p, cluster * teams + team, lane);
    ahead.unit = k_part;
    // While the kernels before still run: the first unit's rows (one a lane) to L2, where a later
    // write of theirs would be seen all the same.
    if (mine > 0 && ahead.tile < p.tiles) {
        const int64_t first = static_cast<int64_t>(ahead.tile) * kOutRows;
        const int64_t row = min(first + (GATED ? lane & 15 : lane), static_cast<int64_t>(p.n - 1));
        const int from = lane >> 4;
        const uint8_t* line = p.q[from] + row * p.ldq[from] + (col_base + k_part * kUnit) / 2;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(line));
    }
    wait_for_earlier_kernels();
    auto start_next = [&] {
        if (ahead.tile < p.tiles) {
            fetch(ahead);
            fetch_scales(ahead, raw);
            ahead.unit += k_warps;
            if (ahead.unit >= units) {
                ahead.unit = k_part;
                ahead.at_tile(p, ahead.tile + tile_step, lane);
            }
        }
        copy_commit();
    };
    if (mine > 0) start_next();

    // (a CTA past the last column has nothing, times nothing)
    if (steps == 0 && !kStepScale && tid < 8 * NT) xscale[tid] = 0.f;
    const bool finite = stage_x<G, NT, X>(p, xs, xscale, col_base, steps, token0, tokens);
    bool odd = false;
    __syncwarp();  // (a warp's two halves may have left the loop apart)
    if constexpr (X != kXBf16) __syncthreads();
    else odd = __syncthreads_or(!finite);
    if (!kLess) {
        sum_x<G, NT>(xs, xsum, steps * kStepGroups, tokens);
        __syncwarp();
        __syncthreads();
    }

    // where a lane reads its part of a row's groups; x's chunks of a token are four lanes apart
    uint32_t x_token[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) x_token[i] = smem_addr(xs) + (4 * min(g + 8 * i, tokens - 1) + t) * 16;
    const uint32_t scales_lane = smem_addr(xscale) + t * 8, sums_lane = smem_addr(xsum) + t * 8;
    // A tile's outputs are shared out over the cluster's CTAs, by octets of rows and then by tokens:
    // every warp puts its sums into the shared memory of the CTA that adds them up.  The cluster's
    // threads meet once a tile, in two halves: a warp leaves its sums, arrives, multiplies the next
    // tile, and only then waits for the others and adds up its share of the tile before.  A buffer is
    // written again two tiles later: after the wait that follows every other thread's reading of it.
    // A share: octets o with o >> octet_drop == rank >> token_bits (of the two or four kinds of
    // octets; the gated pair's W1 and W3 octets of the same rows go together), tokens whose low
    // token_bits are the rank's; in memory [buffer][team][CTA][warp][token][row].
    constexpr int kKinds = GATED ? 2 : 4, kKindBits = GATED ? 1 : 2;
    const int rank_bits = 31 - __clz(ranks);
    const int token_bits = max(0, rank_bits - kKindBits), octet_drop = max(0, kKindBits - rank_bits);
    const int share_octets = kKinds >> (rank_bits - token_bits), share_rows = share_octets * 8 * (GATED ? 2 : 1);
    const int share_tokens = (tokens + (1 << token_bits) - 1) >> token_bits;
    const uint32_t share_bytes = ((p.tokens + (1 << token_bits) - 1) >> token_bits) * share_rows * 4;
    const uint32_t team_sums = sums + team * ranks * k_warps * share_bytes;
    const uint32_t buffer_bytes = teams * ranks * k_warps * share_bytes;
    const int my_octet = (rank >> token_bits) << octet_drop, my_token = rank & ((1 << token_bits) - 1);
    const int out_rows = share_octets * 8, outputs = out_rows * share_tokens;
    uint16_t bias0 = 0, r0 = 0;  // of the thread's first output of the tile before
    const int out0 = k_part * 32 + lane;
    auto output_row = [&](int tile, int i) {
        return static_cast<int64_t>(tile) * kOutRows + my_octet * 8 + i % out_rows;
    };
    auto output_token = [&](int i) { return ((i / out_rows) << token_bits) + my_token; };
    auto finish = [&](int tile, uint32_t buffer) {
        for (int i = out0; i < outputs; i += k_warps * 32) {
            const int64_t n = output_row(tile, i);
            const int token = output_token(i);
            if (n >= p.n || token >= tokens) continue;
            float v = 0.f, v3 = 0.f;
            const uint32_t from = team_sums + buffer * buffer_bytes + 4 * (i / out_rows * share_rows + i % out_rows);
            const int parts = ranks * k_warps;  // added in a fixed order
#pragma unroll 4
            for (int w = 0; w < parts; ++w) {
                v += load_shared_float(from + w * share_bytes);
                if (GATED) v3 += load_shared_float(from + w * share_bytes + 4 * out_rows);
            }
            const int64_t out = token0 + token;
            if (GATED) {
                v = activate(v, 2) * v3;
            } else {
                const bool pre = i == out0;
                if (p.bias) v += __uint_as_float(static_cast<uint32_t>(pre ? bias0 : p.bias[n]) << 16);
                v = activate(v, p.act);
                if (p.r) v += __uint_as_float(static_cast<uint32_t>(pre ? r0 : p.r[out * p.ldr + n]) << 16);
            }
            p.d[out * p.ldd + n] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
        }
        __syncwarp();
    };
    auto leave = [&](int tile, const float (&total)[2][NT][4], uint32_t buffer) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int kind = GATED ? r & 1 : r, owner0 = (kind >> octet_drop) << token_bits;
            const int row = GATED ? (r >> 1) * out_rows + (kind & (share_octets - 1)) * 8 + g
                                  : (kind & (share_octets - 1)) * 8 + g;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int token = 8 * j + 2 * t + i;
                    if (token >= tokens) continue;
                    const uint32_t at = team_sums + buffer * buffer_bytes + (rank * k_warps + k_part) * share_bytes +
                                        4 * ((token >> token_bits) * share_rows + row);
                    float v = total[r / 2][j][i + r % 2 * 2];
                    if (!kStepScale) v *= load_shared_float(scales_lane - t * 8 + 4 * token);
                    if (X == kXBf16 && odd) {
                        const int64_t n = static_cast<int64_t>(tile) * kOutRows + (GATED ? kind * 8 : r * 8) + g;
                        if (n < p.n)
                            v += odd_part<G>(p, GATED ? r >> 1 : 0, n, token0 + token, col_base + k_part * kUnit, mine,
                                             k_warps * kUnit);
                    }
                    store_cluster(mapa_shared(at, owner0 + (token & ((1 << token_bits) - 1))), v);
                }
        }
    };

    if (ranks > 1) cluster_wait();
    uint32_t buffer = 0;
    int before = -1;
    for (int first = cluster * teams; first < p.tiles; first += tile_step) {
        const int tile = first + team;
        float total[2][NT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) total[h][j][i] = 0.f;

        for (int n = 0; n < mine && tile < p.tiles; ++n) {
            const int unit = k_part + n * k_warps;
            // scale (times 2^12) and zero point of each group and row, as two bf16, to shared memory:
            // [group][g][row / 8], so that a lane reads those of its four rows at once
            __syncwarp();  // (every lane is done with the last unit)
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                const uint32_t pair = raw.s[i / 2], z = raw.z[i / 4] >> (8 * (i & 3)) & 15;
                const float scale = __uint_as_float(i & 1 ? pair & 0xffff0000u : pair << 16) * kHalfShift;
                store_shared(scales_of_warp + i * 128 + (lane & 7) * 16 + (lane >> 3) * 4,
                             __float_as_uint(scale) | __float_as_uint(static_cast<float>(z)) >> 16);
            }
            copy_wait<0>();
            __syncwarp();  // the unit is there
            const uint32_t w_at = slot + g * 128;
            // words of rows g, g + 8, g + 16, g + 24 of a group
            auto load_group = [&](int s, int j, uint32_t (&to)[4][kPer]) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint32_t row = w_at + r * 1024;
                    if constexpr (G == 128)
                        load_shared(row + (((4 * s + t) ^ swap(g)) << 4), to[r][0], to[r][1], to[r][2], to[r][3]);
                    else if constexpr (G == 64)
                        load_shared(row + (((4 * s + 2 * j + (t >> 1)) ^ swap(g)) << 4) + (t & 1) * 8, to[r][0], to[r][1]);
                    else
                        load_shared(row + (((4 * s + j) ^ swap(g)) << 4) + t * 4, to[r][0]);
                }
            };
            uint32_t w[kGroups][4][kPer];
#pragma unroll
            for (int f = 0; f < kGroups; ++f) load_group(f / kStepGroups, f % kStepGroups, w[f]);
            __syncwarp();  // the slot may take the next copies
            start_next();

            uint32_t x_at = unit * (kUnit / 8) * 16 * tokens;
            uint32_t scale_at = scales_lane + (kStepScale ? unit * (kUnit / kStep) * 32 * NT : 0);
            uint32_t sums_at = sums_lane + unit * kGroups * 32 * NT;
            auto multiply = [&](int s) {
                float xs0[NT], xs1[NT];  // x's scales of the step, for the lane's two tokens of each eight
                if (kStepScale) {
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        uint32_t e[2];
                        load_shared(scale_at + i * 32, e[0], e[1]);
                        xs0[i] = __uint_as_float(e[0]);
                        xs1[i] = __uint_as_float(e[1]);
                    }
                }
#pragma unroll
                for (int j = 0; j < kStepGroups; ++j) {
                    const uint32_t (&ws)[4][kPer] = w[j];
                    float acc[2][NT][4];
                    uint32_t row_sz[4], zero[4];  // of rows g, g + 8, g + 16, g + 24
                    load_shared(scales_of_warp + (s * kStepGroups + j) * 128 + g * 16, row_sz[0], row_sz[1], row_sz[2],
                                row_sz[3]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if (kLess) zero[r] = static_cast<uint32_t>(__uint_as_float(row_sz[r] << 16)) * 0x00010001u;
                    }
#pragma unroll
                    for (int c = 0; c < kPer; ++c) {
                        uint32_t q[4][4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            if (kLess) widen_less(ws[r][c], zero[r], q[r]);
                            else widen(ws[r][c], q[r]);
                        }
#pragma unroll
                        for (int i = 0; i < NT; ++i) {
                            // (a token past the last one has another's values: its sums are not stored)
                            uint32_t x[4];
                            load_shared(x_token[i] + x_at + (j * kPer + c) * 64 * tokens, x[0], x[1], x[2], x[3]);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t (&a)[4] = q[2 * h], (&b)[4] = q[2 * h + 1];
                                if (c == 0) mma16816_first(acc[h][i], a[0], b[0], a[1], b[1], x[0], x[1]);
                                else mma16816(acc[h][i], a[0], b[0], a[1], b[1], x[0], x[1]);
                            }
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t (&a)[4] = q[2 * h], (&b)[4] = q[2 * h + 1];
                                mma16816(acc[h][i], a[2], b[2], a[3], b[3], x[2], x[3]);
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        uint32_t sum[2] = {0, 0};  // of x, for the lane's two tokens of each eight
                        if (!kLess) load_shared(sums_at + (j * NT + i) * 32, sum[0], sum[1]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float z = __uint_as_float(row_sz[r] << 16);
                            const float scale = __uint_as_float(row_sz[r] & 0xffff0000u);
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float v = acc[r / 2][i][r % 2 * 2 + e];
                                if (!kLess) v = fmaf(-z, __uint_as_float(sum[e]), v);
                                float& to = total[r / 2][i][r % 2 * 2 + e];
                                // (the sum meets one scale and then the other: the two scales' product
                                // need not be finite where the result is)
                                if (kStepScale) to = fmaf(v * scale, e ? xs1[i] : xs0[i], to);
                                else to = fmaf(scale, v, to);
                            }
                        }
                    }
                }
                x_at += 256 * tokens;
                scale_at += NT * 32;
                sums_at += kStepGroups * NT * 32;
            };
            // (rolled where it fits the registers: fewer instructions to fetch)
#pragma unroll(G == 32 ? 2 : 1)
            for (int s = 0; s < kUnit / kStep; ++s) {
                multiply(s);
#pragma unroll
                for (int f = 0; f + kStepGroups < kGroups; ++f)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int c = 0; c < kPer; ++c) w[f][r][c] = w[f + kStepGroups][r][c];
            }
        }

        if (before >= 0) {
            cluster_wait();
            finish(before, buffer ^ 1);
        }
        leave(tile, total, buffer);
        cluster_arrive();
        before = tile;
        buffer ^= 1;
        if (!GATED && out0 < outputs) {
            const int64_t n = output_row(tile, out0);
            const int token = output_token(out0);
            if (n < p.n && token < tokens) {
                if (p.bias) bias0 = p.bias[n];
                if (p.r) r0 = p.r[(token0 + token) * p.ldr + n];
            }
        }
        __syncwarp();
    }
    cluster_wait();
    finish(before, buffer ^ 1);
    copy_wait<0>();
}

}  // namespace w4
}  // namespace gb
