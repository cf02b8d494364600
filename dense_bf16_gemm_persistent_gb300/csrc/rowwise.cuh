// Device code of the operators that walk the rows of a bf16 matrix: dropout from a
// counter-based generator, the root-mean-square norm with the residual's addition, and the
// norm's backward pass.
//
// All three are bound by memory (4 to 10 bytes an element and a few dozen instructions), so
// each row is read once in 16-byte loads, kept in registers, and written once.
//
// Chunks.  A row is cut at the 16-byte boundaries of ITS addresses, not at its first column:
// with `shift` elements between the boundary below the row and its first element, chunk j
// holds the columns 8j - shift .. 8j - shift + 7.  Rows of an odd width then still move in
// full 16-byte words except for their first and last chunk.  That needs every matrix of the
// call to have the same shift on the same row; where they differ (the host's check), every
// chunk moves element by element.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace gb {
namespace rowwise {

// ---------------------------------------------------------------- the generator

// Philox4x32 with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy
// as 1, 2, 3", SC 2011): each round multiplies two of the counter's words by constants, and
// crosses the products' halves with the others and the key, which then moves on by its Weyl
// increments.  Element (row, col) of a matrix takes word col % 4 of the counter
// (col / 4, row, offset low, offset high) under the key `seed`.
struct Key {
    uint32_t k0, k1, c2, c3;
};

__device__ __forceinline__ void philox(uint32_t c0, uint32_t c1, const Key& key, uint32_t (&out)[4]) {
    uint32_t c2 = key.c2, c3 = key.c3, k0 = key.k0, k1 = key.k1;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u, b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
        c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
        c1 = static_cast<uint32_t>(b);
        c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
        c3 = static_cast<uint32_t>(a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    out[0] = c0;
    out[1] = c1;
    out[2] = c2;
    out[3] = c3;
}

// What dropout needs: an element is kept when its word is at least `threshold` = p 2^32 (64
// bits: p = 1 keeps nothing), and a kept one is multiplied by `scale` = 1 / (1 - p).
struct Drop {
    uint64_t threshold;
    uint64_t seed, offset;
    const uint64_t* state;  // device memory {seed, offset} that takes the place of the two above, or null
    float scale;
};

__device__ __forceinline__ Key drop_key(const Drop& d) {
    const uint64_t seed = d.state ? d.state[0] : d.seed, offset = d.state ? d.state[1] : d.offset;
    return Key{static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32), static_cast<uint32_t>(offset),
               static_cast<uint32_t>(offset >> 32)};
}

// Drop the chunk of `row` that starts at column `col0` (-7 at least).  A dropped element is
// zero whatever it was (an infinity or a NaN among them), so it is selected, not multiplied.
__device__ __forceinline__ void drop_chunk(float (&v)[8], int row, int col0, const Drop& d, const Key& key) {
    // a column below 0 is not an element: its word is not used, and the group -1 or -2 wraps
    const int phase = col0 & 3;
    const uint32_t group = static_cast<uint32_t>((col0 - phase) >> 2);
    uint32_t w[12];
    auto words = [&](int at) {
        uint32_t o[4];
        philox(group + at, static_cast<uint32_t>(row), key, o);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[4 * at + i] = o[i];
    };
    words(0);
    words(1);
    if (phase) {  // (the same for the whole row)
        words(2);
#pragma unroll
        for (int i = 0; i < 10; ++i) w[i] = phase & 2 ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < 9; ++i) w[i] = phase & 1 ? w[i + 1] : w[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = w[i] >= d.threshold ? v[i] * d.scale : 0.f;
}

// ---------------------------------------------------------------- chunks

__device__ __forceinline__ void unpack(const uint4& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The chunk's elements of `row` (0 outside the row).  The element-by-element loops are kept
// rolled: they run on a row's two ends (and on rows whose matrices are not aligned alike).
__device__ __forceinline__ uint4 load_chunk(const uint16_t* row, int col0, int cols, bool wide) {
    if (wide && col0 >= 0 && col0 + 8 <= cols) return *reinterpret_cast<const uint4*>(row + col0);
    uint4 u = make_uint4(0, 0, 0, 0);
#pragma unroll 1
    for (int i = 7; i >= 0; --i) {
        const int col = col0 + i;
        const uint32_t e = col >= 0 && col < cols ? row[col] : 0;
        u.w = __funnelshift_l(u.z, u.w, 16);
        u.z = __funnelshift_l(u.y, u.z, 16);
        u.y = __funnelshift_l(u.x, u.y, 16);
        u.x = u.x << 16 | e;
    }
    return u;
}

__device__ __forceinline__ void store_chunk(uint16_t* row, int col0, int cols, bool wide, uint4 u) {
    if (wide && col0 >= 0 && col0 + 8 <= cols) {
        *reinterpret_cast<uint4*>(row + col0) = u;
        return;
    }
#pragma unroll 1
    for (int col = col0; col < col0 + 8; ++col) {
        if (col >= 0 && col < cols) row[col] = static_cast<uint16_t>(u.x);
        u.x = __funnelshift_r(u.x, u.y, 16);
        u.y = __funnelshift_r(u.y, u.z, 16);
        u.z = __funnelshift_r(u.z, u.w, 16);
        u.w >>= 16;
    }
}

// Elements between the 16-byte boundary below row `r` of a matrix and its first element.
__device__ __forceinline__ int row_shift(const uint16_t* row) {
    return static_cast<int>(reinterpret_cast<uintptr_t>(row) >> 1) & 7;
}

// ---------------------------------------------------------------- dropout

struct DropoutParams {
    const uint16_t* x;
    const uint16_t* r;  // added, or null
    uint16_t* d;
    int64_t ldx, ldr, ldd;
    int m, n;
    int chunks;  // of a row, its shift counted in
    int wide;
    Drop drop;
};

constexpr int kDropoutThreads = 256;

__global__ void __launch_bounds__(kDropoutThreads) dropout_kernel(const DropoutParams p) {
    const Key key = drop_key(p.drop);
    const int64_t total = static_cast<int64_t>(p.m) * p.chunks;
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * kDropoutThreads + threadIdx.x; at < total;
         at += static_cast<int64_t>(gridDim.x) * kDropoutThreads) {
        const int row = static_cast<int>(at / p.chunks), j = static_cast<int>(at - static_cast<int64_t>(row) * p.chunks);
        const uint16_t* x = p.x + row * p.ldx;
        const int col0 = 8 * j - (p.wide ? row_shift(x) : 0);
        if (col0 >= p.n) continue;
        float v[8];
        unpack(load_chunk(x, col0, p.n, p.wide), v);
        drop_chunk(v, row, col0, p.drop, key);
        if (p.r) {
            float r[8];
            unpack(load_chunk(p.r + row * p.ldr, col0, p.n, p.wide), r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += r[i];
        }
        store_chunk(p.d + row * p.ldd, col0, p.n, p.wide, pack(v));
    }
}

// ---------------------------------------------------------------- sums over a row

// A row belongs to `threads` threads: one warp (eight rows a block), or the block.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) v += __shfl_xor_sync(0xffffffffu, v, i);
    return v;
}

// The sum over the row's threads, in the same order on every run.  `buf`: 32 floats that no
// other sum in flight uses.
__device__ __forceinline__ float row_sum(float v, float* buf) {
    v = warp_sum(v);
    if (blockDim.y > 1) return v;  // a row is one warp
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < warps ? buf[lane] : 0.f);
}

// The largest of the row's non-negative values as ordered bits (a NaN's are above an infinity's).
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* buf) {
    v = __reduce_max_sync(0xffffffffu, v);
    if (blockDim.y > 1) return v;
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, lane < warps ? buf[lane] : 0u);
}

// ---------------------------------------------------------------- norm, forward

struct NormParams {
    const uint16_t* x;
    const uint16_t* r;       // the residual, or null
    const uint16_t* weight;
    uint16_t* h;             // x (dropped) + r, or null
    uint16_t* y;             // bf16 output (kBf16)
    uint8_t* q;              // e4m3 output (kRowScale, kGroupScale)
    float* rstd;             // [m], or null
    float* scale;            // [m, lds]
    int64_t ldx, ldr, ldh, ldy, ldq, lds;
    int m, d;
    int wide;         // rows move in 16-byte words
    int wide_weight;  // the weight is 16-byte aligned
    float eps;
    Drop drop;
};

enum { kBf16 = 0, kRowScale = 1, kGroupScale = 2 };
constexpr int kScaleGroup = 128;
constexpr float kE4m3Max = 448.f;
// the smallest scale: one that is normal and whose reciprocal is finite, also for an all-zero row
constexpr float kMinScale = 1.17549435e-38f;

__device__ __forceinline__ float scale_of(uint32_t max_bits) {
    const float s = __uint_as_float(max_bits) / kE4m3Max;
    return s < kMinScale ? kMinScale : s;  // (a NaN stays one)
}

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
    uint16_t u;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(u) : "f"(hi), "f"(lo));
    return u;
}

__device__ __forceinline__ void store_e4m3(uint8_t* row, int col0, int cols, bool wide, const float (&v)[8]) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = e4m3x2(v[4 * i], v[4 * i + 1]) | static_cast<uint32_t>(e4m3x2(v[4 * i + 2], v[4 * i + 3])) << 16;
    if (wide && col0 >= 0 && col0 + 8 <= cols) {
        *reinterpret_cast<uint2*>(row + col0) = make_uint2(w[0], w[1]);
        return;
    }
#pragma unroll 1
    for (int col = col0; col < col0 + 8; ++col) {
        if (col >= 0 && col < cols) row[col] = static_cast<uint8_t>(w[0]);
        w[0] = __funnelshift_r(w[0], w[1], 8);
        w[1] >>= 8;
    }
}

// h = dropout(x) + r;  rstd = 1 / sqrt(mean(h^2) + eps);  y = h rstd weight, in fp32 from h
// before its rounding.  V chunks a thread.  Dynamic shared memory: kGroupScale's maxima.
template <int V, bool DROP, int OUT>
__global__ void __launch_bounds__(512, 1) norm_kernel(const NormParams p) {
    __shared__ float sums[32];
    __shared__ uint32_t maxima[32];
    extern __shared__ uint32_t group_max[];
    const int row = blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= p.m) return;  // (only whole warps of a block of several rows)
    const uint16_t* x = p.x + row * p.ldx;
    const int shift = p.wide ? row_shift(x) : 0;
    const int tid = threadIdx.x, threads = blockDim.x;
    Key key{};
    if (DROP) key = drop_key(p.drop);

    uint4 xu[V], ru[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int col0 = 8 * (tid + k * threads) - shift;
        xu[k] = load_chunk(x, col0, p.d, p.wide);
        if (p.r) ru[k] = load_chunk(p.r + row * p.ldr, col0, p.d, p.wide);
    }
    float v[V][8], sum = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int col0 = 8 * (tid + k * threads) - shift;
        unpack(xu[k], v[k]);
        if (DROP && col0 < p.d) drop_chunk(v[k], row, col0, p.drop, key);
        if (p.r) {
            float r[8];
            unpack(ru[k], r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] += r[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(v[k][i], v[k][i], sum);
        if (p.h && col0 < p.d) store_chunk(p.h + row * p.ldh, col0, p.d, p.wide, pack(v[k]));
    }
    const float rstd = 1.f / sqrtf(row_sum(sum, sums) / static_cast<float>(p.d) + p.eps);
    if (p.rstd && tid == 0) p.rstd[row] = rstd;

#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int col0 = 8 * (tid + k * threads) - shift;
        float w[8];
        unpack(load_chunk(p.weight, col0, p.d, shift == 0 && p.wide_weight), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] = v[k][i] * rstd * w[i];
        if (OUT == kBf16 && col0 < p.d) store_chunk(p.y + row * p.ldy, col0, p.d, p.wide, pack(v[k]));
    }
    if (OUT == kRowScale) {
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[k][i]) & 0x7fffffffu);
        const float scale = scale_of(row_max(top, maxima));
        if (tid == 0) p.scale[row * p.lds] = scale;
        const float inv = 1.f / scale;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int col0 = 8 * (tid + k * threads) - shift;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] *= inv;
            if (col0 < p.d) store_e4m3(p.q + row * p.ldq, col0, p.d, p.wide, v[k]);
        }
    }
    if (OUT == kGroupScale) {
        // A chunk lies in one group of columns, or in two where the row is shifted: each is
        // joined into the groups' maxima in shared memory (the order does not matter to a maximum).
        const int groups = (p.d + kScaleGroup - 1) / kScaleGroup;
        uint32_t* top = group_max + threadIdx.y * groups;
        for (int g = tid; g < groups; g += threads) top[g] = 0;
        if (blockDim.y > 1) __syncwarp();
        else __syncthreads();
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int col0 = 8 * (tid + k * threads) - shift;
            if (col0 >= p.d) continue;
            const int first = max(col0, 0) / kScaleGroup, cut = (first + 1) * kScaleGroup;
            uint32_t a = 0, b = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t u = __float_as_uint(v[k][i]) & 0x7fffffffu;
                if (col0 + i < cut) a = max(a, u);
                else b = max(b, u);
            }
            atomicMax(&top[first], a);
            if (col0 + 7 >= cut && cut < p.d) atomicMax(&top[first + 1], b);
        }
        if (blockDim.y > 1) __syncwarp();
        else __syncthreads();
        for (int g = tid; g < groups; g += threads) p.scale[row * p.lds + g] = scale_of(top[g]);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int col0 = 8 * (tid + k * threads) - shift;
            if (col0 >= p.d) continue;
            const int first = max(col0, 0) / kScaleGroup, cut = (first + 1) * kScaleGroup;
            const float ia = 1.f / scale_of(top[first]);
            const float ib = cut < p.d ? 1.f / scale_of(top[first + 1]) : 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] *= col0 + i < cut ? ia : ib;
            store_e4m3(p.q + row * p.ldq, col0, p.d, p.wide, v[k]);
        }
    }
}

// ---------------------------------------------------------------- norm, backward

struct NormBwdParams {
    const uint16_t* dy;
    const uint16_t* h;
    const uint16_t* weight;
    const float* rstd;
    const uint16_t* dh;   // the gradient that reaches h past the norm, or null
    uint16_t* dr;
    uint16_t* dx;         // dropout's: dr where kept, over 1 - p (or null)
    float* partial;       // [gridDim.x, d]: each block's part of the weight's gradient
    int64_t lddy, ldh, lddh, lddr, lddx;
    int m, d;
    int wide, wide_weight;
    int per_thread;       // chunks a thread, where they are not a constant of the kernel
    Drop drop;
};

// With xhat = h rstd and g = dy weight:  dr = rstd (g - xhat mean(g xhat)) + dh,
// dx = dropout's gradient of dr,  dweight = sum over rows of dy xhat.
// A block takes the rows row0, row0 + stride, ...: `stride` is a multiple of 8 rows, so a
// thread's rows all have the same shift and it owns the same columns in each; the weight's
// gradient stays in its registers until the end.
// V chunks a thread, in registers; V = 0: p.per_thread chunks, in places of the thread's own in
// shared memory (four chunks' rows and sums do not fit its registers).
template <int V, bool DROP>
__global__ void __launch_bounds__(512, 1) norm_bwd_kernel(const NormBwdParams p) {
    constexpr bool kShared = V == 0;
    constexpr int kHeld = kShared ? 1 : V;
    __shared__ float sums[2][32];
    extern __shared__ __align__(16) uint8_t smem[];
    const int row0 = blockIdx.x * blockDim.y + threadIdx.y, stride = gridDim.x * blockDim.y;
    const int shift = p.wide ? row_shift(p.dy + row0 * p.lddy) : 0;
    const int tid = threadIdx.x, threads = blockDim.x;
    const int held = kShared ? p.per_thread : V;
    Key key{};
    if (DROP) key = drop_key(p.drop);
    float dw[kHeld][8];
    uint4 dyu[kHeld], hu[kHeld], wu[kHeld];
    // kShared: chunk k of thread t has the words 4k .. 4k + 3, `threads` apart: dY, H and the sums
    uint4* own = reinterpret_cast<uint4*>(smem) + tid;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
        wu[k] = load_chunk(p.weight, 8 * (tid + k * threads) - shift, p.d, shift == 0 && p.wide_weight);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[k][i] = 0.f;
    }
    if (kShared)
        for (int k = 0; k < held; ++k) own[(4 * k + 2) * threads] = own[(4 * k + 3) * threads] = make_uint4(0, 0, 0, 0);

    int turn = 0;
    for (int64_t r = row0; r < p.m; r += stride, turn ^= 1) {
        const int row = static_cast<int>(r);
        const float rstd = p.rstd[row];
        float sum = 0.f;
        if (!kShared) {
#pragma unroll
            for (int k = 0; k < kHeld; ++k) {
                const int col0 = 8 * (tid + k * threads) - shift;
                dyu[k] = load_chunk(p.dy + row * p.lddy, col0, p.d, p.wide);
                hu[k] = load_chunk(p.h + row * p.ldh, col0, p.d, p.wide);
            }
        }
#pragma unroll kHeld
        for (int k = 0; k < held; ++k) {
            const int col0 = 8 * (tid + k * threads) - shift, at = kShared ? 0 : k;
            if (kShared) {
                own[4 * k * threads] = dyu[0] = load_chunk(p.dy + row * p.lddy, col0, p.d, p.wide);
                own[(4 * k + 1) * threads] = hu[0] = load_chunk(p.h + row * p.ldh, col0, p.d, p.wide);
                wu[0] = load_chunk(p.weight, col0, p.d, shift == 0 && p.wide_weight);
            }
            float t[8], h[8], w[8];
            unpack(dyu[at], t);
            unpack(hu[at], h);
            unpack(wu[at], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                t[i] *= h[i] * rstd;
                sum = fmaf(t[i], w[i], sum);
            }
            if (kShared) {
                float4* acc = reinterpret_cast<float4*>(own) + (4 * k + 2) * threads;
                const float4 a = acc[0], b = acc[threads];
                acc[0] = make_float4(a.x + t[0], a.y + t[1], a.z + t[2], a.w + t[3]);
                acc[threads] = make_float4(b.x + t[4], b.y + t[5], b.z + t[6], b.w + t[7]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) dw[at][i] += t[i];
            }
        }
        const float mean = row_sum(sum, sums[turn]) / static_cast<float>(p.d);
#pragma unroll kHeld
        for (int k = 0; k < held; ++k) {
            const int col0 = 8 * (tid + k * threads) - shift, at = kShared ? 0 : k;
            if (col0 >= p.d) continue;
            // (one chunk after the other: the generators of several do not fit the registers)
            if (V > 1) asm volatile("" : "+r"(key.k0) : : "memory");
            if (kShared) {
                dyu[0] = own[4 * k * threads];
                hu[0] = own[(4 * k + 1) * threads];
                wu[0] = load_chunk(p.weight, col0, p.d, shift == 0 && p.wide_weight);
            }
            float v[8], h[8], w[8];
            unpack(dyu[at], v);
            unpack(hu[at], h);
            unpack(wu[at], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = rstd * (v[i] * w[i] - h[i] * rstd * mean);
            if (p.dh) {
                unpack(load_chunk(p.dh + row * p.lddh, col0, p.d, p.wide), h);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] += h[i];
            }
            store_chunk(p.dr + row * p.lddr, col0, p.d, p.wide, pack(v));
            if (DROP) {
                drop_chunk(v, row, col0, p.drop, key);
                store_chunk(p.dx + row * p.lddx, col0, p.d, p.wide, pack(v));
            }
        }
    }

    float* part = p.partial + static_cast<int64_t>(blockIdx.x) * p.d;
    if (kShared) {
        for (int k = 0; k < held; ++k)
            for (int i = 0; i < 8; ++i) {
                const int col = 8 * (tid + k * threads) - shift + i;
                const float* acc = reinterpret_cast<const float*>(own + (4 * k + 2 + i / 4) * threads);
                if (col >= 0 && col < p.d) part[col] = acc[i & 3];
            }
        return;
    }
    if (blockDim.y == 1) {
#pragma unroll
        for (int k = 0; k < kHeld; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int col = 8 * (tid + k * threads) - shift + i;
                if (col >= 0 && col < p.d) part[col] = dw[k][i];
            }
        return;
    }
    // several rows a block: the warps add theirs one after the other
    float* total = reinterpret_cast<float*>(smem);
    for (int c = threadIdx.y * 32 + tid; c < p.d; c += 32 * blockDim.y) total[c] = 0.f;
    for (int w = 0; w < static_cast<int>(blockDim.y); ++w) {
        __syncthreads();
        if (w != static_cast<int>(threadIdx.y)) continue;
#pragma unroll
        for (int k = 0; k < kHeld; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int col = 8 * (tid + k * threads) - shift + i;
                if (col >= 0 && col < p.d) total[col] += dw[k][i];
            }
    }
    __syncthreads();
    for (int c = threadIdx.y * 32 + tid; c < p.d; c += 32 * blockDim.y) part[c] = total[c];
}

// dweight[c] = the sum of the blocks' parts, in the same order on every run.
constexpr int kJoinColumns = 32, kJoinParts = 16;
__global__ void __launch_bounds__(kJoinColumns * kJoinParts) join_kernel(const float* partial, int parts, int d,
                                                                         float* dweight) {
    __shared__ float sum[kJoinParts][kJoinColumns];
    const int c = blockIdx.x * kJoinColumns + threadIdx.x;
    float v = 0.f;
    if (c < d)
        for (int i = threadIdx.y; i < parts; i += kJoinParts) v += partial[static_cast<int64_t>(i) * d + c];
    sum[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y != 0 || c >= d) return;
    for (int i = 1; i < kJoinParts; ++i) v += sum[i][threadIdx.x];
    dweight[c] = v;
}

}  // namespace rowwise
}  // namespace gb
