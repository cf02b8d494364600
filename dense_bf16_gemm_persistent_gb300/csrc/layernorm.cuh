// Device code of the layer norm (mean and variance) with the residual's addition, and of its backward
// pass.  Rows are cut into chunks, fetched ahead of their turn and given to threads as rowwise.cuh's
// norm does; both passes are bound by memory (8 bytes an element).
#pragma once

#include "rowwise.cuh"

namespace gb {
namespace rowwise {

// The sums of two values over the row's threads, in the same order on every run; `half`: half of the power of two
// that the row's warps fit in.  `buf`: 32 pairs that no other sum in flight uses.
__device__ __forceinline__ float2 row_sum2(float a, float b, int half, float2* buf) {
    a = warp_sum(a);
    b = warp_sum(b);
    if (blockDim.y > 1) return make_float2(a, b);  // a row is one warp
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31, at = lane & (2 * half - 1);
    if (lane == 0) buf[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    float2 t = at < warps ? buf[at] : make_float2(0.f, 0.f);
    for (int i = half; i > 0; i >>= 1) {
        t.x += __shfl_xor_sync(0xffffffffu, t.x, i);
        t.y += __shfl_xor_sync(0xffffffffu, t.y, i);
    }
    return t;
}

// Half of the least power of two (2 or more) that `warps` fit in.
__device__ __forceinline__ int half_of(int warps) { return warps <= 2 ? 1 : 1 << (31 - __clz(warps - 1)); }

// sum / n, by way of `inverse` = 1 / n, and once more for what that leaves: where n values are equal, that value.
__device__ __forceinline__ float mean_of(float sum, float n, float inverse) {
    const float mean = sum * inverse, rest = fmaf(-mean, n, sum);
    return fabsf(sum) <= 3.4028235e38f ? fmaf(rest, inverse, mean) : mean;  // (an infinite sum leaves nothing)
}

// Elements of the chunk at `col0` that lie in the row.
__device__ __forceinline__ int inside(int col0, int cols) { return max(0, min(col0 + 8, cols) - max(col0, 0)); }

// Eight elements of a vector at `col0` (zeros outside it), which lies aligned: the two 16-byte words that hold them.
__device__ __forceinline__ uint4 load_vector(const uint16_t* vec, int col0, int cols, bool aligned) {
    const int first = col0 & ~7, by = col0 & 7;
    if (!aligned || col0 < 0 || first + 16 > cols || by == 0) return load_chunk(vec, col0, cols, aligned && by == 0);
    const uint4 a = *reinterpret_cast<const uint4*>(vec + first), b = *reinterpret_cast<const uint4*>(vec + first + 8);
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (by & 4) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (by & 2) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    if (by & 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A chunk that a row ends in (`wide`: it begins on 16 bytes), in pieces of 8, 4 and 2 bytes: the warps that hold a
// row's ends are waited for by all others, and element after element took twice as long.
__device__ __forceinline__ void store_end(uint16_t* row, int col0, int cols, bool wide, const uint4& u) {
    if (!wide || (col0 < 0 && col0 + 8 > cols)) {
        store_chunk(row, col0, cols, false, u);
        return;
    }
    uint16_t* to = row + col0;
    if (col0 < 0) {  // elements s .. 7
        const int s = -col0, even = s + (s & 1);
        if (s & 1) to[s] = static_cast<uint16_t>((s == 1 ? u.x : s == 3 ? u.y : s == 5 ? u.z : u.w) >> 16);
        if (even & 2) *reinterpret_cast<uint32_t*>(to + even) = even == 2 ? u.y : u.w;
        if (even <= 4) *reinterpret_cast<uint2*>(to + 4) = make_uint2(u.z, u.w);
    } else {  // elements 0 .. n - 1
        const int n = cols - col0;
        if (n & 4) *reinterpret_cast<uint2*>(to) = make_uint2(u.x, u.y);
        if (n & 2) *reinterpret_cast<uint32_t*>(to + (n & 4)) = n & 4 ? u.z : u.x;
        if (n & 1) to[n & 6] = static_cast<uint16_t>((n & 6) == 0 ? u.x : (n & 6) == 2 ? u.y : (n & 6) == 4 ? u.z : u.w);
    }
}

// ---------------------------------------------------------------- forward

struct LayerNormParams {
    const uint16_t* x;
    const uint16_t* r;       // the residual, or null
    const uint16_t* weight;
    const uint16_t* bias;    // or null
    uint16_t* h;             // x (dropped) + r, or null
    uint16_t* y;
    float* mean;             // [m], or null
    float* rstd;             // [m], or null
    int64_t ldx, ldr, ldh, ldy;
    int m, d;
    int wide;                     // rows move in 16-byte words
    int wide_weight, wide_bias;   // 16-byte aligned
    float eps;
    Drop drop;
};

// h = dropout(x) + r;  mean, rstd = 1 / sqrt(mean((h - mean)^2) + eps);  y = (h - mean) rstd weight + bias,
// in fp32 from h before its rounding.
//
// The variance is a sum of squares of differences, never a difference of sums (which loses what the mean is larger than
// the deviation by): each warp takes its own part's mean first, from registers, and the parts' sums of squares are moved
// to the row's mean when they are joined,
//     sum (h - mean)^2 = sum over warps [ S_w + n_w (mean_w - mean)^2 ],
// so that a row has one barrier, as the root-mean-square norm's has. Means are quotients to the last bit or nearly (mean_of),
// so that a row of one value has that as its mean, and no variance: as a product by 1 / d, of 777 columns and -30000, rstd
// was 306 and not 316.
//
// FULL: rows of whole, aligned 16-byte words (no chunk begins or ends inside one); other rows' chunks are the same but
// for those that a row begins and ends in.
//
// 8192 x 4096 with a residual and a bias on a GB300: 45 us, 5.9 TB/s (0.88 of the copy bandwidth), 43 us by ncu; with
// dropout 63. Rows that begin anywhere, 3001 x 4099: 32 us (0.46), with dropout 54. What a chunk costs decides: with every chunk's ends looked at it took 610 instructions a warp's part
// of a row, 62 % of issue slots and 55 us.
//
// Dynamic shared memory: the rows [stage][x or r][chunk][thread], the weight, the bias.  (Three stages of 16384 columns
// and both vectors would be 256 KB.)
__host__ __device__ constexpr int layer_norm_stages(int v) { return v == 4 ? 2 : kRowStages; }

// 16 bytes to the thread's own place, which it alone reads.
__device__ __forceinline__ void fetch_16(uint4* to, const uint16_t* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))),
                 "l"(from)
                 : "memory");
}

template <int V, int DROP, bool FULL>
__global__ void __maxnreg__(V == 4 ? 128 : 80) layer_norm_kernel(const __grid_constant__ LayerNormParams p) {
    allow_next_kernel();
    wait_for_earlier_kernels();
    constexpr int kStages = layer_norm_stages(V);
    constexpr bool kHeld = FULL && V == 2;  // the weight and the bias in registers
    __shared__ float2 parts[2][32];
    __shared__ float2 counts[32];  // and one over them
    extern __shared__ __align__(16) uint8_t smem[];
    const int row0 = blockIdx.x * blockDim.y + threadIdx.y, stride = gridDim.x * blockDim.y;
    const int shift = !FULL && p.wide ? row_shift(p.x + row0 * p.ldx) : 0;
    const int tid = threadIdx.x, threads = blockDim.x, all = blockDim.x * blockDim.y, lane = tid & 31;
    const int warps = threads >> 5, half = half_of(warps);
    uint4* slots = reinterpret_cast<uint4*>(smem) + threadIdx.y * threads + tid;
    const Draw<DROP> draw(p.drop);
    // a chunk that lies in the row whole (a thread's chunks do so in all its rows, or in none)
    auto whole = [&](int col0) { return FULL ? col0 < p.d : p.wide && col0 >= 0 && col0 + 8 <= p.d; };
    const uint16_t *x_next = p.x + row0 * p.ldx, *r_next = p.r + row0 * p.ldr;  // (of the row that is fetched next)
    auto fetch = [&](int64_t row, int stage) {
        if (row < p.m) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int col0 = 8 * (tid + k * threads) - shift;
                uint4* to = slots + stage * 2 * V * all + k * all;
                if (whole(col0)) {
                    fetch_16(to, x_next + col0);
                    if (p.r) fetch_16(to + V * all, r_next + col0);
                } else if (!FULL && col0 < p.d) {
                    fetch_chunk(to, x_next, col0, p.d, p.wide, row > 0 && p.ldx >= 8);
                    if (p.r) fetch_chunk(to + V * all, r_next, col0, p.d, p.wide, row > 0 && p.ldr >= 8);
                }
            }
            x_next += stride * p.ldx;
            r_next += stride * p.ldr;
        }
        fetch_commit();
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(row0 + static_cast<int64_t>(s) * stride, s);
    uint4* weight = slots + kStages * 2 * V * all;  // (the thread's own part of it, and of the bias)
    uint4* bias = weight + V * all;
    float held[2][kHeld ? V : 1][8];
    float count = 0.f;  // of the warp's elements in a row: the same in every row
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int col0 = 8 * (tid + k * threads) - shift;
        const uint4 w = load_vector(p.weight, col0, p.d, p.wide_weight);
        const uint4 b = p.bias ? load_vector(p.bias, col0, p.d, p.wide_bias) : make_uint4(0, 0, 0, 0);
        if constexpr (kHeld) {
            unpack(w, held[0][k]);
            unpack(b, held[1][k]);
        } else {
            weight[k * all] = w;
            bias[k * all] = b;
        }
        count += static_cast<float>(inside(col0, p.d));
    }
    count = warp_sum(count);
    const float of_row = 1.f / static_cast<float>(p.d), of_warp = count > 0.f ? 1.f / count : 0.f;
    if (blockDim.y == 1 && lane == 0) counts[tid >> 5] = make_float2(count, of_warp);  // (read after a row's barrier)

    int stage = 0, turn = 0;
    uint16_t *h_row = p.h + row0 * p.ldh, *y_row = p.y + row0 * p.ldy;
    for (int64_t r = row0; r < p.m; r += stride, turn ^= 1, h_row += stride * p.ldh, y_row += stride * p.ldy) {
        const int row = static_cast<int>(r);
        fetch(r + static_cast<int64_t>(kStages - 1) * stride, stage == 0 ? kStages - 1 : stage - 1);
        fetch_wait<kStages - 1>();
        float v[V][8], sum = 0.f;
        const uint4* at = slots + stage * 2 * V * all;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int col0 = 8 * (tid + k * threads) - shift;
            if (col0 >= p.d) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[k][i] = 0.f;
                continue;
            }
            unpack(FULL || col0 >= 0 ? at[k * all] : read_chunk(at + k * all, col0), v[k]);
            if (DROP) draw.chunk(v[k], row, col0);
            if (p.r) {
                float r[8];
                unpack(FULL || col0 >= 0 ? at[(V + k) * all] : read_chunk(at + (V + k) * all, col0), r);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[k][i] += r[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += v[k][i];  // (outside the row: zeros)
            if (p.h) {
                if (whole(col0)) *reinterpret_cast<uint4*>(h_row + col0) = pack(v[k]);
                else store_end(h_row, col0, p.d, p.wide, pack(v[k]));
            }
        }
        stage = stage == kStages - 1 ? 0 : stage + 1;
        sum = warp_sum(sum);
        float mean = mean_of(sum, count, of_warp), squares = 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int col0 = 8 * (tid + k * threads) - shift;
            if (FULL ? col0 < p.d : col0 >= 0 && col0 + 8 <= p.d) {  // (also where rows are not wide)
#pragma unroll
                for (int i = 0; i < 8; ++i) squares = fmaf(v[k][i] - mean, v[k][i] - mean, squares);
            } else if (!FULL) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (col0 + i >= 0 && col0 + i < p.d) squares = fmaf(v[k][i] - mean, v[k][i] - mean, squares);
            }
        }
        squares = warp_sum(squares);
        if (blockDim.y == 1) {
            float2* part = parts[turn];
            if (lane == 0) part[tid >> 5] = make_float2(sum, squares);
            __syncthreads();
            const int place = lane & (2 * half - 1);
            const bool on = place < warps;
            const float2 t = on ? part[place] : make_float2(0.f, 0.f);
            const float2 n = on ? counts[place] : make_float2(0.f, 0.f);
            mean = t.x;
            for (int i = half; i > 0; i >>= 1) mean += __shfl_xor_sync(0xffffffffu, mean, i);
            mean = mean_of(mean, static_cast<float>(p.d), of_row);
            const float off = fmaf(-n.x, mean, t.x) * n.y;  // of the warp's mean from the row's
            squares = fmaf(n.x * off, off, t.y);
            for (int i = half; i > 0; i >>= 1) squares += __shfl_xor_sync(0xffffffffu, squares, i);
        }
        const float rstd = 1.f / sqrtf(squares * of_row + p.eps);
        if (tid == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int col0 = 8 * (tid + k * threads) - shift;
            if (col0 >= p.d) continue;
            if constexpr (kHeld) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[k][i] = fmaf((v[k][i] - mean) * rstd, held[0][k][i], held[1][k][i]);
            } else {
                float w[8], b[8];
                unpack(weight[k * all], w);
                unpack(bias[k * all], b);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[k][i] = fmaf((v[k][i] - mean) * rstd, w[i], b[i]);
            }
            if (whole(col0)) *reinterpret_cast<uint4*>(y_row + col0) = pack(v[k]);
            else store_end(y_row, col0, p.d, p.wide, pack(v[k]));
        }
    }
}

// ---------------------------------------------------------------- backward

struct LayerNormBwdParams {
    const uint16_t* dy;
    const uint16_t* h;
    const uint16_t* weight;
    const float* mean;
    const float* rstd;
    const uint16_t* dh;   // the gradient that reaches h past the norm, or null
    uint16_t* dr;
    uint16_t* dx;         // dropout's: dr where kept, over 1 - p (or null)
    float* partial;       // [gridDim.x][2][pitch]: each block's part of the weight's and the bias's gradient
    int64_t lddy, ldh, lddh, lddr, lddx;
    int m, d;
    int wide, wide_weight;
    int pitch;            // columns of a row's chunks, its shift counted in
    Drop drop;
};

// With xhat = (h - mean) rstd and g = dy weight:  dr = rstd (g - mean(g) - xhat mean(g xhat)) + dh,
// dx = dropout's gradient of dr,  dweight = sum over rows of dy xhat,  dbias = sum over rows of dy.
// Rows and the gradients' sums in registers as in norm_bwd_kernel. FULL as in layer_norm_kernel: g and xhat stay in
// registers from the first pass over a row to the second; with chunks that end inside a row xhat does, for two blocks of
// nine warps an SM.
//
// 8192 x 4096 with dH on a GB300, the join with it: 51 us, 5.3 TB/s (0.78 of the copy bandwidth), with dropout 72; 3001 x
// 4099 32 us (0.45), with dropout 50. With g and xhat made again from shared memory, and every chunk's ends looked at, 8192 x 4096 took 700
// instructions a warp's part of a row and 69 us, 3001 x 4099 40.
//
// Dynamic shared memory: the rows [stage][dY, H or dH][chunk][thread], then the weight.
__host__ __device__ constexpr int layer_bwd_stages(int v) { return v == 2 ? 3 : kBwdStages; }

template <int V, int DROP, bool FULL>
__global__ void __maxnreg__(V == 4 || FULL ? 128 : 96) layer_norm_bwd_kernel(const __grid_constant__ LayerNormBwdParams p) {
    allow_next_kernel();
    wait_for_earlier_kernels();
    constexpr int kStages = layer_bwd_stages(V);
    constexpr bool kXhat = V == 2 && (FULL || DROP == kNoDrop), kHeld = FULL && V == 2;  // xhat; g and the weight in registers
    __shared__ float2 sums[2][32];
    extern __shared__ __align__(16) uint8_t smem[];
    const int row0 = blockIdx.x * blockDim.y + threadIdx.y, stride = gridDim.x * blockDim.y;
    const int shift = !FULL && p.wide ? row_shift(p.dy + row0 * p.lddy) : 0;
    const int tid = threadIdx.x, threads = blockDim.x, all = blockDim.x * blockDim.y, half = half_of(threads >> 5);
    uint4* slots = reinterpret_cast<uint4*>(smem) + threadIdx.y * threads + tid;
    uint4* weight = slots + kStages * 3 * V * all;  // (the thread's own part of it)
    const Draw<DROP> draw(p.drop);
    // a chunk that lies in the row whole (a thread's chunks do so in all its rows, or in none)
    auto whole = [&](int col0) { return FULL ? col0 < p.d : p.wide && col0 >= 0 && col0 + 8 <= p.d; };
    auto slot = [&](int stage, int matrix, int k) { return slots + ((stage * 3 + matrix) * V + k) * all; };
    auto chunk = [&](int stage, int matrix, int k, int col0) {
        return FULL || col0 >= 0 ? *slot(stage, matrix, k) : read_chunk(slot(stage, matrix, k), col0);
    };
    const uint16_t *dy_next = p.dy + row0 * p.lddy, *h_next = p.h + row0 * p.ldh, *dh_next = p.dh + row0 * p.lddh;
    auto fetch = [&](int64_t row, int stage) {
        if (row < p.m) {
            if (V == 4) {  // (fewer registers than addresses that move along)
                dy_next = p.dy + row * p.lddy;
                h_next = p.h + row * p.ldh;
                dh_next = p.dh + row * p.lddh;
            }
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int col0 = 8 * (tid + k * threads) - shift;
                if (whole(col0)) {
                    fetch_16(slot(stage, 0, k), dy_next + col0);
                    fetch_16(slot(stage, 1, k), h_next + col0);
                    if (p.dh) fetch_16(slot(stage, 2, k), dh_next + col0);
                } else if (!FULL && col0 < p.d) {
                    fetch_chunk(slot(stage, 0, k), dy_next, col0, p.d, p.wide, row > 0 && p.lddy >= 8);
                    fetch_chunk(slot(stage, 1, k), h_next, col0, p.d, p.wide, row > 0 && p.ldh >= 8);
                    if (p.dh) fetch_chunk(slot(stage, 2, k), dh_next, col0, p.d, p.wide, row > 0 && p.lddh >= 8);
                }
            }
            if (V == 2) {
                dy_next += stride * p.lddy;
                h_next += stride * p.ldh;
                dh_next += stride * p.lddh;
            }
        }
        fetch_commit();
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(row0 + static_cast<int64_t>(s) * stride, s);
    float dw[V][8], db[V][8], held[kHeld ? V : 1][8];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const uint4 w = load_vector(p.weight, 8 * (tid + k * threads) - shift, p.d, p.wide_weight);
        if constexpr (kHeld) unpack(w, held[k]);
        else weight[k * all] = w;
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[k][i] = db[k][i] = 0.f;
    }
    const float of_row = 1.f / static_cast<float>(p.d);

    int stage = 0, turn = 0;  // (of row_sum2's places)
    for (int64_t r = row0; r < p.m; r += stride, turn ^= 1) {
        const int row = static_cast<int>(r);
        const float rstd = p.rstd[row], mean = p.mean[row];
        fetch(r + static_cast<int64_t>(kStages - 1) * stride, stage == 0 ? kStages - 1 : stage - 1);
        fetch_wait<kStages - 1>();
        float sum = 0.f, dot = 0.f;  // of g and of g xhat
        float g[kHeld ? V : 1][8], xhat[kXhat ? V : 1][8];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int col0 = 8 * (tid + k * threads) - shift;
            if (col0 >= p.d) continue;
            float t[8], h[8], w[8];
            unpack(chunk(stage, 0, k, col0), t);  // (outside the row dY is zero, and adds nothing)
            unpack(chunk(stage, 1, k, col0), h);
            if constexpr (kHeld) {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = held[k][i];
            } else {
                unpack(weight[k * all], w);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float gi = t[i] * w[i], xi = (h[i] - mean) * rstd;
                db[k][i] += t[i];
                sum += gi;
                dot = fmaf(gi, xi, dot);
                dw[k][i] = fmaf(t[i], xi, dw[k][i]);
                if constexpr (kHeld) g[k][i] = gi;
                if constexpr (kXhat) xhat[k][i] = xi;
            }
        }
        const float2 total = row_sum2(sum, dot, half, sums[turn]);
        const float mean_g = total.x * of_row, mean_gx = total.y * of_row;
        uint16_t *dr_row = p.dr + r * p.lddr, *dx_row = p.dx + r * p.lddx;
#pragma unroll(V == 4 ? 1 : V)  // (of four chunks, one at a time, for the registers)
        for (int k = 0; k < V; ++k) {
            const int col0 = 8 * (tid + k * threads) - shift;
            if (col0 >= p.d) continue;
            float v[8], h[8], w[8];
            if constexpr (kHeld) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = g[k][i] - fmaf(xhat[k][i], mean_gx, mean_g);
            } else {
                unpack(chunk(stage, 0, k, col0), v);
                unpack(weight[k * all], w);
                if constexpr (kXhat) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) h[i] = xhat[k][i];
                } else {
                    unpack(chunk(stage, 1, k, col0), h);
#pragma unroll
                    for (int i = 0; i < 8; ++i) h[i] = (h[i] - mean) * rstd;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = v[i] * w[i] - fmaf(h[i], mean_gx, mean_g);
            }
            if (p.dh) {
                unpack(chunk(stage, 2, k, col0), h);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = fmaf(rstd, v[i], h[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= rstd;
            }
            if (whole(col0)) *reinterpret_cast<uint4*>(dr_row + col0) = pack(v);
            else store_end(dr_row, col0, p.d, p.wide, pack(v));
            if (DROP) {
                draw.chunk(v, row, col0);
                if (whole(col0)) *reinterpret_cast<uint4*>(dx_row + col0) = pack(v);
                else store_end(dx_row, col0, p.d, p.wide, pack(v));
            }
        }
        stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    fetch_wait<0>();

    float* part = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * p.pitch;
    if (blockDim.y == 1) {
        // as the chunks lie: the join moves them by the block's shift.  (What is outside the row is not read.)
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int at = 8 * (tid + k * threads);
            if (at >= p.pitch) continue;
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                *reinterpret_cast<float4*>(part + at + i) = make_float4(dw[k][i], dw[k][i + 1], dw[k][i + 2], dw[k][i + 3]);
                *reinterpret_cast<float4*>(part + p.pitch + at + i) =
                    make_float4(db[k][i], db[k][i + 1], db[k][i + 2], db[k][i + 3]);
            }
        }
        return;
    }
    // several rows a block: the warps add theirs one after the other, where the rows were
    __syncthreads();
    float* total = reinterpret_cast<float*>(smem);
    for (int c = threadIdx.y * 32 + tid; c < 2 * p.d; c += 32 * blockDim.y) total[c] = 0.f;
    for (int w = 0; w < static_cast<int>(blockDim.y); ++w) {
        __syncthreads();
        if (w != static_cast<int>(threadIdx.y)) continue;
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int col = 8 * (tid + k * threads) - shift + i;
                if (col >= 0 && col < p.d) {
                    total[col] += dw[k][i];
                    total[p.d + col] += db[k][i];
                }
            }
    }
    __syncthreads();
    for (int c = threadIdx.y * 32 + tid; c < p.d; c += 32 * blockDim.y) {
        part[c] = total[c];
        part[p.pitch + c] = total[p.d + c];
    }
}

// The sums of the blocks' parts of both gradients, as join_kernel's.  Column c of block b's part is at c + shift, where
// shift is row b's in the matrices: (first + b step) mod 8.
__global__ void __launch_bounds__(kJoinColumns * kJoinParts) join2_kernel(const float* partial, int parts, int d, int pitch,
                                                                          int first, int step, float* dweight, float* dbias) {
    allow_next_kernel();
    wait_for_earlier_kernels();
    __shared__ float sum[kJoinParts][kJoinColumns + 1];
    const int c = blockIdx.x * kJoinColumns + threadIdx.x;
    float v = 0.f;
    if (c < 2 * d) {
        const float* from = partial + (c < d ? c : c - d + pitch);
#pragma unroll 8
        for (int i = threadIdx.y; i < parts; i += kJoinParts) v += from[static_cast<int64_t>(i) * 2 * pitch + ((first + i * step) & 7)];
    }
    sum[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    // a warp to a column
    const int column = blockIdx.x * kJoinColumns + threadIdx.y;
    v = warp_sum(sum[threadIdx.x][threadIdx.y]);
    if (threadIdx.x == 0 && column < 2 * d) (column < d ? dweight + column : dbias + (column - d))[0] = v;
}

}  // namespace rowwise
}  // namespace gb
