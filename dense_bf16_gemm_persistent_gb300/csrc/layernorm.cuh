// Device code of the layer norm (mean and variance) with the residual's addition, and of its backward
// pass.  Rows are cut into chunks, fetched ahead of their turn and given to threads as rowwise.cuh's
// norm does; both passes are bound by memory (8 bytes an element).
#pragma once

#include "rowwise.cuh"

namespace gb {
namespace rowwise {

// The two sums over the row's threads, as row_sum().  `buf`: 32 pairs that no other sum in flight uses.
__device__ __forceinline__ float2 row_sum2(float a, float b, float2* buf) {
    a = warp_sum(a);
    b = warp_sum(b);
    if (blockDim.y > 1) return make_float2(a, b);  // a row is one warp
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) buf[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    const float2 t = lane < warps ? buf[lane] : make_float2(0.f, 0.f);
    return make_float2(warp_sum(t.x), warp_sum(t.y));
}

// Elements of the chunk at `col0` that lie in the row.
__device__ __forceinline__ int inside(int col0, int cols) { return max(0, min(col0 + 8, cols) - max(col0, 0)); }

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
// The variance is a sum of squares of differences, never a difference of sums (which loses what the mean is
// larger than the deviation by): each warp takes its own part's mean first, from registers, and the parts'
// sums of squares are moved to the row's mean when they are joined,
//     sum (h - mean)^2 = sum over warps [ S_w + n_w (mean_w - mean)^2 ],
// so that a row has one barrier, as the root-mean-square norm's has.
// Dynamic shared memory: the rows [stage][x or r][chunk][thread], the weight, the bias.  (Three stages of
// 16384 columns and both vectors would be 256 KB.)
__host__ __device__ constexpr int layer_norm_stages(int v) { return v == 4 ? 2 : kRowStages; }

template <int V, int DROP>
__global__ void __maxnreg__(V == 4 ? 128 : DROP ? 80 : 64) layer_norm_kernel(const __grid_constant__ LayerNormParams p) {
    allow_next_kernel();
    wait_for_earlier_kernels();
    constexpr int kStages = layer_norm_stages(V);
    __shared__ float2 parts[2][32];
    __shared__ float counts[32];
    extern __shared__ __align__(16) uint8_t smem[];
    const int row0 = blockIdx.x * blockDim.y + threadIdx.y, stride = gridDim.x * blockDim.y;
    const int shift = p.wide ? row_shift(p.x + row0 * p.ldx) : 0;
    const int tid = threadIdx.x, threads = blockDim.x, all = blockDim.x * blockDim.y, lane = tid & 31;
    uint4* slots = reinterpret_cast<uint4*>(smem) + threadIdx.y * threads + tid;
    const Draw<DROP> draw(p.drop);
    auto fetch = [&](int64_t row, int stage) {
        if (row < p.m) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int col0 = 8 * (tid + k * threads) - shift;
                fetch_chunk(slots + (stage * 2 * V + k) * all, p.x + row * p.ldx, col0, p.d, p.wide, row > 0 && p.ldx >= 8);
                if (p.r)
                    fetch_chunk(slots + ((stage * 2 + 1) * V + k) * all, p.r + row * p.ldr, col0, p.d, p.wide,
                                row > 0 && p.ldr >= 8);
            }
        }
        fetch_commit();
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(row0 + static_cast<int64_t>(s) * stride, s);
    uint4* weight = slots + kStages * 2 * V * all;  // (the thread's own part of it, and of the bias)
    uint4* bias = weight + V * all;
    float count = 0.f;  // of the warp's elements in a row: the same in every row
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int col0 = 8 * (tid + k * threads) - shift;
        weight[k * all] = load_chunk(p.weight, col0, p.d, shift == 0 && p.wide_weight);
        if (p.bias) bias[k * all] = load_chunk(p.bias, col0, p.d, shift == 0 && p.wide_bias);
        count += static_cast<float>(inside(col0, p.d));
    }
    count = warp_sum(count);
    if (blockDim.y == 1 && lane == 0) counts[tid >> 5] = count;  // (read after a row's barrier)
    const float of_row = 1.f / static_cast<float>(p.d), of_warp = count > 0.f ? 1.f / count : 0.f;

    int stage = 0, turn = 0;
    for (int64_t r = row0; r < p.m; r += stride, turn ^= 1) {
        const int row = static_cast<int>(r);
        fetch(r + static_cast<int64_t>(kStages - 1) * stride, stage == 0 ? kStages - 1 : stage - 1);
        fetch_wait<kStages - 1>();
        float v[V][8], sum = 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int col0 = 8 * (tid + k * threads) - shift;
            unpack(read_chunk(slots + (stage * 2 * V + k) * all, col0), v[k]);
            if (DROP) draw.chunk(v[k], row, col0);
            if (p.r) {
                float r[8];
                unpack(read_chunk(slots + ((stage * 2 + 1) * V + k) * all, col0), r);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[k][i] += r[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += v[k][i];  // (outside the row: zeros)
            if (p.h && col0 < p.d) store_chunk(p.h + row * p.ldh, col0, p.d, p.wide, pack(v[k]));
        }
        stage = stage == kStages - 1 ? 0 : stage + 1;
        sum = warp_sum(sum);
        float mean = sum * of_warp, squares = 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int col0 = 8 * (tid + k * threads) - shift;
            if (col0 >= 0 && col0 + 8 <= p.d) {
#pragma unroll
                for (int i = 0; i < 8; ++i) squares = fmaf(v[k][i] - mean, v[k][i] - mean, squares);
            } else {
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
            const bool on = lane < threads >> 5;
            const float2 t = on ? part[lane] : make_float2(0.f, 0.f);
            const float n = on ? counts[lane] : 0.f;
            mean = warp_sum(t.x) * of_row;
            const float off = n > 0.f ? t.x / n - mean : 0.f;
            squares = warp_sum(fmaf(n * off, off, t.y));
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
            float w[8];
            unpack(weight[k * all], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] = (v[k][i] - mean) * rstd * w[i];
            if (p.bias) {
                unpack(bias[k * all], w);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[k][i] += w[i];
            }
            store_chunk(p.y + row * p.ldy, col0, p.d, p.wide, pack(v[k]));
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
    float* partial;       // [gridDim.x][2][d]: each block's part of the weight's and the bias's gradient
    int64_t lddy, ldh, lddh, lddr, lddx;
    int m, d;
    int wide, wide_weight;
    Drop drop;
};

// With xhat = (h - mean) rstd and g = dy weight:  dr = rstd (g - mean(g) - xhat mean(g xhat)) + dh,
// dx = dropout's gradient of dr,  dweight = sum over rows of dy xhat,  dbias = sum over rows of dy.
// Rows, stages and the gradients' sums in registers as in norm_bwd_kernel.
// Dynamic shared memory: the rows [stage][dY, H or dH][chunk][thread], then the weight.
template <int V, int DROP>
__global__ void __maxnreg__(V == 4 ? 128 : 80) layer_norm_bwd_kernel(const __grid_constant__ LayerNormBwdParams p) {
    allow_next_kernel();
    wait_for_earlier_kernels();
    __shared__ float2 sums[2][32];
    extern __shared__ __align__(16) uint8_t smem[];
    const int row0 = blockIdx.x * blockDim.y + threadIdx.y, stride = gridDim.x * blockDim.y;
    const int shift = p.wide ? row_shift(p.dy + row0 * p.lddy) : 0;
    const int tid = threadIdx.x, threads = blockDim.x, all = blockDim.x * blockDim.y;
    uint4* slots = reinterpret_cast<uint4*>(smem) + threadIdx.y * threads + tid;
    uint4* weight = slots + kBwdStages * 3 * V * all;  // (the thread's own part of it)
    const Draw<DROP> draw(p.drop);
    auto slot = [&](int stage, int matrix, int k) { return slots + ((stage * 3 + matrix) * V + k) * all; };
    auto fetch = [&](int64_t row, int stage) {
        if (row < p.m) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int col0 = 8 * (tid + k * threads) - shift;
                fetch_chunk(slot(stage, 0, k), p.dy + row * p.lddy, col0, p.d, p.wide, row > 0 && p.lddy >= 8);
                fetch_chunk(slot(stage, 1, k), p.h + row * p.ldh, col0, p.d, p.wide, row > 0 && p.ldh >= 8);
                if (p.dh) fetch_chunk(slot(stage, 2, k), p.dh + row * p.lddh, col0, p.d, p.wide, row > 0 && p.lddh >= 8);
            }
        }
        fetch_commit();
    };
    fetch(row0, 0);
    float dw[V][8], db[V][8];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        weight[k * all] = load_chunk(p.weight, 8 * (tid + k * threads) - shift, p.d, shift == 0 && p.wide_weight);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[k][i] = db[k][i] = 0.f;
    }
    const float of_row = 1.f / static_cast<float>(p.d);

    int turn = 0;  // of the stages and of row_sum2's places
    for (int64_t r = row0; r < p.m; r += stride, turn ^= 1) {
        const int row = static_cast<int>(r);
        const float rstd = p.rstd[row], mean = p.mean[row];
        fetch(r + stride, turn ^ 1);
        fetch_wait<1>();
        float sum = 0.f, dot = 0.f;  // of g and of g xhat
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int col0 = 8 * (tid + k * threads) - shift;
            float t[8], h[8], w[8];
            unpack(read_chunk(slot(turn, 0, k), col0), t);  // (outside the row dY is zero, and adds nothing)
            unpack(read_chunk(slot(turn, 1, k), col0), h);
            unpack(weight[k * all], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                db[k][i] += t[i];
                sum = fmaf(t[i], w[i], sum);
                t[i] *= (h[i] - mean) * rstd;
                dot = fmaf(t[i], w[i], dot);
                dw[k][i] += t[i];
            }
        }
        const float2 total = row_sum2(sum, dot, sums[turn]);
        const float mean_g = total.x * of_row, mean_gx = total.y * of_row;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int col0 = 8 * (tid + k * threads) - shift;
            if (col0 >= p.d) continue;
            float v[8], h[8], w[8];
            unpack(read_chunk(slot(turn, 0, k), col0), v);
            unpack(read_chunk(slot(turn, 1, k), col0), h);
            unpack(weight[k * all], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = rstd * (v[i] * w[i] - mean_g - (h[i] - mean) * rstd * mean_gx);
            if (p.dh) {
                unpack(read_chunk(slot(turn, 2, k), col0), h);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] += h[i];
            }
            store_chunk(p.dr + row * p.lddr, col0, p.d, p.wide, pack(v));
            if (DROP) {
                draw.chunk(v, row, col0);
                store_chunk(p.dx + row * p.lddx, col0, p.d, p.wide, pack(v));
            }
        }
    }
    fetch_wait<0>();

    float* part = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * p.d;
    if (blockDim.y == 1) {
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int col = 8 * (tid + k * threads) - shift + i;
                if (col >= 0 && col < p.d) {
                    part[col] = dw[k][i];
                    part[p.d + col] = db[k][i];
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
    for (int c = threadIdx.y * 32 + tid; c < 2 * p.d; c += 32 * blockDim.y) part[c] = total[c];
}

// The sums of the blocks' parts of both gradients, as join_kernel's.
__global__ void __launch_bounds__(kJoinColumns * kJoinParts) join2_kernel(const float* partial, int parts, int d,
                                                                          float* dweight, float* dbias) {
    allow_next_kernel();
    wait_for_earlier_kernels();
    __shared__ float sum[kJoinParts][kJoinColumns + 1];
    const int c = blockIdx.x * kJoinColumns + threadIdx.x;
    float v = 0.f;
    if (c < 2 * d) {
#pragma unroll 8
        for (int i = threadIdx.y; i < parts; i += kJoinParts) v += partial[static_cast<int64_t>(i) * 2 * d + c];
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
