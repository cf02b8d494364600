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

#include "ptx.cuh"

namespace gb {
namespace rowwise {

// ---------------------------------------------------------------- the generator

// Philox4x32 with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy
// as 1, 2, 3", SC 2011): each round multiplies two of the counter's words by constants, and
// crosses the products' halves with the others and the key, which then moves on by its Weyl
// increments.  Element (row, col) of a matrix takes word col % 4 of the counter
// (col / 4, row, offset low, offset high) under the key `seed`.
//
// The ten rounds' keys come with the launch (constant memory: no instruction and no register), or
// are made from a seed in device memory.
struct Drop {
    uint32_t keys[10][2];
    uint32_t offset[2];
    const uint64_t* state;  // device memory {seed, offset} in the place of the two above, or null
    uint32_t limit;         // kept: words above it
    float scale;            // of a kept element: 1 / (1 - p)
};

// What a kernel draws with: kNoDrop nothing, kKeys the launch's keys, kState those of `state`.
enum { kNoDrop = 0, kKeys = 1, kState = 2 };

template <int DROP>
struct Draw {
    const Drop& d;
    uint32_t seed[2], offset[2];

    __device__ __forceinline__ explicit Draw(const Drop& drop) : d(drop), seed{0, 0}, offset{0, 0} {
        if (DROP == kState) {
            const uint64_t s = drop.state[0], o = drop.state[1];
            seed[0] = static_cast<uint32_t>(s);
            seed[1] = static_cast<uint32_t>(s >> 32);
            offset[0] = static_cast<uint32_t>(o);
            offset[1] = static_cast<uint32_t>(o >> 32);
        } else if (DROP == kKeys) {
            offset[0] = drop.offset[0];
            offset[1] = drop.offset[1];
        }
    }

    __device__ __forceinline__ void words(uint32_t group, uint32_t row, uint32_t (&out)[4]) const {
        uint32_t c0 = group, c1 = row, c2 = offset[0], c3 = offset[1], k0 = seed[0], k1 = seed[1];
        // (in a form that the compiler does not see to be the same on every call: else it keeps the
        // twenty keys in registers across the loop over rows)
        if (DROP == kState) asm volatile("" : "+r"(k0), "+r"(k1));
#pragma unroll
        for (int i = 0; i < 10; ++i) {
            if (DROP == kKeys) {
                k0 = d.keys[i][0];
                k1 = d.keys[i][1];
            }
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

    // Which of four elements of a group are kept (bits 0 .. 3).
    __device__ __forceinline__ uint32_t kept(uint32_t group, int row) const {
        uint32_t w[4], bits = 0;
        words(group, static_cast<uint32_t>(row), w);
#pragma unroll
        for (int i = 0; i < 4; ++i) bits |= w[i] > d.limit ? 1u << i : 0u;
        return bits;
    }

    // Drop the chunk of `row` at columns col0 .. col0 + 7.  A dropped element is zero whatever it was
    // (an infinity or a NaN among them): it is selected, not multiplied.
    __device__ __forceinline__ void chunk(float (&v)[8], int row, int col0) const {
        // a column below 0 is not an element: its word is not used, and the group -1 or -2 wraps
        const int phase = col0 & 3;  // (the same for the whole row)
        const uint32_t group = static_cast<uint32_t>((col0 - phase) >> 2);
        if (phase == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t w[4];
                words(group + h, static_cast<uint32_t>(row), w);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[4 * h + i] = w[i] > d.limit ? v[4 * h + i] * d.scale : 0.f;
            }
            return;
        }
        uint32_t bits = kept(group, row);
        bits |= kept(group + 1, row) << 4;
        if (phase) bits |= kept(group + 2, row) << 8;
        bits >>= phase;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = bits >> i & 1 ? v[i] * d.scale : 0.f;
    }
};

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

// The chunk's elements of `row` (0 outside the row).
__device__ __forceinline__ uint4 load_chunk(const uint16_t* row, int col0, int cols, bool wide) {
    if (wide && col0 >= 0 && col0 + 8 <= cols) return *reinterpret_cast<const uint4*>(row + col0);
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = col0 + i >= 0 && col0 + i < cols ? row[col0 + i] : 0u;
    return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
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

// A chunk on its way to the thread's own 16 bytes of shared memory: a thread reads only what it
// asked for itself, so that waiting for its own copies is all the order there has to be.  A row's
// first chunk may start before the row: `inside` says that this is memory of the matrix too (of the
// row before); what it holds of that is cleared by read_chunk().
__device__ __forceinline__ void fetch_chunk(uint4* to, const uint16_t* row, int col0, int cols, bool wide, bool inside) {
    if (wide && col0 < cols && (col0 >= 0 || inside)) {
        const int bytes = min(16, 2 * (cols - col0));  // (zeros after a row's end)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         static_cast<uint32_t>(__cvta_generic_to_shared(to))),
                     "l"(row + col0), "r"(bytes)
                     : "memory");
    } else {
        *to = load_chunk(row, col0, cols, false);
    }
}

__device__ __forceinline__ uint4 read_chunk(const uint4* from, int col0) {
    uint4 u = *from;
    if (col0 < 0) {  // (-7 .. -1)
        const int n = -col0;
        uint32_t* w = &u.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = n >= 2 * i + 2 ? 0u : n == 2 * i + 1 ? w[i] & 0xffff0000u : w[i];
    }
    return u;
}

__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void fetch_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---------------------------------------------------------------- dropout

struct DropoutParams {
    const uint16_t* x;
    const uint16_t* r;  // added, or null
    uint16_t* d;
    int64_t ldx, ldr, ldd;
    int m, n;
    int chunks;  // of a row, its shift counted in
    int64_t step_rows;  // the grid's threads in rows and chunks
    int step_chunks;
    int wide;
    Drop drop;
};

constexpr int kDropoutThreads = 256, kDropoutBatch = 2;

// Threads walk the matrix's chunks a grid's width apart, kDropoutBatch at a time; a step of the
// walk is `step_rows` rows and `step_chunks` chunks, so that no thread divides again.
//
// Four words take twenty 32 x 32 -> 64 bit multiplications: at 8192 x 14336 the multiplier's pipe is
// busy 62 % and the logic's 55 % of the time (4096 rows), and the generator, not the memory, is the bound:
// 120 us for 470 MB (3.9 TB/s, 0.58 of the copy bandwidth), 133 us for 705 MB with a residual (5.3 TB/s,
// 0.78) on a GB300.  One chunk at a time took 138 us, three 139, 40 registers instead of 48 took 142,
// and blocks that walk rows 150.
template <int DROP>
__global__ void __launch_bounds__(kDropoutThreads, 5) dropout_kernel(const __grid_constant__ DropoutParams p) {
    allow_next_kernel();
    wait_for_earlier_kernels();
    const Draw<DROP> draw(p.drop);
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kDropoutThreads + threadIdx.x;
    int64_t row = at / p.chunks;
    int j = static_cast<int>(at - row * p.chunks);
    while (row < p.m) {
        uint4 xu[kDropoutBatch], ru[kDropoutBatch];
        int rows[kDropoutBatch], col0[kDropoutBatch];
#pragma unroll
        for (int u = 0; u < kDropoutBatch; ++u) {
            rows[u] = static_cast<int>(row);
            const uint16_t* x = p.x + row * p.ldx;
            col0[u] = row < p.m ? 8 * j - (p.wide ? row_shift(x) : 0) : p.n;
            if (col0[u] < p.n) {
                xu[u] = load_chunk(x, col0[u], p.n, p.wide);
                if (p.r) ru[u] = load_chunk(p.r + row * p.ldr, col0[u], p.n, p.wide);
            }
            row += p.step_rows;
            j += p.step_chunks;
            if (j >= p.chunks) {
                j -= p.chunks;
                ++row;
            }
        }
#pragma unroll
        for (int u = 0; u < kDropoutBatch; ++u) {
            if (col0[u] >= p.n) continue;
            float v[8];
            unpack(xu[u], v);
            if (DROP) draw.chunk(v, rows[u], col0[u]);
            if (p.r) {
                float r[8];
                unpack(ru[u], r);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] += r[i];
            }
            store_chunk(p.d + static_cast<int64_t>(rows[u]) * p.ldd, col0[u], p.n, p.wide, pack(v));
        }
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
// before its rounding.  V chunks a thread.  A block takes the rows row0, row0 + stride, ...:
// `stride` is a multiple of 8 rows, so a thread's rows all have the same shift and it keeps its
// part of the weight; kRowStages - 1 rows are on their way beside the one that is worked on.
// Dynamic shared memory: the rows [stage][x or r][chunk][thread], the weight, kGroupScale's maxima.
//
// 8192 x 4096 with a residual on a GB300: 45 to 46 us, 5.9 TB/s (0.87 of the copy bandwidth); with
// dropout 57 us, bound by the generator's instructions (64 % of issue slots used); 8-bit output 46 us
// with a scale a row (0.75), 54 us for each 128 columns.  The first kernel, blocks that each load one
// row and end, took 85 us with dropout; rows ahead of their turn and keys in constant memory 66.
constexpr int kRowStages = 3;

template <int V, int DROP, int OUT>
__global__ void __maxnreg__(V == 4 ? 128 : DROP ? 80 : 64) norm_kernel(const __grid_constant__ NormParams p) {
    allow_next_kernel();
    wait_for_earlier_kernels();
    __shared__ float sums[2][32];
    __shared__ uint32_t maxima[2][32];
    extern __shared__ __align__(16) uint8_t smem[];
    const int row0 = blockIdx.x * blockDim.y + threadIdx.y, stride = gridDim.x * blockDim.y;
    const int shift = p.wide ? row_shift(p.x + row0 * p.ldx) : 0;
    const int tid = threadIdx.x, threads = blockDim.x, all = blockDim.x * blockDim.y;
    uint4* slots = reinterpret_cast<uint4*>(smem) + threadIdx.y * threads + tid;
    uint32_t* group_max = reinterpret_cast<uint32_t*>(smem + static_cast<size_t>(kRowStages * 2 + 1) * V * all * 16);
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
    for (int s = 0; s < kRowStages - 1; ++s) fetch(row0 + static_cast<int64_t>(s) * stride, s);
    uint4* weight = slots + kRowStages * 2 * V * all;  // (the thread's own part of it)
#pragma unroll
    for (int k = 0; k < V; ++k)
        weight[k * all] = load_chunk(p.weight, 8 * (tid + k * threads) - shift, p.d, shift == 0 && p.wide_weight);

    int stage = 0, turn = 0;
    for (int64_t r = row0; r < p.m; r += stride, turn ^= 1) {
    const int row = static_cast<int>(r);
    fetch(r + static_cast<int64_t>(kRowStages - 1) * stride, stage == 0 ? kRowStages - 1 : stage - 1);
    fetch_wait<kRowStages - 1>();
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
        for (int i = 0; i < 8; ++i) sum = fmaf(v[k][i], v[k][i], sum);
        if (p.h && col0 < p.d) store_chunk(p.h + row * p.ldh, col0, p.d, p.wide, pack(v[k]));
    }
    stage = stage == kRowStages - 1 ? 0 : stage + 1;
    const float rstd = 1.f / sqrtf(row_sum(sum, sums[turn]) / static_cast<float>(p.d) + p.eps);
    if (p.rstd && tid == 0) p.rstd[row] = rstd;

#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int col0 = 8 * (tid + k * threads) - shift;
        float w[8];
        unpack(weight[k * all], w);
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
        const float scale = scale_of(row_max(top, maxima[turn]));
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
    if (OUT == kGroupScale && shift == 0) {
        // a group is sixteen lanes' chunks
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int col0 = 8 * (tid + k * threads);
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[k][i]) & 0x7fffffffu);
#pragma unroll
            for (int i = 8; i > 0; i >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, i));
            const float scale = scale_of(top), inv = 1.f / scale;
            if (col0 >= p.d) continue;
            if ((tid & 15) == 0) p.scale[row * p.lds + col0 / kScaleGroup] = scale;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] *= inv;
            store_e4m3(p.q + row * p.ldq, col0, p.d, p.wide, v[k]);
        }
        __syncwarp();
    } else if (OUT == kGroupScale) {
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
        if (blockDim.y > 1) __syncwarp();
        else __syncthreads();  // (the next row clears the maxima)
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
    Drop drop;
};

// With xhat = h rstd and g = dy weight:  dr = rstd (g - xhat mean(g xhat)) + dh,
// dx = dropout's gradient of dr,  dweight = sum over rows of dy xhat.
// A block takes the rows row0, row0 + stride, ...: `stride` is a multiple of 8 rows, so a
// thread's rows all have the same shift and it owns the same columns in each; the weight's
// gradient stays in its registers until the end.
// V chunks a thread.  The rows come through shared memory as the forward pass's do, in two stages.
// Dynamic shared memory: the rows [stage][dY, H or dH][chunk][thread], then the weight.
//
// 8192 x 4096 with dH on a GB300, the join of the weight's gradient with it: 51.2 us, 5.2 TB/s (0.77 of
// the copy bandwidth), and 78 us with dropout (10 bytes an element and the generator; 0.63).  The first
// kernel, with its rows in registers and two blocks an SM, took 110 us; 512 threads an SM take 107 us,
// or 82 with a third stage, where 768 take 78.
constexpr int kBwdStages = 2;

template <int V, int DROP>
__global__ void __maxnreg__(V == 4 ? 128 : 80) norm_bwd_kernel(const __grid_constant__ NormBwdParams p) {
    allow_next_kernel();
    wait_for_earlier_kernels();
    __shared__ float sums[2][32];
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
    float dw[V][8];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        weight[k * all] = load_chunk(p.weight, 8 * (tid + k * threads) - shift, p.d, shift == 0 && p.wide_weight);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[k][i] = 0.f;
    }

    int turn = 0;  // of the stages and of row_sum's places
    for (int64_t r = row0; r < p.m; r += stride, turn ^= 1) {
        const int row = static_cast<int>(r);
        const float rstd = p.rstd[row];
        fetch(r + stride, turn ^ 1);
        fetch_wait<1>();
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int col0 = 8 * (tid + k * threads) - shift;
            float t[8], h[8], w[8];
            unpack(read_chunk(slot(turn, 0, k), col0), t);
            unpack(read_chunk(slot(turn, 1, k), col0), h);
            unpack(weight[k * all], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                t[i] *= h[i] * rstd;
                sum = fmaf(t[i], w[i], sum);
                dw[k][i] += t[i];
            }
        }
        const float mean = row_sum(sum, sums[turn]) / static_cast<float>(p.d);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int col0 = 8 * (tid + k * threads) - shift;
            if (col0 >= p.d) continue;
            float v[8], h[8], w[8];
            unpack(read_chunk(slot(turn, 0, k), col0), v);
            unpack(read_chunk(slot(turn, 1, k), col0), h);
            unpack(weight[k * all], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = rstd * (v[i] * w[i] - h[i] * rstd * mean);
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

    float* part = p.partial + static_cast<int64_t>(blockIdx.x) * p.d;
    if (blockDim.y == 1) {
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int col = 8 * (tid + k * threads) - shift + i;
                if (col >= 0 && col < p.d) part[col] = dw[k][i];
            }
        return;
    }
    // several rows a block: the warps add theirs one after the other, where the rows were
    __syncthreads();
    float* total = reinterpret_cast<float*>(smem);
    for (int c = threadIdx.y * 32 + tid; c < p.d; c += 32 * blockDim.y) total[c] = 0.f;
    for (int w = 0; w < static_cast<int>(blockDim.y); ++w) {
        __syncthreads();
        if (w != static_cast<int>(threadIdx.y)) continue;
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int col = 8 * (tid + k * threads) - shift + i;
                if (col >= 0 && col < p.d) total[col] += dw[k][i];
            }
    }
    __syncthreads();
    for (int c = threadIdx.y * 32 + tid; c < p.d; c += 32 * blockDim.y) part[c] = total[c];
}

// dweight[c] = the sum of the blocks' parts, in the same order on every run: 32 threads to a column,
// each with eight of its parts on their way at a time.
constexpr int kJoinColumns = 32, kJoinParts = 32;
__global__ void __launch_bounds__(kJoinColumns * kJoinParts) join_kernel(const float* partial, int parts, int d,
                                                                         float* dweight) {
    allow_next_kernel();
    wait_for_earlier_kernels();
    __shared__ float sum[kJoinParts][kJoinColumns + 1];
    const int c = blockIdx.x * kJoinColumns + threadIdx.x;
    float v = 0.f;
    if (c < d) {
#pragma unroll 8
        for (int i = threadIdx.y; i < parts; i += kJoinParts) v += partial[static_cast<int64_t>(i) * d + c];
    }
    sum[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    // a warp to a column
    const int column = blockIdx.x * kJoinColumns + threadIdx.y;
    v = warp_sum(sum[threadIdx.x][threadIdx.y]);
    if (threadIdx.x == 0 && column < d) dweight[column] = v;
}

}  // namespace rowwise
}  // namespace gb
