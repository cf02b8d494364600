// Device code of the low-rank adapters of many requests:
//
//   D[m] = act( R[m] + s[a] B[a] (A[a] X[m]) )      a = ids[m], none where it is outside 0 .. adapters - 1
//
// Two launches: down to the rank (S = X A^T, the columns split over CTAs), and up to D.  Rows come in any order:
// each CTA takes a tile of consecutive rows and sorts it by adapter for itself, so that rows of one adapter
// share its matrices' fragments and no launch is spent on an order of the whole batch.  Both are bound by memory:
// X, R and D once, and the adapters' matrices.
#pragma once

#include "skinny.cuh"

namespace gb {
namespace lora {

using namespace skinny;

constexpr int kMaxRank = 256;
constexpr int kMaxTile = 64;
constexpr int kDownWarps = 8, kDownThreads = 32 * kDownWarps;
constexpr int kUpWarps = 4, kUpThreads = 32 * kUpWarps;
constexpr int kUpColumns = 32;  // of a warp

struct Params {
    const uint16_t* x;
    const uint16_t* a;       // [adapters, r, k]
    const uint16_t* b;       // [adapters, n, r]
    const int32_t* ids;
    const float* scale;      // or null: 1
    const uint16_t* r;       // or null
    uint16_t* d;
    float* low;              // [splits, m, ldlow]: the splits' parts of X A^T
    int64_t ldx, lda, ldb, ldr, ldd;
    int64_t apart_a, apart_b;  // elements between adapters
    int m, n, k, rank, adapters;
    int ldlow;               // the rank, in whole tiles of 16
    int act;
    int splits, split_steps; // the columns' parts, and their steps
    int tile;                // rows of a tile (of the launch at hand)
    int chunks;              // of 128 columns: CTAs of a tile
    int wide_r, wide_d;      // rows start on 16 bytes
};

// ---------------------------------------------------------------- a tile's rows by adapter

struct Order {
    int id[kMaxTile];          // as given; then in order
    int row[kMaxTile];         // in order: rows of one adapter together, those without one last
    int start[kMaxTile + 1];   // the groups' first places
    int groups;
};

// By all threads of a block of at least 64; a row without an adapter has id -1 afterwards.
__device__ __forceinline__ void make_order(Order& o, const Params& p, int64_t row0, int rows) {
    __shared__ int given[kMaxTile];
    const int t = threadIdx.x;
    int key = p.adapters;  // (without one: after all others)
    if (t < rows) {
        const int id = p.ids[row0 + t];
        if (id >= 0 && id < p.adapters) key = id;
        given[t] = key;
    }
    __syncthreads();
    if (t < rows) {
        int at = 0;
        for (int i = 0; i < rows; ++i) at += given[i] < key || (given[i] == key && i < t);
        o.row[at] = t;
        o.id[at] = key < p.adapters ? key : -1;
    }
    __syncthreads();
    if (t < 32) {
        int groups = 0;
        for (int base = 0; base < rows; base += 32) {
            const int i = base + t;
            const bool first = i < rows && (i == 0 || o.id[i] != o.id[i - 1]);
            const uint32_t on = __ballot_sync(0xffffffffu, first);
            if (first) o.start[groups + __popc(on & ((1u << t) - 1))] = i;
            groups += __popc(on);
        }
        if (t == 0) {
            o.start[groups] = rows;
            o.groups = groups;
        }
    }
    __syncthreads();
}

// ---------------------------------------------------------------- down to the rank

// 16 MT ranks of one adapter with up to 8 NT rows of X, over the steps first, first + by, ... before last.
template <int MT, int NT>
__device__ __forceinline__ void down_sums(float (&c)[MT][NT][4], const Params& p, const Order& o, int64_t row0, int adapter,
                                          int rank0, int place, int rows, int first, int by, int last) {
    constexpr int kUnroll = MT * NT <= 2 ? 4 : NT <= 2 ? 2 : 1;
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    // (ranks beyond the last are the last's, rows the first's: their sums are not used)
    const uint16_t* a[2 * MT];
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) a[i] = p.a + adapter * p.apart_a + min(rank0 + g + 8 * i, p.rank - 1) * p.lda;
    const uint16_t* x[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) x[t] = p.x + (row0 + o.row[place + (8 * t + g < rows ? 8 * t + g : 0)]) * p.ldx;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) c[m][t][i] = 0.f;
    const int whole = min(last, p.k / kStep);
    int s = first;
    for (; s + (kUnroll - 1) * by < whole; s += kUnroll * by) {
        uint4 u[kUnroll][2 * MT], v[kUnroll][NT];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            const int col = (s + j * by) * kStep + 8 * q;
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) u[j][i] = *reinterpret_cast<const uint4*>(a[i] + col);
#pragma unroll
            for (int t = 0; t < NT; ++t) v[j][t] = *reinterpret_cast<const uint4*>(x[t] + col);
        }
#pragma unroll
        for (int j = 0; j < kUnroll; ++j)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int t = 0; t < NT; ++t) mma_step(c[m][t], u[j][2 * m], u[j][2 * m + 1], v[j][t]);
    }
    for (; s < last; s += by) {
        const int col = s * kStep + 8 * q;
        uint4 u[2 * MT];
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) u[i] = load_edge(a[i], col, p.k);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint4 v = load_edge(x[t], col, p.k);
#pragma unroll
            for (int m = 0; m < MT; ++m) mma_step(c[m][t], u[2 * m], u[2 * m + 1], v);
        }
    }
}

// A group's rows place .. place + rows - 1 (up to 8 NT): the warps share 16 MT ranks each, and the columns.
template <int MT, int NT>
__device__ __forceinline__ void down_part(const Params& p, const Order& o, float* joined, int64_t row0, int split, int adapter,
                                          int place, int rows) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int teams = 1;  // of the ranks
    while (teams < kDownWarps && teams * 16 * MT < p.rank) teams *= 2;
    const int sharing = kDownWarps / teams, team = warp / sharing, part = warp % sharing;
    const int begin = split * p.split_steps, last = min(begin + p.split_steps, (p.k + kStep - 1) / kStep);
    // (256 ranks at most: one turn of eight warps with two tiles)
    float c[MT][NT][4];
    down_sums<MT, NT>(c, p, o, row0, adapter, team * 16 * MT, place, rows, begin + part, sharing, last);
    __syncthreads();  // (the part before has been read)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) joined[((warp * MT + m) * NT + t) * 128 + i * 32 + lane] = c[m][t][i];
    __syncthreads();
    constexpr int kOf = MT * NT * 128;  // sums of a warp
    float* low = p.low + (static_cast<int64_t>(split) * p.m + row0) * p.ldlow;
    for (int at = threadIdx.x; at < teams * kOf; at += kDownThreads) {
        const int its = at / kOf, in = at % kOf;
        float v = 0.f;
        for (int k = 0; k < sharing; ++k) v += joined[(its * sharing + k) * kOf + in];
        const int from = in & 31, i = in >> 5 & 3, t = (in >> 7) % NT, m = (in >> 7) / NT;
        const int rank = (its * MT + m) * 16 + (from >> 2) + 8 * (i >> 1), row = 8 * t + 2 * (from & 3) + (i & 1);
        if (rank < p.rank && row < rows) low[static_cast<int64_t>(o.row[place + row]) * p.ldlow + rank] = v;
    }
}

template <int MT>
__global__ void __launch_bounds__(kDownThreads, 2) down_kernel(const __grid_constant__ Params p) {
    allow_next_kernel();
    wait_for_earlier_kernels();
    __shared__ Order o;
    __shared__ float joined[kDownWarps * MT * 4 * 128];
    const int split = blockIdx.x % p.splits;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / p.splits) * p.tile;
    make_order(o, p, row0, static_cast<int>(min(static_cast<int64_t>(p.tile), p.m - row0)));
    for (int i = 0; i < o.groups; ++i) {
        const int adapter = o.id[o.start[i]];
        if (adapter < 0) break;  // (the last group)
        for (int place = o.start[i]; place < o.start[i + 1]; place += 32) {
            const int rows = min(o.start[i + 1] - place, 32);
            if (rows <= 8) down_part<MT, 1>(p, o, joined, row0, split, adapter, place, rows);
            else if (rows <= 16) down_part<MT, 2>(p, o, joined, row0, split, adapter, place, rows);
            else down_part<MT, 4>(p, o, joined, row0, split, adapter, place, rows);
        }
    }
}

// ---------------------------------------------------------------- up to D

// Words of a row of S in shared memory (a term): an odd multiple of 8, so that the eight rows of a fragment's
// 8-byte loads are in different banks.
__host__ __device__ constexpr int low_words(int ldlow) { return ldlow / 16 % 2 ? ldlow / 2 : ldlow / 2 + 8; }

// Four elements of a row of B (zeros from `cols` on).
__device__ __forceinline__ uint2 load_four(const uint16_t* row, int col, int cols) {
    if (col + 4 <= cols) return *reinterpret_cast<const uint2*>(row + col);
    uint32_t e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = col + i < cols ? row[col + i] : 0u;
    return make_uint2(e[0] | e[1] << 16, e[2] | e[3] << 16);
}

__device__ __forceinline__ void load_row8(float (&v)[8], const uint16_t* row, int col, int cols, bool wide) {
    uint4 u;
    if (wide && col + 8 <= cols) {
        u = *reinterpret_cast<const uint4*>(row + col);
    } else {
        uint32_t e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = col + i < cols ? row[col + i] : 0u;
        u = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
    }
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ void store_row8(uint16_t* row, int col, int cols, bool wide, const float (&v)[8]) {
    if (wide && col + 8 <= cols) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = bf16_bits(v[2 * i]) | static_cast<uint32_t>(bf16_bits(v[2 * i + 1])) << 16;
        *reinterpret_cast<uint4*>(row + col) = make_uint4(w[0], w[1], w[2], w[3]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (col + i < cols) row[col + i] = bf16_bits(v[i]);
}

// A CTA: a tile of rows, 128 columns of D.  S, scaled, is multiplied as two bf16 terms.  The mma's columns are
// taken in an order in which a lane's sums are 8 neighbouring columns of a row: of the four mma tiles of a warp's
// 32 columns, column i of tile j is number 8 (i / 2) + 2 j + i % 2.
// Dynamic shared memory: S's first terms [row in order][low_words], then its second ones.
__global__ void __launch_bounds__(kUpThreads) up_kernel(const __grid_constant__ Params p) {
    allow_next_kernel();
    wait_for_earlier_kernels();
    __shared__ Order o;
    extern __shared__ __align__(16) uint32_t low[];
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / p.chunks) * p.tile;
    const int rows = static_cast<int>(min(static_cast<int64_t>(p.tile), p.m - row0));
    make_order(o, p, row0, rows);
    const int words = low_words(p.ldlow), second = p.tile * words;
    uint16_t* terms = reinterpret_cast<uint16_t*>(low);
    for (int i = threadIdx.x; i < rows * p.ldlow; i += kUpThreads) {
        const int place = i / p.ldlow, j = i - place * p.ldlow, id = o.id[place];
        float v = 0.f;
        if (id >= 0 && j < p.rank) {
            const float* from = p.low + (row0 + o.row[place]) * p.ldlow + j;
            for (int s = 0; s < p.splits; ++s) v += from[static_cast<int64_t>(s) * p.m * p.ldlow];
            if (p.scale) v *= p.scale[id];
        }
        split(v, terms[2 * place * words + j], terms[2 * (second + place * words) + j]);
    }
    __syncthreads();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int64_t col64 = (static_cast<int64_t>(blockIdx.x % p.chunks) * kUpWarps + warp) * kUpColumns;
    if (col64 >= p.n) return;
    const int col0 = static_cast<int>(col64), col = col0 + 8 * q;
    for (int i = 0; i < o.groups; ++i) {
        const int adapter = o.id[o.start[i]], end = o.start[i + 1];
        const uint16_t* b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)  // (columns beyond the last are the last's)
            b[j] = p.b + max(adapter, 0) * p.apart_b + min(col0 + 8 * (g >> 1) + 2 * j + (g & 1), p.n - 1) * p.ldb;
        for (int place = o.start[i]; place < end; place += 16) {
            int64_t row[2];
            float v[2][8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = place + g + 8 * h;
                row[h] = at < end ? row0 + o.row[at] : -1;
                if (p.r && row[h] >= 0) {
                    load_row8(v[h], p.r + row[h] * p.ldr, col, p.n, p.wide_r);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[h][k] = 0.f;
                }
            }
            if (adapter >= 0) {
                float c[4][4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) c[j][k] = 0.f;
                const uint32_t* s0 = low + min(place + g, end - 1) * words + 2 * q;
                const uint32_t* s1 = low + min(place + g + 8, end - 1) * words + 2 * q;
#pragma unroll 4
                for (int k0 = 0; k0 < p.ldlow; k0 += 16) {
                    uint2 u[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) u[j] = load_four(b[j], k0 + 4 * q, p.rank);
#pragma unroll
                    for (int term = 0; term < 2; ++term) {
                        const uint2 lo = *reinterpret_cast<const uint2*>(s0 + term * second + k0 / 2);
                        const uint2 hi = *reinterpret_cast<const uint2*>(s1 + term * second + k0 / 2);
#pragma unroll
                        for (int j = 0; j < 4; ++j) mma(c[j], lo.x, hi.x, lo.y, hi.y, u[j].x, u[j].y);
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[h][2 * j] += c[j][2 * h];
                        v[h][2 * j + 1] += c[j][2 * h + 1];
                    }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (row[h] < 0) continue;
#pragma unroll
                for (int k = 0; k < 8; ++k) v[h][k] = activate(v[h][k], p.act);
                store_row8(p.d + row[h] * p.ldd, col, p.n, p.wide_d, v[h]);
            }
        }
    }
}

}  // namespace lora
}  // namespace gb
