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
constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kColumns = 32;  // of D: a warp's at a time

struct Params {
    const uint16_t* x;
    const uint16_t* a;       // [adapters, r, k]
    const uint16_t* b;       // [adapters, n, r]
    const int32_t* ids;
    const float* scale;      // or null: 1
    const uint16_t* r;       // or null
    uint16_t* d;
    uint16_t* low;           // [m][2][ldlow]: scale X A^T as the sum of two bf16
    int64_t ldx, lda, ldb, ldr, ldd;
    int64_t apart_a, apart_b;  // elements between adapters
    int m, n, k, rank, adapters;
    int ldlow;               // the rank, in whole tiles (of 16, or 32 beyond 16), zeros in the rest
    int act;
    int cluster;             // CTAs that share the columns of X
    int tile;                // rows of a tile (of the launch at hand)
    int parts;               // CTAs of a tile that share the columns of D
    int teams;               // of a CTA's warps: 16 or 32 ranks each
    int wide_r, wide_d;      // rows start on 16 bytes
};

// ---------------------------------------------------------------- a tile's rows by adapter

struct Order {
    int id[kMaxTile];          // as given; then in order
    int row[kMaxTile];         // in order: rows of one adapter together, those without one last
    int start[kMaxTile + 1];   // the groups' first places
    int groups;
};

// By all threads of a block; a row without an adapter has id -1 afterwards.
__device__ __forceinline__ void make_order(Order& o, const Params& p, int64_t row0, int rows) {
    __shared__ int given[kMaxTile];
    const int t = threadIdx.x;
    int key = p.adapters, first = p.adapters;  // (without one: after all others)
    if (t < rows) {
        const int id = p.ids[row0 + t], id0 = p.ids[row0];
        if (id >= 0 && id < p.adapters) key = id;
        if (id0 >= 0 && id0 < p.adapters) first = id0;
        given[t] = key;
    }
    if (__syncthreads_and(key == first || t >= rows)) {  // (a prompt's rows: one group)
        if (t < rows) {
            o.row[t] = t;
            o.id[t] = key < p.adapters ? key : -1;
        }
        if (t == 0) {
            o.start[0] = 0;
            o.start[1] = rows;
            o.groups = 1;
        }
        __syncthreads();
        return;
    }
    if (t < rows) {
        int at = 0;
#pragma unroll 8
        for (int i = 0; i < rows; ++i) at += given[i] < key || (given[i] == key && i < t);
        o.row[at] = t;
        o.id[at] = key < p.adapters ? key : -1;
    }
    __syncthreads();
    if (t < 32) {
        int groups = 0;
        for (int base = 0; base < rows; base += 32) {
            const int i = base + t;
            const bool begins = i < rows && (i == 0 || o.id[i] != o.id[i - 1]);
            const uint32_t on = __ballot_sync(0xffffffffu, begins);
            if (begins) o.start[groups + __popc(on & ((1u << t) - 1))] = i;
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
    constexpr int kUnroll = 2 * MT + NT <= 4 ? 4 : 2;
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

// A group's rows place .. place + rows - 1 (up to 8 NT).  The cluster's CTAs share the columns, and in each CTA a
// team of warps 16 MT ranks and, again, the columns; the sums are joined over the warps, then over the CTAs, in
// the same order on every run.  `joined`: the warps' sums; `mine`: the CTA's, one of two places in turn, so
// that a turn has one barrier of the cluster.
template <int MT, int NT>
__device__ __forceinline__ void down_part(const Params& p, const Order& o, float* joined, float* mine, int64_t row0, int rank,
                                          int adapter, int place, int rows) {
    constexpr int kOf = MT * NT * 128;  // sums of a warp
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sharing = kWarps / p.teams, team = warp / sharing, part = warp % sharing;
    const int by = p.cluster * sharing, last = (p.k + kStep - 1) / kStep;
    float c[MT][NT][4];
    down_sums<MT, NT>(c, p, o, row0, adapter, team * 16 * MT, place, rows, rank * sharing + part, by, last);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) joined[warp * kOf + (m * NT + t) * 128 + i * 32 + lane] = c[m][t][i];
    __syncthreads();
    for (int at = threadIdx.x; at < p.teams * kOf; at += kThreads) {
        const int its = at / kOf, in = at % kOf;
        float v = 0.f;
        for (int k = 0; k < sharing; ++k) v += joined[(its * sharing + k) * kOf + in];
        mine[at] = v;
    }
    cluster_sync();
    const float scale = p.scale ? p.scale[adapter] : 1.f;
    for (int at = rank * kThreads + threadIdx.x; at < p.teams * kOf; at += p.cluster * kThreads) {
        float v = 0.f;
        for (int k = 0; k < p.cluster; ++k) {
            float other;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(other) : "r"(mapa_shared(smem_addr(mine + at), k)) : "memory");
            v += other;
        }
        const int its = at / kOf, in = at % kOf;
        const int from = in & 31, i = in >> 5 & 3, t = (in >> 7) % NT, m = (in >> 7) / NT;
        const int j = (its * MT + m) * 16 + (from >> 2) + 8 * (i >> 1), row = 8 * t + 2 * (from & 3) + (i & 1);
        if (j < p.ldlow && row < rows) {
            uint16_t* to = p.low + (row0 + o.row[place + row]) * 2 * p.ldlow + j;
            split(j < p.rank ? v * scale : 0.f, to[0], to[p.ldlow]);
        }
    }
}

// Dynamic shared memory: the warps' sums, and two of the CTA's.
template <int MT>
__global__ void __launch_bounds__(kThreads, 2) down_kernel(const __grid_constant__ Params p) {
    allow_next_kernel();
    wait_for_earlier_kernels();
    __shared__ Order o;
    extern __shared__ float sums[];
    const int rank = blockIdx.x % p.cluster;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / p.cluster) * p.tile;
    make_order(o, p, row0, static_cast<int>(min(static_cast<int64_t>(p.tile), p.m - row0)));
    constexpr int kMost = MT * 4 * 128;
    int turn = 0;
    for (int i = 0; i < o.groups; ++i) {
        const int adapter = o.id[o.start[i]];
        if (adapter < 0) break;  // (the last group)
        for (int place = o.start[i]; place < o.start[i + 1]; place += 32, turn ^= 1) {
            const int rows = min(o.start[i + 1] - place, 32);
            float* mine = sums + (kWarps + turn * p.teams) * kMost;
            if (rows <= 8) down_part<MT, 1>(p, o, sums, mine, row0, rank, adapter, place, rows);
            else if (rows <= 16) down_part<MT, 2>(p, o, sums, mine, row0, rank, adapter, place, rows);
            else down_part<MT, 4>(p, o, sums, mine, row0, rank, adapter, place, rows);
        }
    }
    cluster_sync();  // (the others may still read this CTA's sums)
}

// ---------------------------------------------------------------- up to D

// Words of a row of one of S's terms in shared memory, so that the rows of a fragment's loads are in different banks:
// an odd multiple of 8 for 8-byte loads (eight rows of 8 words), of 16 for 16-byte ones.
__host__ __device__ constexpr int low_words(int ldlow) {
    const int unit = ldlow <= 16 ? 8 : 16, words = ldlow / 2;
    return words / unit % 2 ? words : words + unit;
}

// S's fragment words and B's: RS / 4 elements of a row at `col` (zeros from `cols` on).
template <int RS>
struct __align__(RS / 2) Words {
    uint32_t w[RS / 8];
};

template <int RS>
__device__ __forceinline__ Words<RS> load_words(const uint16_t* row, int col, int cols) {
    Words<RS> v;
    if (col + RS / 4 <= cols) {
        if constexpr (RS == 16) {
            const uint2 u = *reinterpret_cast<const uint2*>(row + col);
            v.w[0] = u.x, v.w[1] = u.y;
        } else {
            const uint4 u = *reinterpret_cast<const uint4*>(row + col);
            v.w[0] = u.x, v.w[1] = u.y, v.w[2] = u.z, v.w[3] = u.w;
        }
        return v;
    }
#pragma unroll
    for (int i = 0; i < RS / 8; ++i) {
        v.w[i] = col + 2 * i < cols ? row[col + 2 * i] : 0u;
        if (col + 2 * i + 1 < cols) v.w[i] |= static_cast<uint32_t>(row[col + 2 * i + 1]) << 16;
    }
    return v;
}

__device__ __forceinline__ uint4 load_row8(const uint16_t* row, int col, int cols, bool wide) {
    if (wide && col + 8 <= cols) return *reinterpret_cast<const uint4*>(row + col);
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = col + i < cols ? row[col + i] : 0u;
    return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
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

// A CTA: a tile of rows, and a part of D's columns in blocks of 32, a warp each.  The mma's columns are taken in an
// order in which a lane's sums are 8 neighbouring columns of a row: of a block's four mma tiles, column i of tile j
// is number 8 (i / 2) + 2 j + i % 2.  Rows are taken 32 at a time (two mma tiles), their R on its way together.
// Dynamic shared memory: S's first terms [row in order][low_words], then its second ones.
template <int RS>
__global__ void __launch_bounds__(kThreads, 2) up_kernel(const __grid_constant__ Params p) {
    allow_next_kernel();
    wait_for_earlier_kernels();
    __shared__ Order o;
    extern __shared__ __align__(16) uint32_t low[];
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / p.parts) * p.tile;
    const int rows = static_cast<int>(min(static_cast<int64_t>(p.tile), p.m - row0));
    make_order(o, p, row0, rows);
    const int words = low_words(p.ldlow), second = p.tile * words, chunks = p.ldlow / 8;
    for (int i = threadIdx.x; i < rows * 2 * chunks; i += kThreads) {
        const int place = i / (2 * chunks), j = i - place * 2 * chunks, term = j >= chunks;
        if (o.id[place] < 0) continue;
        *reinterpret_cast<uint4*>(low + term * second + place * words + 4 * (j - term * chunks)) =
            *reinterpret_cast<const uint4*>(p.low + ((row0 + o.row[place]) * 2 + term) * p.ldlow + 8 * (j - term * chunks));
    }
    __syncthreads();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int64_t step = static_cast<int64_t>(p.parts) * kWarps * kColumns;
    for (int64_t at64 = (static_cast<int64_t>(blockIdx.x % p.parts) * kWarps + warp) * kColumns; at64 < p.n; at64 += step) {
        const int col0 = static_cast<int>(at64), col = col0 + 8 * q;
        for (int i = 0; i < o.groups; ++i) {
            const int adapter = o.id[o.start[i]], end = o.start[i + 1];
            const uint16_t* b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)  // (columns beyond the last are the last's)
                b[j] = p.b + max(adapter, 0) * p.apart_b + min(col0 + 8 * (g >> 1) + 2 * j + (g & 1), p.n - 1) * p.ldb;
            for (int place = o.start[i]; place < end; place += 32) {
                const bool both = place + 16 < end;
                uint4 r[4];
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    if (p.r && place + g + 8 * h < end)
                        r[h] = load_row8(p.r + (row0 + o.row[place + g + 8 * h]) * p.ldr, col, p.n, p.wide_r);
                float c[2][4][4];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int k = 0; k < 4; ++k) c[t][j][k] = 0.f;
                if (adapter >= 0) {
                    const uint32_t* s[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h) s[h] = low + min(place + g + 8 * h, end - 1) * words + RS / 8 * q;
#pragma unroll 2
                    for (int k0 = 0; k0 < p.ldlow; k0 += RS) {
                        Words<RS> u[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) u[j] = load_words<RS>(b[j], k0 + RS / 4 * q, p.rank);
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (t && !both) continue;
#pragma unroll
                            for (int term = 0; term < 2; ++term) {
                                const Words<RS> x = *reinterpret_cast<const Words<RS>*>(s[2 * t] + term * second + k0 / 2);
                                const Words<RS> y = *reinterpret_cast<const Words<RS>*>(s[2 * t + 1] + term * second + k0 / 2);
#pragma unroll
                                for (int w = 0; w < RS / 8; w += 2)
#pragma unroll
                                    for (int j = 0; j < 4; ++j)
                                        mma(c[t][j], x.w[w], y.w[w], x.w[w + 1], y.w[w + 1], u[j].w[w], u[j].w[w + 1]);
                            }
                        }
                    }
                }
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    if (place + g + 8 * h >= end) continue;
                    float v[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = c[h >> 1][k >> 1][2 * (h & 1) + (k & 1)];
                    if (p.r) {
                        const uint32_t w[4] = {r[h].x, r[h].y, r[h].z, r[h].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            v[2 * k] += __uint_as_float(w[k] << 16);
                            v[2 * k + 1] += __uint_as_float(w[k] & 0xffff0000u);
                        }
                    }
                    if (p.act)
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] = activate(v[k], p.act);
                    store_row8(p.d + (row0 + o.row[place + g + 8 * h]) * p.ldd, col, p.n, p.wide_d, v);
                }
            }
        }
    }
}

}  // namespace lora
}  // namespace gb
