// Device code of the low-rank adapters of many requests:
//
//   D[m] = act( R[m] + s[a] B[a] (A[a] X[m]) )      a = ids[m], none where it is outside 0 .. adapters - 1
//
// Two launches: down to the rank (S = X A^T, the columns split over CTAs), and up to D.  Rows come in any order, and
// rows of one adapter share its matrices' fragments: from 32 rows on they are sorted (up to 128 by each CTA for itself,
// more by a launch before the two), and a tile has rows of one adapter.  (A tile in which two requests meet takes a turn
// for each, and the launch waits for it: 1000 rows of 30 requests, with tiles of consecutive rows, 49 us.)  Both products
// are bound by memory: X, R and D once, and the adapters' matrices.
#pragma once

#include <type_traits>

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
    uint16_t* low;           // [m][2 ldlow]: scale X A^T as the sum of two bf16 terms, placed as term_at() says
    int64_t ldx, lda, ldb, ldr, ldd;
    int64_t apart_a, apart_b;  // elements between adapters
    int m, n, k, rank, adapters;
    int ldlow;               // the rank, in whole tiles (of 16, or 32 beyond 16), zeros in the rest
    int act;
    int cluster;             // CTAs that share the columns of X
    int tile;                // rows of a tile (of the launch at hand)
    int parts;               // CTAs of a tile that share the columns of D (of sorted rows: tiles[0] has them)
    int up_blocks;           // of the product up to D
    int teams;               // of a CTA's warps: 16 or 32 ranks each
    // of sorted rows (else null): {tiles whose rows have an adapter, all tiles, blocks of a tile in the product up to D},
    // then the tiles; the rows in order
    const int4* tiles;
    const int32_t* order;
    int here;                // few rows, which each CTA sorts for itself
};

// A tile of sorted rows.
__device__ __forceinline__ int4 tile_of(int adapter, int start, int count) { return make_int4(adapter, start, count, 0); }

// Blocks that share a tile's columns in the product up to D, by a warp: of least time if a tile's order and S take a
// block what 32 columns take a warp.
__device__ __forceinline__ int parts_of(int tiles, int blocks, int n) {
    const int turns = (n + kWarps * kColumns - 1) / (kWarps * kColumns), each = min(static_cast<int>(threadIdx.x & 15) + 1, turns);
    const uint32_t parts = (turns + each - 1) / each, rounds = (tiles * parts + blocks - 1) / blocks;
    const uint32_t best = __reduce_min_sync(0xffffffffu, rounds * (each + 1) * 32 + each);
    return (turns + (best & 31) - 1) / (best & 31);
}

// ---------------------------------------------------------------- all rows by adapter

// One block: 5.5 us for 1000 rows, 7.8 for 8192, of which the launch and the first loads are the half.
constexpr int kSortThreads = 1024, kSortBatch = 8, kMaxSorted = 8191;  // adapters: a counter each in shared memory

// A count of the rows of each adapter (and of those without one), the starts, and each row to its adapter's next
// place.  Which place is its own decides nothing: a row's result does not depend on where in a tile it stands.
__global__ void __launch_bounds__(kSortThreads) sort_kernel(const __grid_constant__ Params p, int4* tiles, int32_t* order) {
    allow_next_kernel();
    wait_for_earlier_kernels();
    extern __shared__ int next[];  // of an adapter: its rows, then their next place
    __shared__ int sums[32][2];
    const int tid = threadIdx.x, lane = tid & 31, bins = p.adapters + 1;
    for (int i = tid; i < bins; i += kSortThreads) next[i] = 0;
    __syncthreads();
    // A batch of rows from `base` on: their adapters' counters, and each row's place among its adapter's.  (The lanes of
    // one adapter as one: rows of a request lie together.)
    int key[kSortBatch], place[kSortBatch];
    auto count_rows = [&](int64_t base) {
#pragma unroll
        for (int u = 0; u < kSortBatch; ++u) {
            const int64_t row = base + u * kSortThreads + tid;
            const int id = row < p.m ? p.ids[row] : 0;
            key[u] = row >= p.m ? -1 : id >= 0 && id < p.adapters ? id : p.adapters;
        }
#pragma unroll
        for (int u = 0; u < kSortBatch; ++u) {
            if (base + u * kSortThreads >= p.m) break;
            const uint32_t same = __match_any_sync(0xffffffffu, key[u]);
            const int leader = __ffs(same) - 1;
            int at = 0;
            if (key[u] >= 0 && lane == leader) at = atomicAdd(&next[key[u]], __popc(same));
            place[u] = __shfl_sync(0xffffffffu, at, leader) + __popc(same & ((1u << lane) - 1));
        }
    };
    constexpr int kBatchRows = kSortThreads * kSortBatch;
    for (int64_t base = 0; base < p.m; base += kBatchRows) count_rows(base);
    __syncthreads();
    // the starts, and the tiles: a thread to a part of the counters
    const int per = (bins + kSortThreads - 1) / kSortThreads, first = min(tid * per, bins), last = min(first + per, bins);
    int rows = 0, count = 0;
    for (int i = first; i < last; ++i) {
        rows += next[i];
        count += (next[i] + p.tile - 1) / p.tile;
    }
    int rows_to = rows, count_to = count;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, rows_to, i), b = __shfl_up_sync(0xffffffffu, count_to, i);
        if (lane >= i) rows_to += a, count_to += b;
    }
    if (lane == 31) sums[tid >> 5][0] = rows_to, sums[tid >> 5][1] = count_to;
    __syncthreads();
    if (tid < 32) {
        int a = sums[tid][0], b = sums[tid][1];
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) {
            const int c = __shfl_up_sync(0xffffffffu, a, i), d = __shfl_up_sync(0xffffffffu, b, i);
            if (lane >= i) a += c, b += d;
        }
        sums[tid][0] = a, sums[tid][1] = b;
    }
    __syncthreads();
    int start = rows_to - rows, tile = count_to - count;
    if (tid >= 32) start += sums[(tid >> 5) - 1][0], tile += sums[(tid >> 5) - 1][1];
    __syncthreads();
    for (int i = first; i < last; ++i) {
        const int n = next[i];
        if (i == p.adapters) sums[0][0] = tile, sums[0][1] = tile + (n + p.tile - 1) / p.tile;
        next[i] = start;
        for (int at = 0; at < n; at += p.tile)
            tiles[1 + tile++] = tile_of(i < p.adapters ? i : -1, start + at, min(p.tile, n - at));
        start += n;
    }
    __syncthreads();
    if (tid < 32) {
        const int parts = parts_of(sums[0][1], p.up_blocks, p.n);
        if (tid == 0) tiles[0] = make_int4(sums[0][0], sums[0][1], parts, 0);
    }
    // (a batch that is the only one is known already; else the places are counted again, from the starts)
    for (int64_t base = 0; base < p.m; base += kBatchRows) {
        const bool again = p.m > kBatchRows;
        if (again) count_rows(base);
#pragma unroll
        for (int u = 0; u < kSortBatch; ++u) {
            const int64_t row = base + u * kSortThreads + tid;
            if (row < p.m) order[again ? place[u] : next[key[u]] + place[u]] = static_cast<int>(row);
        }
    }
}

// The same of up to kHere rows by each CTA for itself, in the order of the rows (so that a cluster's CTAs agree): a row's
// place is the count of the rows that go before it.  All comparisons take every CTA's issue slots: 1 us in both launches
// for 64 rows, 2.5 for 128, 5 for 256.
constexpr int kHere = 128, kMaxHere = (1 << 22) - 1;  // adapters: an adapter and a row are one number

struct Sorted {
    int4 tiles[1 + kHere];
    int order[kHere];
    uint32_t begin[2][kHere / 32];  // the places that an adapter, and a tile, begins at
};

__device__ __forceinline__ void sort_here(Sorted& s, const Params& p) {
    int *keys = reinterpret_cast<int*>(s.tiles), *adapters = keys + kHere;  // (until the tiles are written)
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const bool on = t < p.m;  // (m <= kHere)
    int key = 0x7fffffff;
    if (on) {
        const int id = p.ids[t];
        key = (id >= 0 && id < p.adapters ? id : p.adapters) * kHere + t;
    }
    if (t < kHere) keys[t] = key;
    __syncthreads();
    if (on) {
        int place = 0;
#pragma unroll 4
        for (int i = 0; i < p.m; i += 4) {  // (those beyond the last row are above all)
            const int4 four = *reinterpret_cast<const int4*>(keys + i);
            place += (four.x < key) + (four.y < key) + (four.z < key) + (four.w < key);
        }
        s.order[place] = t;
        adapters[place] = key / kHere;
    }
    __syncthreads();
    const int adapter = on ? adapters[t] : 0;
    const uint32_t begin = __ballot_sync(0xffffffffu, on && (t == 0 || adapters[t - 1] != adapter));
    if (lane == 0 && t < kHere) s.begin[0][warp] = begin;
    __syncthreads();
    // the adapter's first place, and the next one's
    const uint32_t upto = 0xffffffffu >> (31 - lane);
    uint32_t low = begin & upto, high = begin & ~upto;
    int w = warp;
    while (on && low == 0 && w > 0) low = s.begin[0][--w];
    const int first = 32 * w + 31 - __clz(low);
    w = warp;
    while (high == 0 && w < kHere / 32 - 1) high = s.begin[0][++w];
    const int end = high ? 32 * w + __ffs(high) - 1 : p.m;
    const bool tile = on && ((t - first) & (p.tile - 1)) == 0;  // (32 or 64)
    const uint32_t tiles = __ballot_sync(0xffffffffu, tile);
    if (lane == 0 && t < kHere) s.begin[1][warp] = tiles;
    const int with = __syncthreads_count(tile && adapter < p.adapters);
    int all = 0, at = __popc(tiles & (upto >> 1));
#pragma unroll
    for (int i = 0; i < kHere / 32; ++i) {
        const int n = __popc(s.begin[1][i]);
        at += i < warp ? n : 0;
        all += n;
    }
    if (tile) s.tiles[1 + at] = tile_of(adapter < p.adapters ? adapter : -1, t, min(p.tile, end - t));
    if (warp == 0) {
        const int parts = parts_of(all, gridDim.x, p.n);
        if (lane == 0) s.tiles[0] = make_int4(with, all, parts, 0);
    }
    __syncthreads();
}

// Where a row ends inside eight elements: the first `columns` of them, zeros for the rest.  (Not inlined: it is wanted
// once in a while, and code that is not there need not be fetched.  With the ends in line a launch of a few blocks
// waited for instructions more than for memory.)
static __device__ __noinline__ uint4 load_cut(const uint16_t* at, int columns) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < columns) w[i >> 1] |= static_cast<uint32_t>(at[i]) << (i & 1) * 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
}
static __device__ __noinline__ void store_cut(uint16_t* at, uint4 v, int columns) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < columns) at[i] = static_cast<uint16_t>(w[i >> 1] >> (i & 1) * 16);
}

// Where the terms of rank j of a row of S are, of RS ranks a step of the product up to D (16, or 32 beyond 16 ranks):
// a lane's quarter of a step lies together, first terms and second terms.
template <int RS>
__device__ __forceinline__ int term_at(int j, int term) {
    return j / RS * 2 * RS + j % RS / (RS / 4) * (RS / 2) + term * (RS / 4) + j % (RS / 4);
}

// ---------------------------------------------------------------- a tile's rows by adapter

// Units of up to UNIT rows of one adapter.
struct Order {
    int id[kMaxTile];          // in order
    int row[kMaxTile];         // in order: rows of one adapter together, those without one last
    int start[kMaxTile + 1];   // the units' first places
    int units;
    int ends;                  // bit 0: the matrix's first row is in the tile, bit 1: its last
    __device__ __forceinline__ int adapter(int unit) const { return id[start[unit]]; }  // -1: none
};

// Tile `tile`, by all threads of a block: its first row (what o.row counts from) and how many it has.
template <int UNIT>
__device__ __forceinline__ int64_t make_order(Order& o, const Sorted& s, const Params& p, int tile, int& rows) {
    __shared__ int given[kMaxTile];
    __shared__ bool begins[kMaxTile];  // (in order) a unit
    const int t = threadIdx.x;
    if (p.here || p.tiles) {
        const int4 sorted = p.here ? s.tiles[1 + tile] : p.tiles[1 + tile];
        rows = sorted.z;
        int ends = 0;
        if (t < rows) {
            const int row = p.here ? s.order[sorted.y + t] : p.order[sorted.y + t];
            o.row[t] = row;
            o.id[t] = sorted.x;
            ends = (row == 0 ? 1 : 0) | (row == p.m - 1 ? 2 : 0);
        }
        const int units = (rows + UNIT - 1) / UNIT;
        if (t <= units) o.start[t] = min(t * UNIT, rows);
        const int any0 = __syncthreads_or(ends & 1), any1 = __syncthreads_or(ends & 2);
        if (t == 0) {
            o.units = units;
            o.ends = (any0 ? 1 : 0) | (any1 ? 2 : 0);
        }
        __syncthreads();
        return 0;
    }
    const int64_t row0 = static_cast<int64_t>(tile) * p.tile;
    rows = static_cast<int>(min(static_cast<int64_t>(p.tile), p.m - row0));
    if (t == 0) o.ends = (row0 == 0 ? 1 : 0) | (row0 + rows == p.m ? 2 : 0);
    int key = p.adapters, first = p.adapters;  // (without one: after all others)
    if (t < rows) {
        const int id = p.ids[row0 + t], id0 = p.ids[row0];
        if (id >= 0 && id < p.adapters) key = id;
        if (id0 >= 0 && id0 < p.adapters) first = id0;
        given[t] = key;
    }
    if (__syncthreads_and(key == first || t >= rows)) {  // (a prompt's rows: one adapter)
        const int units = (rows + UNIT - 1) / UNIT;
        if (t < rows) {
            o.row[t] = t;
            o.id[t] = key < p.adapters ? key : -1;
        }
        if (t <= units) o.start[t] = min(t * UNIT, rows);
        if (t == 0) o.units = units;
        __syncthreads();
        return row0;
    }
    if (t < rows) {
        int less = 0, same = 0;
#pragma unroll 8
        for (int i = 0; i < rows; ++i) {
            less += given[i] < key;
            same += given[i] == key && i < t;
        }
        o.row[less + same] = t;
        o.id[less + same] = key < p.adapters ? key : -1;
        begins[less + same] = same % UNIT == 0;
    }
    __syncthreads();
    if (t < 32) {
        int units = 0;
        for (int base = 0; base < rows; base += 32) {
            const int i = base + t;
            const bool one = i < rows && begins[i];
            const uint32_t on = __ballot_sync(0xffffffffu, one);
            if (one) o.start[units + __popc(on & ((1u << t) - 1))] = i;
            units += __popc(on);
        }
        if (t == 0) {
            o.start[units] = rows;
            o.units = units;
        }
    }
    __syncthreads();
    return row0;
}

// ---------------------------------------------------------------- down to the rank

// 16 MT ranks of one adapter with NT units of its rows, over the steps first, first + by, ...: the lane's sums, at `mine` in
// shared memory.
//
// Loads go straight to the fragments.  Each row's 64 bytes come from one warp, 512 contiguous bytes from the block's
// eight, and two blocks an SM have 70 to 80 KB on their way: 64 rows of 4096 columns a block and a cluster of two, of 8192
// rows (67 MB), take 21 us by ncu with caches cold (3.2 TB/s), 19 in a stream of calls.  A ring of steps in shared memory,
// filled by cp.async, took half as long again on rows that lay in L2.
template <int MT, int NT>
__device__ __forceinline__ void down_sums(float* mine, const Params& p, const Order& o, int64_t row0, int rank0, int unit0,
                                          int units, int first, int by) {
    constexpr int kOf = 2 * MT + NT, kUnroll = kOf <= 4 ? 4 : kOf < 8 ? 2 : 1;
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    // (ranks beyond the last are the last's, rows the unit's first's, units the last's: their sums are not used;
    // distances within a tile's rows and within an adapter's matrix are within 32 bits: the host sees to it)
    const uint16_t *a = p.a + o.adapter(unit0) * p.apart_a + 8 * q, *tile = p.x + row0 * p.ldx + 8 * q;
    uint32_t a_at[2 * MT], x[NT];
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) a_at[i] = min(rank0 + g + 8 * i, p.rank - 1) * static_cast<uint32_t>(p.lda);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int unit = unit0 + min(t, units - 1), place = o.start[unit] + g;
        x[t] = o.row[place < o.start[unit + 1] ? place : place - g] * static_cast<uint32_t>(p.ldx);
    }
    float c[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) c[m][t][i] = 0.f;
    constexpr int kSteps = kChain / 2;  // (two mma each)
    const int whole = p.k / kStep, chain = kSteps * by;
    const bool chains = whole - first > chain;
    for (int from = first; from < whole; from += chain) {
        const int to = min(whole, from + chain);
        for (int s = from; s < to; s += kUnroll * by) {
            uint4 u[kUnroll][2 * MT], v[kUnroll][NT];
#pragma unroll
            for (int j = 0; j < kUnroll; ++j) {  // (all loads at once; beyond the last step, it again)
                const int col = min(s + j * by, whole - 1) * kStep;
#pragma unroll
                for (int i = 0; i < 2 * MT; ++i) u[j][i] = *reinterpret_cast<const uint4*>(a + a_at[i] + col);
#pragma unroll
                for (int t = 0; t < NT; ++t)  // (up to 16 ranks X is read by one warp only)
                    v[j][t] = MT == 1 ? load_once(tile + x[t] + col) : *reinterpret_cast<const uint4*>(tile + x[t] + col);
            }
#pragma unroll
            for (int j = 0; j < kUnroll; ++j) {
                if (s + j * by >= to) continue;
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma_step(c[m][t], u[j][2 * m], u[j][2 * m + 1], v[j][t]);
            }
        }
        if (chains) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float& sum = mine[(m * NT + t) * 128 + i * 32];
                        sum = from == first ? c[m][t][i] : sum + c[m][t][i];
                        c[m][t][i] = 0.f;
                    }
        }
    }
    if (whole * kStep < p.k && first == 0) {
        const int col = whole * kStep, left = p.k - 8 * q - col;
        uint4 u[2 * MT];
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) u[i] = load_cut(a + a_at[i] + col, left);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint4 v = load_cut(tile + x[t] + col, left);
#pragma unroll
            for (int m = 0; m < MT; ++m) mma_step(c[m][t], u[2 * m], u[2 * m + 1], v);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float& sum = mine[(m * NT + t) * 128 + i * 32];
                sum = chains ? sum + c[m][t][i] : c[m][t][i];
            }
}

// A turn: `units` units of rows of one adapter (up to NT).  The cluster's CTAs share the columns, and in each CTA a team
// of warps 16 MT ranks and, again, the columns; the sums are joined over the warps, then over the CTAs, in the same
// order on every run.  `joined`: the warps' sums; `mine`: the CTA's, one of two places in turn, so that a turn has one
// barrier of the cluster.
template <int MT, int NT>
__device__ __forceinline__ void down_turn(const Params& p, const Order& o, float* joined, float* mine, int64_t row0, int rank,
                                          int unit0, int units) {
    constexpr int kOf = MT * NT * 128;  // sums of a warp
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sharing = kWarps / p.teams, team = warp / sharing, part = warp % sharing;
    down_sums<MT, NT>(joined + warp * kOf + lane, p, o, row0, team * 16 * MT, unit0, units, rank * sharing + part,
                      p.cluster * sharing);
    __syncthreads();
    for (int at = threadIdx.x; at < p.teams * kOf; at += kThreads) {
        const int its = at / kOf, in = at % kOf;
        float v = 0.f;
        for (int k = 0; k < sharing; ++k) v += joined[(its * sharing + k) * kOf + in];
        mine[at] = v;
    }
    cluster_sync();
    for (int at = rank * kThreads + threadIdx.x; at < p.teams * kOf; at += p.cluster * kThreads) {
        const int its = at / kOf, in = at % kOf;
        const int from = in & 31, i = in >> 5 & 3, t = (in >> 7) % NT, m = (in >> 7) / NT;
        const int j = (its * MT + m) * 16 + (from >> 2) + 8 * (i >> 1);
        if (t >= units || j >= p.ldlow) continue;
        const int place = o.start[unit0 + t] + 2 * (from & 3) + (i & 1);
        if (place >= o.start[unit0 + t + 1]) continue;
        float v = 0.f;
        for (int k = 0; k < p.cluster; ++k) {
            float other;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(other) : "r"(mapa_shared(smem_addr(mine + at), k)) : "memory");
            v += other;
        }
        uint16_t* to = p.low + (row0 + o.row[place]) * 2 * p.ldlow;
        constexpr int kStepRanks = MT == 1 ? 16 : 32;
        split(j < p.rank ? v * (p.scale ? p.scale[o.id[place]] : 1.f) : 0.f, to[term_at<kStepRanks>(j, 0)],
              to[term_at<kStepRanks>(j, 1)]);
    }
}

// Units of one adapter that a turn takes.
__host__ __device__ constexpr int turn_units(int mt) { return mt == 1 ? 8 : 4; }
constexpr int kSums = 8 * 128;  // of a warp in a turn, at most

// Dynamic shared memory: the warps' sums, and two places for the CTA's.
template <int MT>
__global__ void __launch_bounds__(kThreads, 2) down_kernel(const __grid_constant__ Params p) {
    allow_next_kernel();
    wait_for_earlier_kernels();
    __shared__ Order o;
    extern __shared__ __align__(16) float sums[];
    const int rank = blockIdx.x % p.cluster;
    constexpr int kMost = turn_units(MT);
    __shared__ int next_tile;  // (here for the registers: it is wanted once a tile)
    __shared__ Sorted sorted;
    if (p.here) sort_here(sorted, p);
    if (threadIdx.x == 0) next_tile = blockIdx.x / p.cluster;
    int turn = 0;
    for (;;) {
    int rows;
    __syncthreads();  // (the tile before has been read)
    const int tile = next_tile, clusters = gridDim.x / p.cluster;
    if (tile >= (p.here ? sorted.tiles[0].x : p.tiles ? p.tiles[0].x : clusters)) break;
    const int64_t row0 = make_order<8>(o, sorted, p, tile, rows);  // (by when all have read next_tile)
    if (threadIdx.x == 0) next_tile = tile + clusters;
    for (int unit = 0, n; unit < o.units && o.adapter(unit) >= 0; unit += n, turn ^= 1) {  // (those without are last)
        n = 1;
        while (n < kMost && unit + n < o.units && o.adapter(unit + n) == o.adapter(unit)) ++n;
        float* mine = sums + (kWarps + turn * p.teams) * kSums;
        if (n == 1) down_turn<MT, 1>(p, o, sums, mine, row0, rank, unit, n);
        else if (n == 2) down_turn<MT, 2>(p, o, sums, mine, row0, rank, unit, n);
        else if (MT == 2 || n <= 4) down_turn<MT, 4>(p, o, sums, mine, row0, rank, unit, n);
        else if constexpr (MT == 1) down_turn<MT, 8>(p, o, sums, mine, row0, rank, unit, n);
    }
    }
    cluster_sync();  // (the others may still read this CTA's sums)
}

// ---------------------------------------------------------------- up to D

// Words of a row of S in shared memory: the rows of a fragment's 16-byte loads are in different banks.
__host__ __device__ constexpr int low_words(int ldlow) { return ldlow <= 16 ? 16 : ldlow + 4; }

// A lane's words of a step of a row of B: RS / 4 elements.
template <int RS>
struct __align__(RS / 2) Words {
    uint32_t w[RS / 8];
};

// Those at `col` (zeros from `cols` on).  WHOLE: there are always so many (a load that may branch waits for the one
// before).
template <int RS, bool WHOLE>
__device__ __forceinline__ Words<RS> load_words(const uint16_t* row, int col, int cols) {
    if (WHOLE || col + RS / 4 <= cols) return *reinterpret_cast<const Words<RS>*>(row + col);
    Words<RS> v;
#pragma unroll
    for (int i = 0; i < RS / 8; ++i) {
        v.w[i] = col + 2 * i < cols ? row[col + 2 * i] : 0u;
        if (col + 2 * i + 1 < cols) v.w[i] |= static_cast<uint32_t>(row[col + 2 * i + 1]) << 16;
    }
    return v;
}

// Eight elements of two neighbouring 16-byte words, from the element `by` (0 .. 8) on.
__device__ __forceinline__ uint4 window(const uint4& a, const uint4& b, int by) {
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
    return by & 8 ? b : make_uint4(w[0], w[1], w[2], w[3]);
}

// Elements between the 16-byte boundary below p and p.
__device__ __forceinline__ int shift_of(const uint16_t* p) { return static_cast<int>(reinterpret_cast<uintptr_t>(p) >> 1) & 7; }

// A lane's eight columns of 32 in a row (8q .. 8q + 7, at `at`), on their way.  SHIFT: rows start anywhere; the two
// 16-byte words are loaded that hold them.
template <bool SHIFT>
struct Row8 {
    uint4 a, b;
    __device__ __forceinline__ void load(const uint16_t* at) {
        const uint16_t* from = SHIFT ? at - shift_of(at) : at;
        a = SHIFT ? *reinterpret_cast<const uint4*>(from) : load_once(from);
        if (SHIFT) b = *reinterpret_cast<const uint4*>(shift_of(at) ? from + 8 : from);
    }
    __device__ __forceinline__ uint4 get(const uint16_t* at, bool edge) const {
        return SHIFT && !edge ? window(a, b, shift_of(at)) : a;
    }
};

// A lane's eight columns of 32 in a row (8q .. 8q + 7, at `at`) written.  With rows that start anywhere a lane writes
// the 16-byte word that ends in its columns, with its neighbour's; the four lanes' first and last words are parts, in
// pieces of 8, 4 and 2 bytes. By all lanes of a warp; `on`: the lane's row is written.
template <bool SHIFT>
__device__ __forceinline__ void store_row8(uint16_t* at, const uint4& v, int q, bool on) {
    if (!SHIFT) {
        if (on) *reinterpret_cast<uint4*>(at) = v;
        return;
    }
    const uint4 before = make_uint4(__shfl_up_sync(0xffffffffu, v.x, 1), __shfl_up_sync(0xffffffffu, v.y, 1),
                                    __shfl_up_sync(0xffffffffu, v.z, 1), __shfl_up_sync(0xffffffffu, v.w, 1));
    if (!on) return;
    const int s = shift_of(at);
    const uint4 word = window(before, v, 8 - s);
    uint16_t* to = at - s;
    if (q > 0 || s == 0) {
        *reinterpret_cast<uint4*>(to) = word;
    } else {
        const int even = s + (s & 1);  // (elements s .. 7)
        if (s & 1) to[s] = static_cast<uint16_t>((s == 1 ? word.x : s == 3 ? word.y : s == 5 ? word.z : word.w) >> 16);
        if (even & 2) *reinterpret_cast<uint32_t*>(to + even) = even == 2 ? word.y : word.w;
        if (even <= 4) *reinterpret_cast<uint2*>(to + 4) = make_uint2(word.z, word.w);
    }
    if (q == 3 && s) {
        const uint4 rest = window(v, v, 8 - s);  // (elements 0 .. s - 1)
        uint16_t* end = to + 8;
        if (s & 4) *reinterpret_cast<uint2*>(end) = make_uint2(rest.x, rest.y);
        if (s & 2) *reinterpret_cast<uint32_t*>(end + (s & 4)) = s & 4 ? rest.z : rest.x;
        if (s & 1) end[s & 6] = static_cast<uint16_t>(s == 1 ? rest.x : s == 3 ? rest.y : s == 5 ? rest.z : rest.w);
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// A row of a unit, as the loop over columns wants it: what lies between the tile's first row and this one, in elements
// (the host keeps a tile's rows within 32 bits), and its place of S.
struct __align__(16) RowAt {
    uint32_t r, d, low;
    int on;  // else beyond the unit's last row, which stands in its place
};

// A CTA: a tile of rows, and a part of D's columns in blocks of 32, a warp each. The mma's columns are taken in an order
// in which a lane's sums are 8 neighbouring columns of a row: of a block's four mma tiles, column i of tile j is number
// 8 (i / 2) + 2 j + i % 2. Of a block a warp takes two units (16 rows) of one adapter at a time: their R, and B, are
// asked for at once, and B's fragments serve both. All that a row needs comes from shared memory in one load, since the
// blocks are short.
// RS: ranks of a step (of a lane's loads of 8 or 16 bytes); STEPS: steps of B in registers (0: the rank has more than
// two, and B is read step by step, after the first unit from L1).
// Dynamic shared memory: S [row in order][low_words].
//
// 8192 x 4096 of rank 16 (134 MB), rows of 12 requests, on a GB300: 31 us, 4.3 TB/s (0.64 of the copy bandwidth).  While
// all SMs are full it moves 5 TB/s; the rest is the start of a tile (1.5 us until its rows and S are there) and blocks
// that are not done together.  Left out for a measurement, the mma, S's loads and B's took 8 % together, R's loads 40 %,
// D's stores 25 %.  Four units at a time in twice the registers took as long, and so did R and B fetched four turns
// ahead to a ring in shared memory.  30 tiles of one or two rows with 14336 columns and rank 64: 16.5 us for 55 MB of B.
template <int RS, int STEPS, bool SHIFT>
__global__ void __launch_bounds__(kThreads, RS == 16 && !SHIFT ? 3 : 2) up_kernel(const __grid_constant__ Params p) {
    constexpr int kBatch = SHIFT && STEPS != 1 ? 1 : 2;  // (units at once: for the registers)
    allow_next_kernel();
    wait_for_earlier_kernels();
    __shared__ Order o;
    __shared__ RowAt rows_at[kMaxTile * 16];
    extern __shared__ __align__(16) uint32_t low[];
    __shared__ int next_item;  // (here for the registers: it is wanted once an item)
    __shared__ Sorted sorted;
    if (p.here) sort_here(sorted, p);
    __shared__ int items, parts;
    if (threadIdx.x == 0) {
        const int4 all = p.here ? sorted.tiles[0] : p.tiles ? p.tiles[0] : make_int4(0, 0, p.parts, 0);
        items = all.y > 0 ? all.y * all.z : gridDim.x;
        parts = all.z;
        next_item = blockIdx.x;
    }
    for (;;) {
    int rows;
    __syncthreads();  // (the item before has been read)
    const int item = next_item;
    if (item >= items) break;
    const int64_t row0 = make_order<16>(o, sorted, p, item / parts, rows);  // (by when all have read next_item)
    if (threadIdx.x == 0) next_item = item + gridDim.x;
    const int words = low_words(p.ldlow), chunks = p.ldlow / 4, units = o.units;
    for (int i = threadIdx.x; i < units * 16; i += kThreads) {
        const int end = o.start[i / 16 + 1], place = o.start[i / 16] + i % 16, at = min(place, end - 1);
        rows_at[i] = {o.row[at] * static_cast<uint32_t>(p.ldr), o.row[at] * static_cast<uint32_t>(p.ldd),
                      static_cast<uint32_t>(at * words), place < end};
    }
    for (int i = threadIdx.x; i < rows * chunks; i += kThreads) {
        const int place = i / chunks, j = i - place * chunks;
        if (o.id[place] >= 0)
            *reinterpret_cast<uint4*>(low + place * words + 4 * j) =
                *reinterpret_cast<const uint4*>(p.low + (row0 + o.row[place]) * 2 * p.ldlow + 8 * j);
    }
    __syncthreads();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    // (of sorted rows, whose distances are the matrix's, 0)
    const uint16_t* r_tile = p.r + row0 * p.ldr;
    uint16_t* d_tile = p.d + row0 * p.ldd;
    for (uint32_t at = (item % parts * kWarps + warp) * kColumns; at < static_cast<uint32_t>(p.n);
         at += static_cast<uint32_t>(parts) * kWarps * kColumns) {  // (twice N is within 32 bits)
        const int col0 = static_cast<int>(at), col = col0 + 8 * q;
        // Element by element: a block that is cut off, and, since rows that start anywhere are read in whole 16-byte
        // words, where those may begin before the matrix or end after it.
        const bool edge = col0 + kColumns > p.n ||
                          (SHIFT && ((col0 == 0 && (o.ends & 1)) || (col0 + kColumns + 8 > p.n && (o.ends & 2))));
        uint32_t b_at[4];  // (columns beyond the last are the last's; the host keeps 32 rows of B within 32 bits)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            b_at[j] = min(8 * (g >> 1) + 2 * j + (g & 1), p.n - 1 - col0) * static_cast<uint32_t>(p.ldb) + RS / 4 * q;
        for (int unit = 0, n; unit < units; unit += n) {
            const int adapter = o.adapter(unit);
            n = kBatch == 2 && unit + 1 < units && o.adapter(unit + 1) == adapter ? 2 : 1;
            const int here = 16 * unit + g;
            Row8<SHIFT> r[kBatch][2];
            auto load_r = [&](auto units_here) {
#pragma unroll
                for (int i = 0; i < decltype(units_here)::value; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) r[i][h].load(r_tile + rows_at[here + 16 * i + 8 * h].r + col);
            };
            if (p.r && !edge) {
                if (n == 2) load_r(std::integral_constant<int, kBatch>());
                else load_r(std::integral_constant<int, 1>());
            } else if (p.r) {
#pragma unroll
                for (int i = 0; i < 2 * kBatch; ++i)
                    if (i < 2 * n) r[i / 2][i % 2].a = load_cut(r_tile + rows_at[here + 8 * i].r + col, p.n - col);
            }
            const uint16_t* b = p.b + (max(adapter, 0) * p.apart_b + col0 * p.ldb);
            auto load_b = [&](Words<RS>(&to)[4], int k0) {
                if (p.rank == p.ldlow) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) to[j] = load_words<RS, true>(b + b_at[j], k0, p.rank);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) to[j] = load_words<RS, false>(b + b_at[j], k0, p.rank - RS / 4 * q);
                }
            };
            Words<RS> held[STEPS > 0 ? STEPS : 1][4];
            if (adapter >= 0) {
#pragma unroll
                for (int i = 0; i < STEPS; ++i) load_b(held[i], i * RS);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (i >= n) continue;
                const RowAt* row = rows_at + here + 16 * i;  // (and 8 on; read where they are wanted, for the registers)
                float c[4][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 u = p.r ? r[i][h].get(r_tile + row[8 * h].r + col, edge) : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        c[j][2 * h] = __uint_as_float(w[j] << 16);
                        c[j][2 * h + 1] = __uint_as_float(w[j] & 0xffff0000u);
                    }
                }
                if (adapter >= 0) {
                    auto add = [&](const Words<RS>(&u)[4], int k0) {
                        Words<RS> s[2][2];  // [row][term]
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const Words<RS>* from = reinterpret_cast<const Words<RS>*>(low + row[8 * h].low + k0 + RS / 4 * q);
                            s[h][0] = from[0], s[h][1] = from[1];
                        }
#pragma unroll
                        for (int term = 0; term < 2; ++term)
#pragma unroll
                            for (int w = 0; w < RS / 8; w += 2)
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    mma(c[j], s[0][term].w[w], s[1][term].w[w], s[0][term].w[w + 1], s[1][term].w[w + 1],
                                        u[j].w[w], u[j].w[w + 1]);
                    };
                    if (STEPS > 0) {
#pragma unroll
                        for (int k = 0; k < STEPS; ++k) add(held[k], k * RS);
                    } else {
#pragma unroll 2
                        for (int k0 = 0; k0 < p.ldlow; k0 += RS) {
                            Words<RS> u[4];
                            load_b(u, k0);
                            add(u, k0);
                        }
                    }
                }
                if (p.act) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int k = 0; k < 4; ++k) c[j][k] = activate(c[j][k], p.act);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = pack2(c[j][2 * h], c[j][2 * h + 1]);
                    uint16_t* to = d_tile + row[8 * h].d + col;
                    if (!edge) {
                        store_row8<SHIFT>(to, make_uint4(w[0], w[1], w[2], w[3]), q, row[8 * h].on);
                    } else if (row[8 * h].on) {
                        store_cut(to, make_uint4(w[0], w[1], w[2], w[3]), p.n - col);
                    }
                }
            }
        }
    }
    }
}

}  // namespace lora
}  // namespace gb
