// Device code of a whole mixture-of-experts layer for a few tokens:
//
//   logits = X G^T        the top k experts of a token, e_1 .. e_k, with their softmax weights w_j
//   D = R + sum_j w_j W2[e_j] ( silu(W1[e_j] x) * (W3[e_j] x) )
//
// Three launches: the router (a cluster to a token), the chosen experts' gated products, and their second
// products with the weighted sum.  Bound by the bytes of the chosen experts' matrices; each is read once for
// all the tokens that chose it (up to kPassTokens of them).
#pragma once

#include "skinny.cuh"

namespace gb {
namespace moe {

using namespace skinny;

constexpr int kMaxExperts = 1024, kMaxTop = 16;
constexpr int kPassTokens = 64;  // of a pass: a bit each in an expert's mask
constexpr int kPairs = kPassTokens * kMaxTop;
constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kRows = 16;        // weight rows of a tile

struct Params {
    const uint16_t* x;
    const uint16_t* router;
    const uint16_t* w[3];    // W1, W3 [experts, inner, d]; W2 [experts, d, inner]
    const uint16_t* r;       // or null
    uint16_t* out;
    int32_t* ids;            // [tokens, top]
    float* weights;          // [tokens, top]
    uint16_t* act[2];        // [pairs, ldact]: the inner activation's two terms
    int64_t ldx, ldrouter, ldr, ldo, ldact;
    int64_t ldw[3], expert[3];  // elements between rows, and between experts
    int tokens, d, inner, experts, top;
    int renormalize;
    int share;               // CTAs of a tile of D in the last launch
};

// ---------------------------------------------------------------- router

// The logits decide which expert a token goes to, and two of them may be nearly equal: they are summed as if
// in more than 32 bits.  A product of two bf16 is exact in fp32; each addition's rounding error is
// computed exactly (Knuth's two-sum) and summed beside it, and the lanes' sums are joined in 64 bits.
__device__ __forceinline__ void add_exact(float& s, float& err, float p) {
    const float t = __fadd_rn(s, p), b = __fsub_rn(t, s);
    err = __fadd_rn(err, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(p, b)));
    s = t;
}

__device__ __forceinline__ double exact_dot(const uint16_t* a, const uint16_t* b, int first, int last, int n, int lane) {
    float s = 0.f, err = 0.f;
    auto add = [&](const uint4& u, const uint4& v) {
        const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            add_exact(s, err, __fmul_rn(__uint_as_float(uw[i] << 16), __uint_as_float(vw[i] << 16)));
            add_exact(s, err, __fmul_rn(__uint_as_float(uw[i] & 0xffff0000u), __uint_as_float(vw[i] & 0xffff0000u)));
        }
    };
    constexpr int kBatch = 8;
    int col = first + 8 * lane;
    for (; col + 256 * (kBatch - 1) + 8 <= last; col += 256 * kBatch) {
        uint4 u[kBatch], v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            u[i] = *reinterpret_cast<const uint4*>(a + col + 256 * i);
            v[i] = load_once(b + col + 256 * i);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) add(u[i], v[i]);
    }
    for (; col < last; col += 256) add(load_edge(a, col, n), load_edge(b, col, n));
    // (of an infinite sum the error is none)
    double v = static_cast<double>(s) + (fabsf(s) <= 3.4028235e38f ? static_cast<double>(err) : 0.0);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) v += __shfl_xor_sync(0xffffffffu, v, i);
    return v;
}

// A logit as a whole number of the same order (comparisons in 64-bit floating point are slow): 0 for a NaN.
__device__ __forceinline__ uint64_t order_of(double v) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v + 0.0));  // (-0 is 0)
    return v != v ? 0 : u >> 63 ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ double value_of(uint64_t key) {
    return __longlong_as_double(static_cast<long long>(key >> 63 ? key & 0x7fffffffffffffffull : ~key));
}

// A cluster to a token: its warps share the experts and, where there are more warps than experts, `parts` of the
// columns; the cluster's first CTA chooses.  A logit that is NaN is chosen last, and makes the token's weights NaN.
// Latency is all it costs: 8 us for a token of 8 experts and 4096 columns, 13 for five of 64 and 2048 (ncu, caches cold);
// one warp to an expert, and choices by comparisons in 64-bit floating point, took longer.
__global__ void __launch_bounds__(kThreads) router_kernel(const __grid_constant__ Params p, int cluster, int parts) {
    allow_next_kernel();
    wait_for_earlier_kernels();
    __shared__ double logits[kMaxExperts];  // [expert][part]; then the logits' order
    const int token = blockIdx.x / cluster, rank = blockIdx.x % cluster;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint16_t* x = p.x + token * p.ldx;
    const uint32_t first = mapa_shared(smem_addr(logits), 0);
    const int span = (p.d + 256 * parts - 1) / (256 * parts) * 256;
    cluster_sync();  // (the first CTA runs: its shared memory may be written)
    for (int i = rank * kWarps + warp; i < p.experts * parts; i += cluster * kWarps) {
        const int e = i / parts, from = i % parts * span;
        const double v = exact_dot(x, p.router + e * p.ldrouter, from, min(from + span, p.d), p.d, lane);
        if (lane == 0) asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(first + 8 * i), "d"(v) : "memory");
    }
    cluster_sync();
    if (rank != 0 || warp != 0) return;

    uint64_t* keys = reinterpret_cast<uint64_t*>(logits);
    bool nan = false;
    for (int base = 0; base < p.experts; base += 32) {
        const int e = base + lane;
        uint64_t key = 0;
        if (e < p.experts) {
            double v = logits[e * parts];
            for (int i = 1; i < parts; ++i) v += logits[e * parts + i];
            key = order_of(v);
            nan |= key == 0;
        }
        __syncwarp();  // (parts > 1: at most 64 experts, whose sums another lane may still read)
        if (e < p.experts) keys[e] = key;
        __syncwarp();
    }
    nan = __any_sync(0xffffffffu, nan);
    uint32_t taken = 0;  // bit i: expert lane + 32 i
    double top = 0.0;
    float mine = 0.f, sum = 0.f;  // lane j has the j-th choice
    int my_id = 0;
    for (int j = 0; j < p.top; ++j) {
        uint64_t best = 0;
        int at = kMaxExperts;
        for (int e = lane, i = 0; e < p.experts; e += 32, ++i) {
            if (taken >> i & 1) continue;
            const uint64_t key = keys[e];
            if (key > best || at == kMaxExperts) {
                best = key;
                at = e;
            }
        }
        const uint32_t high = static_cast<uint32_t>(best >> 32), low = static_cast<uint32_t>(best);
        const uint32_t top_high = __reduce_max_sync(0xffffffffu, high);
        const uint32_t top_low = __reduce_max_sync(0xffffffffu, high == top_high ? low : 0u);
        at = __reduce_min_sync(0xffffffffu, high == top_high && low == top_low ? at : kMaxExperts);
        if ((at & 31) == lane) taken |= 1u << (at >> 5);
        const double v = value_of(static_cast<uint64_t>(top_high) << 32 | top_low);
        if (j == 0) top = v;
        if (lane == j) {
            mine = expf(static_cast<float>(v - top));
            my_id = at;
        }
    }
    if (p.renormalize) {
        sum = lane < p.top ? mine : 0.f;
    } else {
        for (int e = lane; e < p.experts; e += 32) sum += expf(static_cast<float>(value_of(keys[e]) - top));
    }
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
    if (lane < p.top) {
        const int64_t at = static_cast<int64_t>(token) * p.top + lane;
        p.ids[at] = my_id;
        p.weights[at] = nan ? __int_as_float(0x7fffffff) : mine / sum;
    }
}

// ---------------------------------------------------------------- who chose what

// The pass's pairs of a token and an expert, ordered by expert and then by token: pair c of expert e is at
// start[e] .., and is row c of the inner activation.
struct Lists {
    uint32_t mask[kMaxExperts][2];  // the tokens that chose the expert
    uint16_t start[kMaxExperts];
    uint16_t active[kMaxExperts];   // the experts that were chosen, in order
    uint16_t token[kPairs];
    int actives;
};

// By all threads of a block.  (Masks are joined by or: the order of the atomics does not matter.)
__device__ __forceinline__ void make_lists(Lists& l, const Params& p, float* pair_weight) {
    const int pairs = p.tokens * p.top, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < p.experts; e += kThreads) l.mask[e][0] = l.mask[e][1] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < pairs; i += kThreads) {
        const int t = i / p.top;
        atomicOr(&l.mask[p.ids[i]][t >> 5], 1u << (t & 31));
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        int before = 0, actives = 0;
        for (int base = 0; base < p.experts; base += 32) {
            const int e = base + lane;
            const int count = e < p.experts ? __popc(l.mask[e][0]) + __popc(l.mask[e][1]) : 0;
            int sum = count;
#pragma unroll
            for (int i = 1; i < 32; i <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, sum, i);
                if (lane >= i) sum += v;
            }
            const uint32_t on = __ballot_sync(0xffffffffu, count > 0);
            if (e < p.experts) l.start[e] = static_cast<uint16_t>(before + sum - count);
            if (count > 0) l.active[actives + __popc(on & ((1u << lane) - 1))] = static_cast<uint16_t>(e);
            before += __shfl_sync(0xffffffffu, sum, 31);
            actives += __popc(on);
        }
        if (lane == 0) l.actives = actives;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < pairs; i += kThreads) {
        const int t = i / p.top, e = p.ids[i];
        const uint32_t below = (1u << (t & 31)) - 1;
        const int at = l.start[e] + (t < 32 ? __popc(l.mask[e][0] & below) : __popc(l.mask[e][0]) + __popc(l.mask[e][1] & below));
        l.token[at] = static_cast<uint16_t>(t);
        if (pair_weight) pair_weight[at] = p.weights[i];
    }
    __syncthreads();
}

__device__ __forceinline__ int count_of(const Lists& l, int e) { return __popc(l.mask[e][0]) + __popc(l.mask[e][1]); }

// ---------------------------------------------------------------- the gated products

// A unit is 16 rows of W1 and of W3 of one expert, with up to 8 NT of its tokens; the block's warps share the columns a
// step apart (512 contiguous bytes of a row at a time) and join their sums in shared memory, while the SM's other block
// loads.  One token, 2 of 8 experts of 4096 x 14336 (470 MB): 71 us, 6.6 TB/s on a GB300 (0.98 of the copy bandwidth);
// 26 experts of 2048 x 1408 for five tokens (300 MB) 48 us, 6.2 TB/s.  Four steps on their way in 128 registers: three
// or four blocks an SM with two or one were 15 to 40 % slower, one block with eight 5 to 15 %.
template <int NT>
__device__ __forceinline__ void up_unit(const Params& p, const Lists& l, float* joined, int expert, int row0, int pair0, int pairs) {
    constexpr int kUnroll = NT == 1 ? 4 : 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    // (rows beyond the last are the last's, tokens the first's: their sums are not used)
    const uint16_t* w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = p.w[i >> 1] + expert * p.expert[i >> 1] + min(row0 + g + 8 * (i & 1), p.inner - 1) * p.ldw[i >> 1];
    const uint16_t* x[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) x[t] = p.x + l.token[pair0 + (8 * t + g < pairs ? 8 * t + g : 0)] * p.ldx;
    float c[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) c[m][t][i] = 0.f;

    constexpr int kSteps = kChain / 2;  // (of a warp: two mma each)
    const int steps = p.d / kStep;
    const bool chains = steps > kWarps * kSteps;
    float* mine = joined + warp * 2 * NT * 128 + lane;  // [matrix][tokens][i][lane]
    if (chains) __syncthreads();  // (the unit before has been read)
    for (int from = warp; from < steps; from += kWarps * kSteps) {
        const int to = min(steps, from + kWarps * kSteps);
        for (int s = from; s < to; s += kUnroll * kWarps) {
            uint4 a[kUnroll][4], b[kUnroll][NT];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {  // (all loads at once; beyond the last step, it again)
                const int col = min(s + u * kWarps, steps - 1) * kStep + 8 * q;
#pragma unroll
                for (int i = 0; i < 4; ++i) a[u][i] = load_once(w[i] + col);
#pragma unroll
                for (int t = 0; t < NT; ++t) b[u][t] = *reinterpret_cast<const uint4*>(x[t] + col);
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (s + u * kWarps >= to) continue;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    mma_step(c[0][t], a[u][0], a[u][1], b[u][t]);
                    mma_step(c[1][t], a[u][2], a[u][3], b[u][t]);
                }
            }
        }
        if (chains) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float& sum = mine[((m * NT + t) * 4 + i) * 32];
                        sum = from == warp ? c[m][t][i] : sum + c[m][t][i];
                        c[m][t][i] = 0.f;
                    }
        }
    }
    if (steps * kStep < p.d && warp == 0) {
        const int col = steps * kStep + 8 * q;
        uint4 a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = load_edge(w[i], col, p.d);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint4 b = load_edge(x[t], col, p.d);
            mma_step(c[0][t], a[0], a[1], b);
            mma_step(c[1][t], a[2], a[3], b);
        }
    }
    if (!chains) __syncthreads();  // (the unit before has been read)
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float& sum = mine[((m * NT + t) * 4 + i) * 32];
                sum = chains ? sum + c[m][t][i] : c[m][t][i];
            }
    __syncthreads();
    for (int at = threadIdx.x; at < NT * 128; at += kThreads) {
        float gate = 0.f, up = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            gate += joined[k * 2 * NT * 128 + at];
            up += joined[(k * 2 + 1) * NT * 128 + at];
        }
        const int from = at & 31, i = at >> 5 & 3, t = at >> 7;
        const int row = row0 + (from >> 2) + 8 * (i >> 1), pair = 8 * t + 2 * (from & 3) + (i & 1);
        if (row < p.inner && pair < pairs) {
            const int64_t to = (pair0 + pair) * p.ldact + row;
            split(silu(gate) * up, p.act[0][to], p.act[1][to]);
        }
    }
}

__global__ void __launch_bounds__(kThreads, 2) up_kernel(const __grid_constant__ Params p) {
    allow_next_kernel();
    wait_for_earlier_kernels();
    __shared__ Lists l;
    __shared__ float joined[kWarps * 2 * 4 * 128];
    make_lists(l, p, nullptr);
    const int tiles = (p.inner + kRows - 1) / kRows, units = l.actives * tiles;
    for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int a = unit / tiles, row0 = (unit - a * tiles) * kRows, e = l.active[a], pairs = count_of(l, e);
        for (int at = 0; at < pairs; at += 32) {
            const int n = min(pairs - at, 32), pair0 = l.start[e] + at;
            if (n <= 8) up_unit<1>(p, l, joined, e, row0, pair0, n);
            else if (n <= 16) up_unit<2>(p, l, joined, e, row0, pair0, n);
            else up_unit<4>(p, l, joined, e, row0, pair0, n);
        }
    }
}

// ---------------------------------------------------------------- the second products and the weighted sum

// A part of one expert's product with up to 8 NT of its pairs, steps first .. last - 1 of its columns, added to
// the warp's sums y[token][row].
template <int NT>
__device__ __forceinline__ void down_part(const Params& p, const Lists& l, const float* pair_weight, float* y, int expert,
                                          int row0, int pair0, int pairs, int first, int last) {
    constexpr int kUnroll = NT <= 2 ? 4 : 2;
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const uint16_t* w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) w[i] = p.w[2] + expert * p.expert[2] + min(row0 + g + 8 * i, p.d - 1) * p.ldw[2];
    int64_t x[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) x[t] = (pair0 + (8 * t + g < pairs ? 8 * t + g : 0)) * p.ldact;
    float c[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[t][i] = 0.f;
    static_assert(4 * kUnroll <= kChain);  // (what is loaded at once is a chain; ends that are looked for took more registers)
    float total[NT][4] = {};
    const int whole = min(last, p.inner / kStep);
    for (int s = first; s < whole; s += kUnroll) {
        uint4 a[kUnroll][2], b[kUnroll][NT][2];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {  // (all loads at once; beyond the last step, it again)
            const int col = min(s + u, whole - 1) * kStep + 8 * q;
#pragma unroll
            for (int i = 0; i < 2; ++i) a[u][i] = load_once(w[i] + col);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) b[u][t][i] = *reinterpret_cast<const uint4*>(p.act[i] + x[t] + col);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (s + u >= whole) continue;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) mma_step(c[t], a[u][0], a[u][1], b[u][t][i]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) total[t][i] += c[t][i], c[t][i] = 0.f;
    }
    if (whole < last) {
        const int col = whole * kStep + 8 * q;
        uint4 a[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) a[i] = load_edge(w[i], col, p.inner);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) mma_step(c[t], a[0], a[1], load_edge(p.act[i] + x[t], col, p.inner));
    }
    __syncwarp();  // (the part before has been added by other lanes)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int pair = 8 * t + 2 * q + (i & 1);
            if (pair >= pairs) continue;
            float* to = y + l.token[pair0 + pair] * kRows + g + 8 * (i >> 1);
            *to = fmaf(pair_weight[pair0 + pair], total[t][i] + c[t][i], *to);
        }
}

// A cluster to 16 columns of D; the sums of its CTAs' warps are joined in the same order on every run. One token, 2 of 8
// experts of 14336 x 4096 (235 MB): 42 us, 5.6 TB/s on a GB300 (0.83 of the copy bandwidth); 26 experts of 1408 x 2048
// (150 MB) 31 us, 4.8 TB/s: lists, the first loads of each expert in a warp's part and the join are 10 us.
// Dynamic shared memory: the warps' sums [warp][token][16].
__global__ void __launch_bounds__(kThreads, 2) down_kernel(const __grid_constant__ Params p) {
    allow_next_kernel();
    wait_for_earlier_kernels();
    __shared__ Lists l;
    __shared__ float pair_weight[kPairs];
    extern __shared__ float sums[];
    const int outputs = p.tokens * kRows;
    for (int i = threadIdx.x; i < kWarps * outputs; i += kThreads) sums[i] = 0.f;
    make_lists(l, p, pair_weight);
    const int cluster = p.share, rank = blockIdx.x % cluster, row0 = blockIdx.x / cluster * kRows;
    const int warp = threadIdx.x >> 5, steps = (p.inner + kStep - 1) / kStep;
    // The steps of all chosen experts, one after the other, shared out evenly to the cluster's warps.  (Warps that take
    // an expert's steps in turn, so that a block reads 512 contiguous bytes of a row at a time, took 3 to 10 % longer:
    // more experts a warp, and a wait for the first loads of each.)
    const int64_t all = static_cast<int64_t>(l.actives) * steps;
    const int shares = cluster * kWarps, share = rank * kWarps + warp;
    int64_t at = all * share / shares;
    const int64_t end = all * (share + 1) / shares;
    float* y = sums + warp * outputs;
    while (at < end) {
        const int a = static_cast<int>(at / steps), first = static_cast<int>(at - static_cast<int64_t>(a) * steps);
        const int last = static_cast<int>(min(static_cast<int64_t>(steps), first + end - at)), e = l.active[a];
        const int pairs = count_of(l, e);
        for (int done = 0; done < pairs; done += 32) {
            const int n = min(pairs - done, 32), pair0 = l.start[e] + done;
            if (n <= 8) down_part<1>(p, l, pair_weight, y, e, row0, pair0, n, first, last);
            else if (n <= 16) down_part<2>(p, l, pair_weight, y, e, row0, pair0, n, first, last);
            else down_part<4>(p, l, pair_weight, y, e, row0, pair0, n, first, last);
        }
        at += last - first;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < outputs; i += kThreads) {
        float v = sums[i];
#pragma unroll
        for (int k = 1; k < kWarps; ++k) v += sums[k * outputs + i];
        sums[i] = v;
    }
    cluster_sync();
    // (the rank again, as it is wanted: held since the start it was one register too many)
    for (int i = cluster_ctarank() * kThreads + threadIdx.x; i < outputs; i += cluster * kThreads) {
        const int token = i / kRows, col = row0 + i % kRows;
        float v = 0.f;
        for (int k = 0; k < cluster; ++k) {
            float part;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(part) : "r"(mapa_shared(smem_addr(sums + i), k)) : "memory");
            v += part;
        }
        if (col < p.d) {
            if (p.r) v += bf16_value(p.r[token * p.ldr + col]);
            p.out[token * p.ldo + col] = bf16_bits(v);
        }
    }
    cluster_sync();  // (the others may still read this CTA's sums)
}

}  // namespace moe
}  // namespace gb
