// C ABI of the products with 4-bit weights: argument checks, the plan and the launch of the
// kernel in w4_kernel.cuh.
#include <algorithm>
#include <atomic>
#include <cinttypes>
#include <cstring>

#include "host.h"
#include "w4_kernel.cuh"

namespace {

using namespace gb::host;
using gb::w4::kRows;
using gb::w4::kUnit;
using gb::w4::Params;

struct Weights {
    const char* name;
    const void* q;
    int64_t ldq;
    const void* s;
    int64_t lds;
    const void* z;
    int64_t ldz;
};

struct Problem {
    const void* x;
    int64_t ldx;
    int x_type;
    const float* x_scale;
    int64_t ldxs;
    Weights w[2];
    int group;
    const void* bias;
    const void* r;
    int64_t ldr;
    int act;
    void* d;
    int64_t ldd;
    int64_t m, n, k;
    bool gated;
};

gb_status_t validate(const Problem& pr) {
    if (pr.m < 0 || pr.n < 0 || pr.k < 0)
        return fail(GB_ERR_INVALID_ARG, "negative size M=%" PRId64 " N=%" PRId64 " K=%" PRId64, pr.m, pr.n, pr.k);
    if (pr.m > kMaxDim || pr.n > kMaxDim || pr.k > kMaxDim)
        return fail(GB_ERR_UNSUPPORTED, "sizes must be below 2^31 (M=%" PRId64 " N=%" PRId64 " K=%" PRId64 ")", pr.m,
                    pr.n, pr.k);
    if (pr.act < GB_ACT_NONE || pr.act > GB_ACT_RELU) return fail(GB_ERR_INVALID_ARG, "unknown activation %d", pr.act);
    if (pr.group != 32 && pr.group != 64 && pr.group != 128)
        return fail(GB_ERR_INVALID_ARG, "group=%d: 32, 64 or 128 columns", pr.group);
    if (pr.x_type < GB_X_BF16 || pr.x_type > GB_X_E4M3_GROUP_SCALE)
        return fail(GB_ERR_INVALID_ARG, "unknown type of X %d", pr.x_type);
    if (pr.m == 0 || pr.n == 0) return GB_OK;
    const int64_t groups = ceil_div(pr.k, pr.group);
    if (!pr.d) return fail(GB_ERR_INVALID_ARG, "D is null");
    if (pr.ldd < pr.n) return fail(GB_ERR_INVALID_ARG, "ldd=%" PRId64 " < N=%" PRId64, pr.ldd, pr.n);
    if (pr.r && pr.ldr < pr.n) return fail(GB_ERR_INVALID_ARG, "ldr=%" PRId64 " < N=%" PRId64, pr.ldr, pr.n);
    if (!aligned_to(pr.d, 2) || !aligned_to(pr.r, 2) || !aligned_to(pr.bias, 2))
        return fail(GB_ERR_UNSUPPORTED, "D, R and bias must be 2-byte aligned");
    if (pr.k == 0) return GB_OK;
    if (pr.k % 32) return fail(GB_ERR_UNSUPPORTED, "K=%" PRId64 " must be a multiple of 32", pr.k);
    if (!pr.x) return fail(GB_ERR_INVALID_ARG, "X is null");
    if (pr.ldx < pr.k) return fail(GB_ERR_INVALID_ARG, "ldx=%" PRId64 " < K=%" PRId64, pr.ldx, pr.k);
    if (pr.x_type == GB_X_BF16 && !aligned_to(pr.x, 2)) return fail(GB_ERR_UNSUPPORTED, "X must be 2-byte aligned");
    if (pr.x_type != GB_X_BF16) {
        const int64_t scales = pr.x_type == GB_X_E4M3_GROUP_SCALE ? ceil_div(pr.k, 128) : 1;
        if (!pr.x_scale) return fail(GB_ERR_INVALID_ARG, "x_scale is null");
        if (pr.ldxs < scales) return fail(GB_ERR_INVALID_ARG, "ldxs=%" PRId64 " < %" PRId64 " scales a row", pr.ldxs, scales);
        if (!aligned_to(pr.x_scale, 4)) return fail(GB_ERR_UNSUPPORTED, "x_scale must be 4-byte aligned");
    }
    for (int i = 0; i < (pr.gated ? 2 : 1); ++i) {
        const Weights& w = pr.w[i];
        if (!w.q || !w.s) return fail(GB_ERR_INVALID_ARG, "%s%s is null", w.name, w.q ? "'s scales" : "");
        if (w.ldq < pr.k / 2)
            return fail(GB_ERR_INVALID_ARG, "leading dimension %" PRId64 " of %s is below its %" PRId64 " bytes a row", w.ldq,
                        w.name, pr.k / 2);
        if (w.lds < groups || (w.z && w.ldz < groups))
            return fail(GB_ERR_INVALID_ARG, "leading dimension of %s's scales or zeros is below its %" PRId64 " groups",
                        w.name, groups);
        if (!aligned_to(w.q, 16) || (pr.n > 1 && w.ldq % 16))  // (one row has no next one)
            return fail(GB_ERR_UNSUPPORTED, "%s: base address and leading dimension must be multiples of 16 bytes", w.name);
        if (!aligned_to(w.s, 2)) return fail(GB_ERR_UNSUPPORTED, "%s's scales must be 2-byte aligned", w.name);
    }
    return GB_OK;
}

struct Plan {
    int tokens;     // of a pass
    int cluster;    // CTAs that share a row tile's columns
    int clusters;   // at once
    int k_warps;    // warps of a CTA that share them
    int warps;
    int slice_units;
    size_t smem;
};

template <int G, int NT, bool GATED, int X>
gb_status_t launch(const Params& prm, const Plan& pl, int dev, const DeviceInfo& info, cudaStream_t stream) {
    static std::atomic<bool> ready[64];  // (two threads may both set the attribute: to the same value)
    auto kern = gb::w4::w4_kernel<G, NT, GATED, X>;
    cudaError_t e;
    if (!ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(info.smem_optin));
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
        ready[dev].store(true, std::memory_order_release);
    }
    const int64_t groups = ceil_div(prm.tiles, pl.warps / pl.k_warps);
    const int64_t clusters = std::min<int64_t>(groups, pl.clusters);
    const dim3 grid(static_cast<unsigned>(clusters * pl.cluster), static_cast<unsigned>(ceil_div(prm.m, pl.tokens)));
    const gb_status_t st = Launch(grid, 32 * pl.warps, pl.smem, stream, pl.cluster)("w4 kernel launch", kern, prm);
    if (st != GB_OK) return st;
    note_plan("kernel=w4 group=%lld tokens=%lld cluster=%lld warps=%lld k_warps=%lld clusters=%lld", G, pl.tokens, pl.cluster,
              pl.warps, pl.k_warps, clusters);
    return GB_OK;
}

template <int G, int NT, bool GATED>
gb_status_t launch_x(const Params& prm, const Plan& pl, int dev, const DeviceInfo& info, cudaStream_t stream) {
    if (prm.x_type == GB_X_BF16) return launch<G, NT, GATED, gb::w4::kXBf16>(prm, pl, dev, info, stream);
    if (prm.x_type == GB_X_E4M3_ROW_SCALE) return launch<G, NT, GATED, gb::w4::kXRowScale>(prm, pl, dev, info, stream);
    return launch<G, NT, GATED, gb::w4::kXGroupScale>(prm, pl, dev, info, stream);
}

template <int G, bool GATED>
gb_status_t launch_nt(const Params& prm, const Plan& pl, int dev, const DeviceInfo& info, cudaStream_t stream) {
    return pl.tokens <= 8 ? launch_x<G, 1, GATED>(prm, pl, dev, info, stream)
                          : launch_x<G, 2, GATED>(prm, pl, dev, info, stream);
}

template <bool GATED>
gb_status_t launch_g(const Params& prm, const Plan& pl, int group, int dev, const DeviceInfo& info, cudaStream_t stream) {
    if (group == 32) return launch_nt<32, GATED>(prm, pl, dev, info, stream);
    if (group == 64) return launch_nt<64, GATED>(prm, pl, dev, info, stream);
    return launch_nt<128, GATED>(prm, pl, dev, info, stream);
}

// mma tiles of eight tokens that a pass holds
int tiles_of(int tokens) { return tokens <= 8 ? 1 : 2; }

// tokens for which a CTA keeps the sums, times the CTAs that the tokens are shared out to (as the
// kernel does: the rows first, two or four octets of them, then the tokens)
int share_tokens(int tokens, int cluster) {
    const int by_token = std::max(1, cluster / 2);  // (at most)
    return static_cast<int>(ceil_div(tokens, by_token)) * by_token;
}

size_t smem_of(int slice_units, int tokens, int warps, int group, int cluster, bool step_scale) {
    const size_t nt = tiles_of(tokens), units = slice_units;
    return static_cast<size_t>(warps) * gb::w4::kUnitBytes +                        // slots
           units * (kUnit / 8) * tokens * 16 +                                    // x
           ((step_scale ? units * (kUnit / gb::w4::kStep) : 1) + units * (kUnit / group)) * 8 * nt * 4 +  // its scales and sums
           static_cast<size_t>(2) * warps * share_tokens(tokens, cluster) * kRows * 4 +  // the warps' sums
           static_cast<size_t>(warps) * (kUnit / group) * 128;                      // their units' scales
}

// Clusters of `cluster` CTAs that run at once, one CTA an SM (the GPU's partitions need not hold a
// whole number of them).
gb_status_t clusters_at_once(int cluster, int dev, const DeviceInfo& info, int* out) {
    static std::atomic<int> known[64][4];
    std::atomic<int>& slot = known[dev][cluster == 1 ? 0 : cluster == 2 ? 1 : cluster == 4 ? 2 : 3];
    int n = cluster == 1 ? info.sms : slot.load(std::memory_order_relaxed);
    if (n == 0) {
        auto kern = gb::w4::w4_kernel<128, 1, false, gb::w4::kXBf16>;
        cudaError_t e =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(info.smem_optin));
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = cluster;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(info.sms / cluster * cluster, 1, 1);
        cfg.blockDim = dim3(32 * gb::w4::warps_of(128, 1), 1, 1);
        cfg.dynamicSmemBytes = info.smem_optin;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if ((e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg)) != cudaSuccess)
            return cuda_fail(e, "cudaOccupancyMaxActiveClusters");
        n = std::max(1, n);
        slot.store(n, std::memory_order_relaxed);
    }
    *out = n;
    return GB_OK;
}

// The plan of least time by a model fitted to measured plans (GB300, microseconds): a unit takes all
// of an SM's warps together `unit`, each round's join 1.1, or 1.4 over more than two CTAs, and
// x's layout 0.45 for each chunk of a thread, half of that where no largest value is looked for.
// (A round: every team takes one row tile.  Passes of tokens run side by side.)
gb_status_t make_plan(const Problem& pr, int64_t tiles, int dev, const DeviceInfo& info, const W4Override& want,
                      Plan* out) {
    const int units = std::max(1, static_cast<int>(ceil_div(pr.k, kUnit)));
    double best = 0.0;
    int tokens = static_cast<int>(std::min<int64_t>(pr.m, gb::w4::kMaxTokens));
    for (bool last = false; !last; tokens = (tokens + 1) / 2) {
        const int nt = tiles_of(tokens), warps = gb::w4::warps_of(pr.group, nt);
        const int64_t passes = ceil_div(pr.m, tokens);
        const double unit = nt == 1 ? (pr.group == 128 ? 1.5 : pr.group == 64 ? 1.6 : 1.9)
                                    : (pr.group == 128 ? 1.85 : pr.group == 64 ? 1.7 : 2.0);
        for (int cluster = 1; cluster <= 8 && (cluster <= units || want.cluster); cluster *= 2) {
            if (want.cluster && cluster != want.cluster) continue;
            const int slice = static_cast<int>(ceil_div(units, cluster));
            const size_t smem = smem_of(slice, tokens, warps, pr.group, cluster, pr.x_type != GB_X_E4M3_ROW_SCALE);
            if (smem > info.smem_optin) continue;
            int at_once = 0;
            const gb_status_t st = clusters_at_once(cluster, dev, info, &at_once);
            if (st != GB_OK) return st;
            const int64_t clusters = std::max<int64_t>(1, at_once / passes);  // of a pass
            const double chunks = ceil_div(static_cast<int64_t>(slice) * (kUnit / gb::w4::kStep) * tokens, 2 * warps);
            for (int k_warps = 1; k_warps <= warps; ++k_warps) {
                if (warps % k_warps || (want.k_warps && k_warps != want.k_warps)) continue;
                const int64_t rounds = ceil_div(ceil_div(tiles, warps / k_warps), clusters) * ceil_div(passes, at_once);
                const double time = rounds * (ceil_div(slice, k_warps) * unit + (cluster > 2 ? 1.4 : 1.1)) +
                                    chunks * (pr.x_type == GB_X_BF16 ? 0.45 : 0.22);
                if (best == 0.0 || time < best) {
                    best = time;
                    *out = Plan{tokens, cluster, static_cast<int>(clusters), k_warps, warps, slice, smem};
                }
                if (k_warps >= slice && !want.k_warps) break;
            }
        }
        // (as many tokens in a pass as there are, or half of them, or as few as x has room for)
        last = tokens == 1 || (best != 0.0 && 2 * tokens <= std::min<int64_t>(pr.m, gb::w4::kMaxTokens));
    }
    if (best == 0.0)
        return want.cluster || want.k_warps
                   ? fail(GB_ERR_UNSUPPORTED, "no plan has the configured w4_cluster and w4_k_warps")
                   : fail(GB_ERR_UNSUPPORTED, "K=%" PRId64 " is too large", pr.k);
    return GB_OK;
}

gb_status_t run(const Problem& pr, void* stream) {
    gb_status_t st = validate(pr);
    if (st != GB_OK) return st;
    if (pr.m == 0 || pr.n == 0) {
        note_empty();
        return GB_OK;
    }
    int dev = 0;
    DeviceInfo info;
    if ((st = device_info(&dev, &info)) != GB_OK) return st;

    const int out_rows = pr.gated ? kRows / 2 : kRows;
    const int64_t tiles = ceil_div(pr.n, out_rows);
    // (the last plans of the thread, by what a plan depends on: making one takes microseconds)
    struct Known {
        int64_t m = -1, n, k;
        int group, x_type, gated, dev, cluster, k_warps;
        Plan plan;
    };
    static thread_local Known known[8];
    static thread_local int turn = 0;
    const W4Override want = w4_override();
    Plan pl{};
    for (const Known& e : known)
        if (e.m == pr.m && e.n == pr.n && e.k == pr.k && e.group == pr.group && e.x_type == pr.x_type &&
            e.gated == pr.gated && e.dev == dev && e.cluster == want.cluster && e.k_warps == want.k_warps)
            pl = e.plan;
    if (pl.warps == 0) {
        if ((st = make_plan(pr, tiles, dev, info, want, &pl)) != GB_OK) return st;
        known[turn] = Known{pr.m, pr.n, pr.k, pr.group, pr.x_type, pr.gated, dev, want.cluster, want.k_warps, pl};
        turn = (turn + 1) % 8;
    }

    Params prm;
    memset(&prm, 0, sizeof prm);
    prm.ldx = pr.ldx;
    prm.ldxs = pr.ldxs;
    for (int i = 0; i < 2; ++i) {
        const Weights& w = pr.w[pr.gated ? i : 0];
        prm.q[i] = static_cast<const uint8_t*>(w.q);
        prm.s[i] = static_cast<const uint16_t*>(w.s);
        prm.z[i] = static_cast<const uint8_t*>(w.z);
        prm.ldq[i] = w.ldq;
        prm.lds[i] = w.lds;
        prm.ldz[i] = w.ldz;
    }
    const int64_t unit_groups = kUnit / pr.group;
    prm.wide_scales = 1;
    for (int i = 0; i < (pr.gated ? 2 : 1); ++i) {
        const Weights& w = pr.w[i];
        if (!aligned_to(w.s, 2 * unit_groups) || w.lds % unit_groups ||
            (w.z && (!aligned_to(w.z, unit_groups) || w.ldz % unit_groups)))
            prm.wide_scales = 0;
    }
    prm.bias = static_cast<const uint16_t*>(pr.bias);
    prm.ldr = pr.ldr;
    prm.ldd = pr.ldd;
    prm.n = static_cast<int>(pr.n);
    prm.k = static_cast<int>(pr.k);
    prm.act = pr.act;
    prm.x_type = pr.x_type;
    prm.tiles = static_cast<int>(tiles);
    prm.slice_units = pl.slice_units;
    prm.k_warps = pl.k_warps;
    prm.tokens = pl.tokens;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    // a launch has at most 65535 passes
    const int64_t most = int64_t(65535) * pl.tokens, x_bytes = pr.x_type == GB_X_BF16 ? 2 : 1;
    for (int64_t at = 0; at < pr.m && st == GB_OK; at += most) {
        prm.m = static_cast<int>(std::min(pr.m - at, most));
        prm.x = static_cast<const uint8_t*>(pr.x) + at * pr.ldx * x_bytes;
        prm.x_scale = pr.x_scale ? pr.x_scale + at * pr.ldxs : nullptr;
        prm.r = pr.r ? static_cast<const uint16_t*>(pr.r) + at * pr.ldr : nullptr;
        prm.d = static_cast<uint16_t*>(pr.d) + at * pr.ldd;
        st = pr.gated ? launch_g<true>(prm, pl, pr.group, dev, info, s) : launch_g<false>(prm, pl, pr.group, dev, info, s);
    }
    return st;
}

}  // namespace

extern "C" {

gb_status_t gb_gemm_linear_w4(const void* X, int64_t ldx, int x_type, const float* x_scale, int64_t ldxs,
                              const void* Wq, int64_t ldq, const void* scales, int64_t lds, const void* zeros,
                              int64_t ldz, int group, const void* bias, const void* R, int64_t ldr, int act, void* D,
                              int64_t ldd, int64_t M, int64_t N, int64_t K, void* stream) {
    clear_error();
    const Problem pr{X,     ldx,  x_type, x_scale, ldxs, {{"W", Wq, ldq, scales, lds, zeros, ldz}, {}},
                     group, bias, R,      ldr,     act,  D,
                     ldd,   M,    N,      K,       false};
    return run(pr, stream);
}

gb_status_t gb_gemm_ffn_gated_w4(const void* X, int64_t ldx, int x_type, const float* x_scale, int64_t ldxs,
                                 const void* W1q, int64_t ldq1, const void* scales1, int64_t lds1, const void* zeros1,
                                 int64_t ldz1, const void* W3q, int64_t ldq3, const void* scales3, int64_t lds3,
                                 const void* zeros3, int64_t ldz3, int group, void* D, int64_t ldd, int64_t M,
                                 int64_t N, int64_t K, void* stream) {
    clear_error();
    const Problem pr{X,
                     ldx,
                     x_type,
                     x_scale,
                     ldxs,
                     {{"W1", W1q, ldq1, scales1, lds1, zeros1, ldz1}, {"W3", W3q, ldq3, scales3, lds3, zeros3, ldz3}},
                     group,
                     nullptr,
                     nullptr,
                     0,
                     GB_ACT_NONE,
                     D,
                     ldd,
                     M,
                     N,
                     K,
                     true};
    return run(pr, stream);
}

}  // extern "C"
