// C ABI of the mixture-of-experts layer: argument checks, launch shapes and launches of the kernels in
// moe_kernel.cuh.
#include <algorithm>
#include <atomic>
#include <cinttypes>

#include "host.h"
#include "moe_kernel.cuh"

namespace {

using namespace gb::host;
using namespace gb::moe;

struct Matrix {
    const char* name;
    const void* p;
    int64_t ld, rows, cols;
};

// A matrix that is read in 16-byte words.
gb_status_t check_wide(const Matrix& m) {
    if (!m.p) return fail(GB_ERR_INVALID_ARG, "%s is null", m.name);
    if (m.ld < m.cols)
        return fail(GB_ERR_INVALID_ARG, "leading dimension %" PRId64 " of %s is below its row length %" PRId64, m.ld, m.name,
                    m.cols);
    if (!aligned_to(m.p, 16) || (m.rows > 1 && m.ld % 8))  // (one row has no next one)
        return fail(GB_ERR_UNSUPPORTED, "%s: base address and rows must be 16-byte aligned (leading dimension %" PRId64 ")",
                    m.name, m.ld);
    return GB_OK;
}

gb_status_t check_sizes(int64_t T, int64_t D, int64_t I, int64_t E, int top) {
    if (T < 0 || D < 0 || I < 0 || E < 0)
        return fail(GB_ERR_INVALID_ARG, "negative size T=%" PRId64 " D=%" PRId64 " I=%" PRId64 " E=%" PRId64, T, D, I, E);
    if (T > kMaxDim || D > kMaxDim || I > kMaxDim)
        return fail(GB_ERR_UNSUPPORTED, "sizes must be below 2^31 (T=%" PRId64 " D=%" PRId64 " I=%" PRId64 ")", T, D, I);
    // (the kernels count columns in 32 bits: some steps ahead, and the router rounded up to 256 for each of 64 parts)
    if (D > kMaxDim - 65536 || I > kMaxDim - 65536)
        return fail(GB_ERR_UNSUPPORTED, "rows of 2^31 - 65536 columns at most (D=%" PRId64 " I=%" PRId64 ")", D, I);
    if (E > kMaxExperts) return fail(GB_ERR_UNSUPPORTED, "%" PRId64 " experts: at most %d", E, kMaxExperts);
    if (top < 1 || top > E) return fail(GB_ERR_INVALID_ARG, "top_k=%d of %" PRId64 " experts", top, E);
    if (top > kMaxTop) return fail(GB_ERR_UNSUPPORTED, "top_k=%d: at most %d", top, kMaxTop);
    return GB_OK;
}

int64_t act_columns(int64_t inner) { return ceil_div(inner, 8) * 8; }

// Two terms of the inner activation for a pass's pairs.
int64_t workspace_of(int64_t T, int64_t I, int top) {
    return 2 * std::min<int64_t>(T, kPassTokens) * top * act_columns(I) * 2;
}

}  // namespace

extern "C" {

gb_status_t gb_moe_ffn_gated_workspace_bytes(int64_t T, int64_t I, int64_t E, int top_k, size_t* bytes) {
    clear_error();
    if (!bytes) return fail(GB_ERR_INVALID_ARG, "bytes is null");
    *bytes = 0;
    const gb_status_t st = check_sizes(T, 0, I, E, top_k);
    if (st == GB_OK) *bytes = static_cast<size_t>(workspace_of(T, I, top_k));
    return st;
}

gb_status_t gb_moe_ffn_gated(const void* X, int64_t ldx, const void* router, int64_t ldrouter, const void* W1, int64_t ld1,
                             int64_t expert1, const void* W3, int64_t ld3, int64_t expert3, const void* W2, int64_t ld2,
                             int64_t expert2, const void* R, int64_t ldr, int top_k, int renormalize, void* D_, int64_t ldd,
                             int32_t* ids, float* weights, void* workspace, size_t workspace_bytes, int64_t T, int64_t D,
                             int64_t I, int64_t E, void* stream) {
    clear_error();
    gb_status_t st = check_sizes(T, D, I, E, top_k);
    if (st != GB_OK) return st;
    if (T == 0) {
        note_empty();
        return GB_OK;
    }
    if (D == 0 || I == 0) return fail(GB_ERR_INVALID_ARG, "experts of %" PRId64 " x %" PRId64, I, D);
    const Matrix mats[] = {{"X", X, ldx, T, D},       {"router", router, ldrouter, E, D}, {"W1", W1, ld1, I, D},
                           {"W3", W3, ld3, I, D},     {"W2", W2, ld2, D, I}};
    for (const Matrix& m : mats)
        if ((st = check_wide(m)) != GB_OK) return st;
    const int64_t between[] = {expert1, expert3, expert2};
    for (int i = 0; i < 3; ++i) {
        const Matrix& m = mats[2 + i];
        if (E > 1 && (between[i] % 8 || between[i] < (m.rows - 1) * m.ld + m.cols))
            return fail(between[i] % 8 ? GB_ERR_UNSUPPORTED : GB_ERR_INVALID_ARG,
                        "%s: experts %" PRId64 " elements apart (a multiple of 8, and at least a matrix)", m.name, between[i]);
    }
    if (!D_) return fail(GB_ERR_INVALID_ARG, "D is null");
    if (ldd < D) return fail(GB_ERR_INVALID_ARG, "leading dimension %" PRId64 " of D is below its row length %" PRId64, ldd, D);
    if (R && ldr < D) return fail(GB_ERR_INVALID_ARG, "leading dimension %" PRId64 " of R is below its row length %" PRId64, ldr, D);
    if (!aligned_to(D_, 2) || !aligned_to(R, 2)) return fail(GB_ERR_UNSUPPORTED, "D and R must be 2-byte aligned");
    if (!ids || !weights) return fail(GB_ERR_INVALID_ARG, "%s is null", ids ? "weights" : "ids");
    if (!aligned_to(ids, 4) || !aligned_to(weights, 4)) return fail(GB_ERR_UNSUPPORTED, "ids and weights must be 4-byte aligned");
    const size_t need = static_cast<size_t>(workspace_of(T, I, top_k));
    if (!workspace || workspace_bytes < need)
        return fail(GB_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : size_t(0), need);
    if (!aligned_to(workspace, 16)) return fail(GB_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    int dev = 0;
    DeviceInfo info;
    if ((st = device_info(&dev, &info)) != GB_OK) return st;
    static std::atomic<bool> ready[64];
    static ClusterCounts counts;
    const size_t most = kWarps * kPassTokens * kRows * sizeof(float);
    if ((st = allow_smem(down_kernel, ready, dev, most)) != GB_OK) return st;

    Params prm{};
    prm.x = static_cast<const uint16_t*>(X);
    prm.router = static_cast<const uint16_t*>(router);
    const void* w[] = {W1, W3, W2};
    for (int i = 0; i < 3; ++i) {
        prm.w[i] = static_cast<const uint16_t*>(w[i]);
        prm.ldw[i] = mats[2 + i].ld;
        prm.expert[i] = between[i];
    }
    prm.r = static_cast<const uint16_t*>(R);
    prm.out = static_cast<uint16_t*>(D_);
    prm.ids = ids;
    prm.weights = weights;
    prm.ldact = act_columns(I);
    prm.act[0] = static_cast<uint16_t*>(workspace);
    prm.act[1] = prm.act[0] + std::min<int64_t>(T, kPassTokens) * top_k * prm.ldact;
    prm.ldx = ldx;
    prm.ldrouter = ldrouter;
    prm.ldr = ldr;
    prm.ldo = ldd;
    prm.d = static_cast<int>(D);
    prm.inner = static_cast<int>(I);
    prm.experts = static_cast<int>(E);
    prm.top = top_k;
    prm.renormalize = renormalize != 0;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);

    // a token's router: warps for 512 columns of each expert, as far as eight CTAs go
    int route = 1, parts = 1;
    while (route < 8 && route * kWarps < E * ceil_div(D, 512)) route *= 2;
    while (2 * parts * E <= route * kWarps && parts < ceil_div(D, 256)) parts *= 2;
    const int64_t tiles = ceil_div(D, kRows), slots = 2 * info.sms;
    int share = 1;  // CTAs of a tile of D: as many as run at once
    for (int64_t at_once; share < 8; share *= 2) {
        if ((st = counts.get(down_kernel, kThreads, most, dev, 2 * share, &at_once)) != GB_OK) return st;
        if (tiles > at_once) break;
    }
    prm.share = share;
    for (int64_t at = 0; at < T; at += kPassTokens) {
        prm.tokens = static_cast<int>(std::min<int64_t>(T - at, kPassTokens));
        const int64_t chosen = std::min<int64_t>(E, static_cast<int64_t>(prm.tokens) * top_k);
        const int64_t units = chosen * ceil_div(I, kRows), blocks = std::min(units, slots);
        if ((st = Launch(static_cast<unsigned>(prm.tokens * route), kThreads, 0, s, route)("moe router launch", router_kernel,
                                                                                          prm, route, parts)) != GB_OK)
            return st;
        if ((st = Launch(static_cast<unsigned>(blocks), kThreads, 0, s)("moe gated product launch", up_kernel, prm)) != GB_OK)
            return st;
        const size_t smem = static_cast<size_t>(kWarps) * prm.tokens * kRows * 4;
        if ((st = Launch(static_cast<unsigned>(tiles * share), kThreads, smem, s, share)("moe second product launch",
                                                                                        down_kernel, prm)) != GB_OK)
            return st;
        note_plan("kernel=moe_ffn_gated tokens=%lld router=%lld up_blocks=%lld tiles=%lld cluster=%lld passes=%lld", prm.tokens,
                  route, blocks, tiles, share, ceil_div(T, kPassTokens));
        prm.x += prm.tokens * ldx;
        prm.ids += prm.tokens * top_k;
        prm.weights += prm.tokens * top_k;
        if (prm.r) prm.r += prm.tokens * ldr;
        prm.out += prm.tokens * ldd;
    }
    return GB_OK;
}

}  // extern "C"
