// C ABI of the row operators: argument checks, launch shapes and launches of the kernels in
// rowwise.cuh and layernorm.cuh.
#include <algorithm>
#include <atomic>
#include <cinttypes>
#include <cmath>

#include "host.h"
#include "layernorm.cuh"
#include "rowwise.cuh"

namespace {

using namespace gb::host;
using namespace gb::rowwise;

constexpr int kMaxNormColumns = 16384;  // 512 threads x 4 chunks of 8
// The kernels count columns in 32 bits: a chunk's first column and 8 have to be a number of theirs, for the
// last chunk of a row that is shifted by up to 7.
constexpr int64_t kMaxColumns = (int64_t(1) << 31) - 16;

// One matrix of a call, by its name in the messages.
struct Mat {
    const char* name;
    const void* p;
    int64_t ld;
    int64_t bytes;  // of an element
};

gb_status_t check_sizes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return fail(GB_ERR_INVALID_ARG, "negative size %" PRId64 " x %" PRId64, rows, cols);
    if (rows > kMaxDim || cols > kMaxDim)
        return fail(GB_ERR_UNSUPPORTED, "sizes must be below 2^31 (%" PRId64 " x %" PRId64 ")", rows, cols);
    return GB_OK;
}

gb_status_t check_mat(const Mat& m, int64_t cols) {
    if (!m.p) return fail(GB_ERR_INVALID_ARG, "%s is null", m.name);
    if (m.ld < cols)
        return fail(GB_ERR_INVALID_ARG, "leading dimension %" PRId64 " of %s is below its row length %" PRId64, m.ld,
                    m.name, cols);
    if (!aligned_to(m.p, m.bytes))
        return fail(GB_ERR_UNSUPPORTED, "%s must be %d-byte aligned", m.name, static_cast<int>(m.bytes));
    return GB_OK;
}

gb_status_t check_ptr(const char* name, const void* p, uintptr_t align) {
    if (!p) return fail(GB_ERR_INVALID_ARG, "%s is null", name);
    if (!aligned_to(p, align)) return fail(GB_ERR_UNSUPPORTED, "%s must be %d-byte aligned", name, static_cast<int>(align));
    return GB_OK;
}

// The generator's keys, and the words that are kept: those of at least p 2^32, or above one less.
gb_status_t make_drop(double p, uint64_t seed, uint64_t offset, const void* state, Drop* out) {
    if (!(p >= 0.0 && p <= 1.0)) return fail(GB_ERR_INVALID_ARG, "p=%g is not a probability", p);
    if (!aligned_to(state, 8)) return fail(GB_ERR_UNSUPPORTED, "rng_state must be 8-byte aligned");
    const uint64_t least = static_cast<uint64_t>(std::llround(p * 4294967296.0));
    uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
    for (auto& key : out->keys) {
        key[0] = k0;
        key[1] = k1;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    out->offset[0] = static_cast<uint32_t>(offset);
    out->offset[1] = static_cast<uint32_t>(offset >> 32);
    out->state = static_cast<const uint64_t*>(state);
    out->limit = least > 0 ? static_cast<uint32_t>(least - 1) : 0;
    out->scale = static_cast<float>(1.0 / (1.0 - p));
    return GB_OK;
}

int drop_kind(double p, const void* state) { return p == 0.0 ? kNoDrop : state ? kState : kKeys; }

// Whether all matrices have the same shift on every row: the same position, in elements,
// modulo 8 of their bases and of their leading dimensions.
template <size_t N>
bool same_shift(const Mat (&mats)[N], int64_t rows) {
    const Mat& a = mats[0];
    for (const Mat& m : mats) {
        if (!m.p) continue;
        const uintptr_t u = reinterpret_cast<uintptr_t>(m.p) / m.bytes, v = reinterpret_cast<uintptr_t>(a.p) / a.bytes;
        if (((u ^ v) & 7) || (rows > 1 && ((m.ld ^ a.ld) & 7))) return false;
    }
    return true;
}

// Chunks that cover a row of `cols` elements whatever its shift.
int64_t chunks_of(const Mat& m, int64_t rows, int64_t cols, bool wide) {
    const bool shifted = wide && (!aligned_to(m.p, 8 * m.bytes) || (rows > 1 && (m.ld & 7)));
    return ceil_div(cols + (shifted ? 7 : 0), 8);
}

// How the rows of a norm are given to threads.
struct RowPlan {
    int chunks_per_thread = 0;  // 2 or 4
    int threads = 0, rows = 1;  // of a block
    bool wide = false;
};

// Up to 64 chunks a row is one warp's, eight rows to a block: no barrier.  Above, it
// is a block's, with two chunks a thread while 512 threads cover it and four beyond.
constexpr int kWarpChunks = 64;

RowPlan plan_chunks(int64_t chunks) {
    RowPlan pl;
    if (chunks <= kWarpChunks) {
        pl.threads = 32;
        pl.rows = 8;
        pl.chunks_per_thread = 2;
    } else {
        pl.chunks_per_thread = chunks <= 1024 ? 2 : 4;
        pl.threads = static_cast<int>(ceil_div(chunks, 32 * pl.chunks_per_thread)) * 32;
    }
    return pl;
}

template <size_t N>
RowPlan plan_rows(const Mat (&mats)[N], int64_t rows, int64_t cols) {
    RowPlan pl;
    pl.wide = same_shift(mats, rows);
    int64_t chunks = chunks_of(mats[0], rows, cols, pl.wide);
    if (chunks > kMaxNormColumns / 8) {  // (16384 shifted columns: one chunk too many)
        pl.wide = false;
        chunks = ceil_div(cols, 8);
    }
    const bool wide = pl.wide;
    pl = plan_chunks(chunks);
    pl.wide = wide;
    return pl;
}

// Blocks of `per_sm` threads an SM, a multiple of 8 of them (see the kernels' rows); no more than there are
// rows for.  (More than are resident at once in places: of the forward pass's 1024 threads at 4096 columns,
// shared memory holds three blocks of 256, and the fourth of each SM comes after them.)
int64_t blocks_for(int64_t m, const RowPlan& pl, int per_sm, int sms) {
    const int64_t full = static_cast<int64_t>(sms) * std::max(1, per_sm / (pl.threads * pl.rows)) / 8 * 8;
    return std::min(ceil_div(m, pl.rows), std::max<int64_t>(8, full));
}

template <int V, int DROP, int OUT>
gb_status_t launch_norm(const NormParams& p, const RowPlan& pl, int dev, const DeviceInfo& info, cudaStream_t stream) {
    static std::atomic<bool> ready[64];
    gb_status_t st = allow_smem(norm_kernel<V, DROP, OUT>, ready, dev, info.smem_optin - 1024);
    if (st != GB_OK) return st;
    const int64_t blocks = blocks_for(p.m, pl, V == 4 ? 512 : DROP ? 768 : 1024, info.sms);
    size_t smem = static_cast<size_t>(kRowStages * 2 + 1) * V * 16 * pl.threads * pl.rows;
    if (OUT == kGroupScale) smem += static_cast<size_t>(pl.rows) * ceil_div(p.d, kScaleGroup) * 4;
    note_plan("kernel=add_rms_norm output=%lld dropout=%lld threads=%lld rows=%lld blocks=%lld wide=%lld", OUT, DROP,
              pl.threads, pl.rows, blocks, pl.wide);
    return Launch(static_cast<unsigned>(blocks), dim3(pl.threads, pl.rows), smem, stream)(
        "add_rms_norm launch", norm_kernel<V, DROP, OUT>, p);
}

template <int DROP, int OUT>
gb_status_t run_norm(const NormParams& p, const RowPlan& pl, int dev, const DeviceInfo& info, cudaStream_t stream) {
    return pl.chunks_per_thread <= 2 ? launch_norm<2, DROP, OUT>(p, pl, dev, info, stream)
                                     : launch_norm<4, DROP, OUT>(p, pl, dev, info, stream);
}

template <int V, int DROP>
gb_status_t launch_bwd(const NormBwdParams& p, const RowPlan& pl, int blocks, int dev, const DeviceInfo& info,
                       cudaStream_t stream) {
    static std::atomic<bool> ready[64];
    gb_status_t st = allow_smem(norm_bwd_kernel<V, DROP>, ready, dev, info.smem_optin - 1024);
    if (st != GB_OK) return st;
    // two stages of three matrices, and the weight; and the join of a block's rows
    size_t smem = static_cast<size_t>(kBwdStages * 3 + 1) * V * 16 * pl.threads * pl.rows;
    if (pl.rows > 1) smem = std::max(smem, static_cast<size_t>(p.d) * 4);
    return Launch(blocks, dim3(pl.threads, pl.rows), smem, stream)("add_rms_norm_backward launch",
                                                                   norm_bwd_kernel<V, DROP>, p);
}

template <int DROP>
gb_status_t run_bwd(const NormBwdParams& p, const RowPlan& pl, int blocks, int dev, const DeviceInfo& info,
                    cudaStream_t stream) {
    return pl.chunks_per_thread <= 2 ? launch_bwd<2, DROP>(p, pl, blocks, dev, info, stream)
                                     : launch_bwd<4, DROP>(p, pl, blocks, dev, info, stream);
}

// Blocks of the backward pass: each keeps a part of the weight's gradient in the workspace.  The
// workspace's size is asked without the matrices' addresses: with no shift there are most blocks.
int bwd_blocks(int64_t m, const RowPlan& pl, int sms) {
    return static_cast<int>(blocks_for(m, pl, pl.chunks_per_thread == 2 ? 768 : 512, sms));
}

int64_t bwd_workspace(int64_t m, int64_t d, int sms) {
    const int64_t by_warps = bwd_blocks(m, plan_chunks(ceil_div(d, 8)), sms);
    return std::max<int64_t>(by_warps, bwd_blocks(m, plan_chunks(ceil_div(d + 7, 8)), sms)) * d * 4;
}

// ---------------------------------------------------------------- layer norm

// A row's columns in the parts of its two gradients: whole chunks, a shift counted in.
int64_t layer_bwd_pitch(int64_t d) { return ceil_div(d + 7, 8) * 8; }

int64_t layer_bwd_workspace(int64_t m, int64_t d, int sms) { return bwd_workspace(m, d, sms) / d * layer_bwd_pitch(d) * 2; }

// Whether every row of the matrices is whole, aligned 16-byte words.
template <size_t N>
bool full_rows(const Mat (&mats)[N], int64_t rows, int64_t cols) {
    if (cols % 8) return false;
    for (const Mat& m : mats)
        if (m.p && (!aligned_to(m.p, 16) || (rows > 1 && m.ld % 8))) return false;
    return true;
}

template <int V, int DROP, bool FULL>
gb_status_t launch_layer_norm(const LayerNormParams& p, const RowPlan& pl, int dev, const DeviceInfo& info,
                              cudaStream_t stream) {
    static std::atomic<bool> ready[64];
    gb_status_t st = allow_smem(layer_norm_kernel<V, DROP, FULL>, ready, dev, info.smem_optin - 1024);
    if (st != GB_OK) return st;
    const int64_t blocks = blocks_for(p.m, pl, V == 4 ? 512 : 768, info.sms);
    const size_t smem = static_cast<size_t>(layer_norm_stages(V) * 2 + (FULL && V == 2 ? 0 : 2)) * V * 16 * pl.threads * pl.rows;
    note_plan("kernel=add_layer_norm dropout=%lld threads=%lld rows=%lld blocks=%lld wide=%lld full=%lld", DROP,
              pl.threads, pl.rows, blocks, pl.wide, FULL);
    return Launch(static_cast<unsigned>(blocks), dim3(pl.threads, pl.rows), smem, stream)(
        "add_layer_norm launch", layer_norm_kernel<V, DROP, FULL>, p);
}

template <int DROP>
gb_status_t run_layer_norm(const LayerNormParams& p, const RowPlan& pl, bool full, int dev, const DeviceInfo& info,
                           cudaStream_t stream) {
    if (full)
        return pl.chunks_per_thread <= 2 ? launch_layer_norm<2, DROP, true>(p, pl, dev, info, stream)
                                         : launch_layer_norm<4, DROP, true>(p, pl, dev, info, stream);
    return pl.chunks_per_thread <= 2 ? launch_layer_norm<2, DROP, false>(p, pl, dev, info, stream)
                                     : launch_layer_norm<4, DROP, false>(p, pl, dev, info, stream);
}

template <int V, int DROP, bool FULL>
gb_status_t launch_layer_bwd(const LayerNormBwdParams& p, const RowPlan& pl, int* blocks, int dev, const DeviceInfo& info,
                             cudaStream_t stream) {
    static std::atomic<bool> ready[64];
    gb_status_t st = allow_smem(layer_norm_bwd_kernel<V, DROP, FULL>, ready, dev, info.smem_optin - 1024);
    if (st != GB_OK) return st;
    // the stages of three matrices, and the weight; and the join of a block's rows
    size_t smem = static_cast<size_t>(layer_bwd_stages(V) * 3 + (FULL && V == 2 ? 0 : 1)) * V * 16 * pl.threads * pl.rows;
    if (pl.rows > 1) smem = std::max(smem, static_cast<size_t>(p.d) * 8);
    if (V == 2) *blocks = static_cast<int>(blocks_for(p.m, pl, FULL ? 512 : 576, info.sms));  // (the workspace has room for 768)
    return Launch(*blocks, dim3(pl.threads, pl.rows), smem, stream)("add_layer_norm_backward launch",
                                                                    layer_norm_bwd_kernel<V, DROP, FULL>, p);
}

template <int DROP>
gb_status_t run_layer_bwd(const LayerNormBwdParams& p, const RowPlan& pl, bool full, int* blocks, int dev,
                          const DeviceInfo& info, cudaStream_t stream) {
    if (full)
        return pl.chunks_per_thread <= 2 ? launch_layer_bwd<2, DROP, true>(p, pl, blocks, dev, info, stream)
                                         : launch_layer_bwd<4, DROP, true>(p, pl, blocks, dev, info, stream);
    return pl.chunks_per_thread <= 2 ? launch_layer_bwd<2, DROP, false>(p, pl, blocks, dev, info, stream)
                                     : launch_layer_bwd<4, DROP, false>(p, pl, blocks, dev, info, stream);
}

}  // namespace

extern "C" {

gb_status_t gb_dropout(const void* X, int64_t ldx, const void* R, int64_t ldr, double p, uint64_t seed,
                       uint64_t offset, const void* rng_state, void* D, int64_t ldd, int64_t M, int64_t N,
                       void* stream) {
    clear_error();
    gb_status_t st;
    if ((st = check_sizes(M, N)) != GB_OK) return st;
    DropoutParams prm{};
    if ((st = make_drop(p, seed, offset, rng_state, &prm.drop)) != GB_OK) return st;
    if (N > kMaxColumns) return fail(GB_ERR_UNSUPPORTED, "rows of %" PRId64 " columns: at most 2^31 - 16", N);
    if (M == 0 || N == 0) {
        note_empty();
        return GB_OK;
    }
    const Mat mats[] = {{"X", X, ldx, 2}, {"D", D, ldd, 2}, {"R", R, ldr, 2}};
    for (const Mat& m : mats)
        if ((m.p || m.name[0] != 'R') && (st = check_mat(m, N)) != GB_OK) return st;
    int dev = 0;
    DeviceInfo info;
    if ((st = device_info(&dev, &info)) != GB_OK) return st;
    prm.x = static_cast<const uint16_t*>(X);
    prm.r = static_cast<const uint16_t*>(R);
    prm.d = static_cast<uint16_t*>(D);
    prm.ldx = ldx;
    prm.ldr = ldr;
    prm.ldd = ldd;
    prm.m = static_cast<int>(M);
    prm.n = static_cast<int>(N);
    prm.wide = same_shift(mats, M);
    prm.chunks = static_cast<int>(chunks_of(mats[0], M, N, prm.wide));
    const int64_t blocks = std::min<int64_t>(ceil_div(M * prm.chunks, kDropoutThreads * kDropoutBatch), 8 * info.sms);
    prm.step_rows = blocks * kDropoutThreads / prm.chunks;
    prm.step_chunks = static_cast<int>(blocks * kDropoutThreads % prm.chunks);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    note_plan("kernel=dropout blocks=%lld threads=%lld chunks=%lld wide=%lld residual=%lld state=%lld", blocks,
              kDropoutThreads, prm.chunks, prm.wide, R != nullptr, rng_state != nullptr);
    const int kind = drop_kind(p, rng_state);
    const auto kernel = kind == kNoDrop ? dropout_kernel<kNoDrop> : kind == kKeys ? dropout_kernel<kKeys> : dropout_kernel<kState>;
    return Launch(static_cast<unsigned>(blocks), kDropoutThreads, 0, s)("dropout launch", kernel, prm);
}

gb_status_t gb_add_rms_norm(const void* X, int64_t ldx, const void* R, int64_t ldr, const void* weight, double eps,
                            double p, uint64_t seed, uint64_t offset, const void* rng_state, void* H, int64_t ldh,
                            void* Y, int64_t ldy, float* rstd, int64_t M, int64_t D, void* stream) {
    clear_error();
    gb_status_t st;
    if ((st = check_sizes(M, D)) != GB_OK) return st;
    NormParams prm{};
    if ((st = make_drop(p, seed, offset, rng_state, &prm.drop)) != GB_OK) return st;
    if (!(eps >= 0.0 && std::isfinite(eps))) return fail(GB_ERR_INVALID_ARG, "eps=%g is not a finite number >= 0", eps);
    if (M == 0 || D == 0) {
        note_empty();
        return GB_OK;
    }
    const Mat mats[] = {{"X", X, ldx, 2}, {"Y", Y, ldy, 2}, {"R", R, ldr, 2}, {"H", H, ldh, 2}};
    for (const Mat& m : mats)
        if ((m.p || m.name[0] == 'X' || m.name[0] == 'Y') && (st = check_mat(m, D)) != GB_OK) return st;
    if ((st = check_ptr("weight", weight, 2)) != GB_OK) return st;
    if (rstd && (st = check_ptr("rstd", rstd, 4)) != GB_OK) return st;
    if (D > kMaxNormColumns)
        return fail(GB_ERR_UNSUPPORTED, "rows of %" PRId64 " columns: at most %d", D, kMaxNormColumns);
    int dev = 0;
    DeviceInfo info;
    if ((st = device_info(&dev, &info)) != GB_OK) return st;
    prm.x = static_cast<const uint16_t*>(X);
    prm.r = static_cast<const uint16_t*>(R);
    prm.weight = static_cast<const uint16_t*>(weight);
    prm.h = static_cast<uint16_t*>(H);
    prm.y = static_cast<uint16_t*>(Y);
    prm.rstd = rstd;
    prm.ldx = ldx;
    prm.ldr = ldr;
    prm.ldh = ldh;
    prm.ldy = ldy;
    prm.m = static_cast<int>(M);
    prm.d = static_cast<int>(D);
    prm.eps = static_cast<float>(eps);
    const RowPlan pl = plan_rows(mats, M, D);
    prm.wide = pl.wide;
    prm.wide_weight = aligned_to(weight, 16);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (drop_kind(p, rng_state)) {
        case kNoDrop: return run_norm<kNoDrop, kBf16>(prm, pl, dev, info, s);
        case kKeys: return run_norm<kKeys, kBf16>(prm, pl, dev, info, s);
        default: return run_norm<kState, kBf16>(prm, pl, dev, info, s);
    }
}

gb_status_t gb_add_rms_norm_q8(const void* X, int64_t ldx, const void* R, int64_t ldr, const void* weight, double eps,
                               int scale_group, void* H, int64_t ldh, void* Q, int64_t ldq, float* scale, int64_t lds,
                               int64_t M, int64_t D, void* stream) {
    clear_error();
    gb_status_t st;
    if ((st = check_sizes(M, D)) != GB_OK) return st;
    if (!(eps >= 0.0 && std::isfinite(eps))) return fail(GB_ERR_INVALID_ARG, "eps=%g is not a finite number >= 0", eps);
    if (scale_group != 0 && scale_group != kScaleGroup)
        return fail(GB_ERR_INVALID_ARG, "scale_group=%d: 0 (a scale for each row) or %d columns", scale_group, kScaleGroup);
    if (M == 0 || D == 0) {
        note_empty();
        return GB_OK;
    }
    const Mat mats[] = {{"X", X, ldx, 2}, {"Q", Q, ldq, 1}, {"R", R, ldr, 2}, {"H", H, ldh, 2}};
    for (const Mat& m : mats)
        if ((m.p || m.name[0] == 'X' || m.name[0] == 'Q') && (st = check_mat(m, D)) != GB_OK) return st;
    if ((st = check_ptr("weight", weight, 2)) != GB_OK) return st;
    if ((st = check_mat({"scale", scale, lds, 4}, scale_group ? ceil_div(D, kScaleGroup) : 1)) != GB_OK) return st;
    if (D > kMaxNormColumns)
        return fail(GB_ERR_UNSUPPORTED, "rows of %" PRId64 " columns: at most %d", D, kMaxNormColumns);
    int dev = 0;
    DeviceInfo info;
    if ((st = device_info(&dev, &info)) != GB_OK) return st;
    NormParams prm{};
    prm.x = static_cast<const uint16_t*>(X);
    prm.r = static_cast<const uint16_t*>(R);
    prm.weight = static_cast<const uint16_t*>(weight);
    prm.h = static_cast<uint16_t*>(H);
    prm.q = static_cast<uint8_t*>(Q);
    prm.scale = scale;
    prm.ldx = ldx;
    prm.ldr = ldr;
    prm.ldh = ldh;
    prm.ldq = ldq;
    prm.lds = lds;
    prm.m = static_cast<int>(M);
    prm.d = static_cast<int>(D);
    prm.eps = static_cast<float>(eps);
    const RowPlan pl = plan_rows(mats, M, D);
    prm.wide = pl.wide;
    prm.wide_weight = aligned_to(weight, 16);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return scale_group ? run_norm<kNoDrop, kGroupScale>(prm, pl, dev, info, s)
                       : run_norm<kNoDrop, kRowScale>(prm, pl, dev, info, s);
}

gb_status_t gb_add_rms_norm_backward_workspace_bytes(int64_t M, int64_t D, size_t* bytes) {
    clear_error();
    gb_status_t st;
    if (!bytes) return fail(GB_ERR_INVALID_ARG, "bytes is null");
    *bytes = 0;
    if ((st = check_sizes(M, D)) != GB_OK) return st;
    if (M == 0 || D == 0) return GB_OK;
    int dev = 0;
    DeviceInfo info;
    if ((st = device_info(&dev, &info)) != GB_OK) return st;
    *bytes = static_cast<size_t>(bwd_workspace(M, D, info.sms));
    return GB_OK;
}

gb_status_t gb_add_rms_norm_backward(const void* dY, int64_t lddy, const void* H, int64_t ldh, const void* weight,
                                     const float* rstd, const void* dH, int64_t lddh, double p, uint64_t seed,
                                     uint64_t offset, const void* rng_state, void* dR, int64_t lddr, void* dX,
                                     int64_t lddx, float* dweight, void* workspace, size_t workspace_bytes, int64_t M,
                                     int64_t D, void* stream) {
    clear_error();
    gb_status_t st;
    if ((st = check_sizes(M, D)) != GB_OK) return st;
    NormBwdParams prm{};
    if ((st = make_drop(p, seed, offset, rng_state, &prm.drop)) != GB_OK) return st;
    if (D == 0) {
        note_empty();
        return GB_OK;
    }
    const bool drop = p > 0.0;
    if ((st = check_ptr("dweight", dweight, 4)) != GB_OK) return st;
    const Mat mats[] = {{"dY", dY, lddy, 2}, {"H", H, ldh, 2}, {"dR", dR, lddr, 2}, {"dH", dH, lddh, 2},
                        {"dX", drop ? dX : nullptr, lddx, 2}};
    if (M > 0) {
        for (int i = 0; i < 5; ++i)
            if ((i < 3 || mats[i].p || (i == 4 && drop)) && (st = check_mat(mats[i], D)) != GB_OK) return st;
        if ((st = check_ptr("weight", weight, 2)) != GB_OK) return st;
        if ((st = check_ptr("rstd", rstd, 4)) != GB_OK) return st;
    }
    if (D > kMaxNormColumns)
        return fail(GB_ERR_UNSUPPORTED, "rows of %" PRId64 " columns: at most %d", D, kMaxNormColumns);
    int dev = 0;
    DeviceInfo info;
    if ((st = device_info(&dev, &info)) != GB_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int blocks = 0;
    RowPlan pl;
    if (M > 0) {
        const size_t need = static_cast<size_t>(bwd_workspace(M, D, info.sms));
        if (!workspace || workspace_bytes < need)
            return fail(GB_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : size_t(0),
                        need);
        if (!aligned_to(workspace, 4)) return fail(GB_ERR_INVALID_ARG, "workspace must be 4-byte aligned");
        prm.dy = static_cast<const uint16_t*>(dY);
        prm.h = static_cast<const uint16_t*>(H);
        prm.weight = static_cast<const uint16_t*>(weight);
        prm.rstd = rstd;
        prm.dh = static_cast<const uint16_t*>(dH);
        prm.dr = static_cast<uint16_t*>(dR);
        prm.dx = static_cast<uint16_t*>(dX);
        prm.partial = static_cast<float*>(workspace);
        prm.lddy = lddy;
        prm.ldh = ldh;
        prm.lddh = lddh;
        prm.lddr = lddr;
        prm.lddx = lddx;
        prm.m = static_cast<int>(M);
        prm.d = static_cast<int>(D);
        pl = plan_rows(mats, M, D);
        prm.wide = pl.wide;
        prm.wide_weight = aligned_to(weight, 16);
        blocks = bwd_blocks(M, pl, info.sms);
        switch (drop_kind(p, rng_state)) {
            case kNoDrop: st = run_bwd<kNoDrop>(prm, pl, blocks, dev, info, s); break;
            case kKeys: st = run_bwd<kKeys>(prm, pl, blocks, dev, info, s); break;
            default: st = run_bwd<kState>(prm, pl, blocks, dev, info, s); break;
        }
        if (st != GB_OK) return st;
    }
    note_plan("kernel=add_rms_norm_backward blocks=%lld dropout=%lld threads=%lld rows=%lld chunks=%lld wide=%lld", blocks,
              drop, pl.threads, pl.rows, pl.chunks_per_thread, pl.wide);
    return Launch(static_cast<unsigned>(ceil_div(D, kJoinColumns)), dim3(kJoinColumns, kJoinParts), 0, s)(
        "add_rms_norm_backward join launch", join_kernel, static_cast<const float*>(workspace), blocks, static_cast<int>(D),
        dweight);
}

gb_status_t gb_add_layer_norm(const void* X, int64_t ldx, const void* R, int64_t ldr, const void* weight,
                              const void* bias, double eps, double p, uint64_t seed, uint64_t offset,
                              const void* rng_state, void* H, int64_t ldh, void* Y, int64_t ldy, float* mean, float* rstd,
                              int64_t M, int64_t D, void* stream) {
    clear_error();
    gb_status_t st;
    if ((st = check_sizes(M, D)) != GB_OK) return st;
    LayerNormParams prm{};
    if ((st = make_drop(p, seed, offset, rng_state, &prm.drop)) != GB_OK) return st;
    if (!(eps >= 0.0 && std::isfinite(eps))) return fail(GB_ERR_INVALID_ARG, "eps=%g is not a finite number >= 0", eps);
    if (M == 0 || D == 0) {
        note_empty();
        return GB_OK;
    }
    const Mat mats[] = {{"X", X, ldx, 2}, {"Y", Y, ldy, 2}, {"R", R, ldr, 2}, {"H", H, ldh, 2}};
    for (const Mat& m : mats)
        if ((m.p || m.name[0] == 'X' || m.name[0] == 'Y') && (st = check_mat(m, D)) != GB_OK) return st;
    if ((st = check_ptr("weight", weight, 2)) != GB_OK) return st;
    if (bias && (st = check_ptr("bias", bias, 2)) != GB_OK) return st;
    if (mean && (st = check_ptr("mean", mean, 4)) != GB_OK) return st;
    if (rstd && (st = check_ptr("rstd", rstd, 4)) != GB_OK) return st;
    if (D > kMaxNormColumns)
        return fail(GB_ERR_UNSUPPORTED, "rows of %" PRId64 " columns: at most %d", D, kMaxNormColumns);
    int dev = 0;
    DeviceInfo info;
    if ((st = device_info(&dev, &info)) != GB_OK) return st;
    prm.x = static_cast<const uint16_t*>(X);
    prm.r = static_cast<const uint16_t*>(R);
    prm.weight = static_cast<const uint16_t*>(weight);
    prm.bias = static_cast<const uint16_t*>(bias);
    prm.h = static_cast<uint16_t*>(H);
    prm.y = static_cast<uint16_t*>(Y);
    prm.mean = mean;
    prm.rstd = rstd;
    prm.ldx = ldx;
    prm.ldr = ldr;
    prm.ldh = ldh;
    prm.ldy = ldy;
    prm.m = static_cast<int>(M);
    prm.d = static_cast<int>(D);
    prm.eps = static_cast<float>(eps);
    const RowPlan pl = plan_rows(mats, M, D);
    prm.wide = pl.wide;
    prm.wide_weight = aligned_to(weight, 16);
    prm.wide_bias = aligned_to(bias, 16);
    const bool full = full_rows(mats, M, D);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (drop_kind(p, rng_state)) {
        case kNoDrop: return run_layer_norm<kNoDrop>(prm, pl, full, dev, info, s);
        case kKeys: return run_layer_norm<kKeys>(prm, pl, full, dev, info, s);
        default: return run_layer_norm<kState>(prm, pl, full, dev, info, s);
    }
}

gb_status_t gb_add_layer_norm_backward_workspace_bytes(int64_t M, int64_t D, size_t* bytes) {
    clear_error();
    gb_status_t st;
    if (!bytes) return fail(GB_ERR_INVALID_ARG, "bytes is null");
    *bytes = 0;
    if ((st = check_sizes(M, D)) != GB_OK) return st;
    if (M == 0 || D == 0) return GB_OK;
    int dev = 0;
    DeviceInfo info;
    if ((st = device_info(&dev, &info)) != GB_OK) return st;
    *bytes = static_cast<size_t>(layer_bwd_workspace(M, D, info.sms));
    return GB_OK;
}

gb_status_t gb_add_layer_norm_backward(const void* dY, int64_t lddy, const void* H, int64_t ldh, const void* weight,
                                       const float* mean, const float* rstd, const void* dH, int64_t lddh, double p,
                                       uint64_t seed, uint64_t offset, const void* rng_state, void* dR, int64_t lddr,
                                       void* dX, int64_t lddx, float* dweight, float* dbias, void* workspace,
                                       size_t workspace_bytes, int64_t M, int64_t D, void* stream) {
    clear_error();
    gb_status_t st;
    if ((st = check_sizes(M, D)) != GB_OK) return st;
    LayerNormBwdParams prm{};
    if ((st = make_drop(p, seed, offset, rng_state, &prm.drop)) != GB_OK) return st;
    if (D == 0) {
        note_empty();
        return GB_OK;
    }
    const bool drop = p > 0.0;
    if ((st = check_ptr("dweight", dweight, 4)) != GB_OK) return st;
    if ((st = check_ptr("dbias", dbias, 4)) != GB_OK) return st;
    const Mat mats[] = {{"dY", dY, lddy, 2}, {"H", H, ldh, 2}, {"dR", dR, lddr, 2}, {"dH", dH, lddh, 2},
                        {"dX", drop ? dX : nullptr, lddx, 2}};
    if (M > 0) {
        for (int i = 0; i < 5; ++i)
            if ((i < 3 || mats[i].p || (i == 4 && drop)) && (st = check_mat(mats[i], D)) != GB_OK) return st;
        if ((st = check_ptr("weight", weight, 2)) != GB_OK) return st;
        if ((st = check_ptr("mean", mean, 4)) != GB_OK) return st;
        if ((st = check_ptr("rstd", rstd, 4)) != GB_OK) return st;
    }
    if (D > kMaxNormColumns)
        return fail(GB_ERR_UNSUPPORTED, "rows of %" PRId64 " columns: at most %d", D, kMaxNormColumns);
    int dev = 0;
    DeviceInfo info;
    if ((st = device_info(&dev, &info)) != GB_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int blocks = 0;
    RowPlan pl;
    if (M > 0) {
        const size_t need = static_cast<size_t>(layer_bwd_workspace(M, D, info.sms));
        if (!workspace || workspace_bytes < need)
            return fail(GB_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : size_t(0),
                        need);
        if (!aligned_to(workspace, 16)) return fail(GB_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
        prm.dy = static_cast<const uint16_t*>(dY);
        prm.h = static_cast<const uint16_t*>(H);
        prm.weight = static_cast<const uint16_t*>(weight);
        prm.mean = mean;
        prm.rstd = rstd;
        prm.dh = static_cast<const uint16_t*>(dH);
        prm.dr = static_cast<uint16_t*>(dR);
        prm.dx = static_cast<uint16_t*>(dX);
        prm.partial = static_cast<float*>(workspace);
        prm.pitch = static_cast<int>(layer_bwd_pitch(D));
        prm.lddy = lddy;
        prm.ldh = ldh;
        prm.lddh = lddh;
        prm.lddr = lddr;
        prm.lddx = lddx;
        prm.m = static_cast<int>(M);
        prm.d = static_cast<int>(D);
        pl = plan_rows(mats, M, D);
        prm.wide = pl.wide;
        prm.wide_weight = aligned_to(weight, 16);
        blocks = bwd_blocks(M, pl, info.sms);
        const bool full = full_rows(mats, M, D);
        switch (drop_kind(p, rng_state)) {
            case kNoDrop: st = run_layer_bwd<kNoDrop>(prm, pl, full, &blocks, dev, info, s); break;
            case kKeys: st = run_layer_bwd<kKeys>(prm, pl, full, &blocks, dev, info, s); break;
            default: st = run_layer_bwd<kState>(prm, pl, full, &blocks, dev, info, s); break;
        }
        if (st != GB_OK) return st;
    }
    // (a block of several rows has joined them by column)
    const bool shifted = prm.wide && pl.rows == 1;
    const int first = shifted ? static_cast<int>(reinterpret_cast<uintptr_t>(dY) >> 1 & 7) : 0;
    const int step = shifted ? static_cast<int>(lddy & 7) : 0;
    note_plan("kernel=add_layer_norm_backward blocks=%lld dropout=%lld threads=%lld rows=%lld chunks=%lld wide=%lld", blocks,
              drop, pl.threads, pl.rows, pl.chunks_per_thread, pl.wide);
    return Launch(static_cast<unsigned>(ceil_div(2 * D, kJoinColumns)), dim3(kJoinColumns, kJoinParts), 0, s)(
        "add_layer_norm_backward join launch", join2_kernel, static_cast<const float*>(workspace), blocks,
        static_cast<int>(D), prm.pitch, first, step, dweight, dbias);
}

}  // extern "C"
