// C ABI of the low-rank adapters: argument checks, launch shapes and launches of the kernels in
// lora_kernel.cuh.
#include <algorithm>
#include <atomic>
#include <cinttypes>
#include <cmath>

#include "host.h"
#include "lora_kernel.cuh"

namespace {

using namespace gb::host;
using namespace gb::lora;

gb_status_t check_sizes(int64_t M, int64_t N, int64_t K, int64_t r, int64_t adapters) {
    if (M < 0 || N < 0 || K < 0 || r < 0 || adapters < 0)
        return fail(GB_ERR_INVALID_ARG, "negative size M=%" PRId64 " N=%" PRId64 " K=%" PRId64 " r=%" PRId64 " adapters=%" PRId64,
                    M, N, K, r, adapters);
    // (the kernels count columns in 32 bits, some steps ahead)
    if (M > kMaxDim || N > kMaxDim - 4096 || K > kMaxDim - 4096 || adapters > kMaxDim)
        return fail(GB_ERR_UNSUPPORTED, "sizes must be below 2^31 - 4096 (M=%" PRId64 " N=%" PRId64 " K=%" PRId64
                                        " adapters=%" PRId64 ")", M, N, K, adapters);
    if (r > kMaxRank) return fail(GB_ERR_UNSUPPORTED, "rank %" PRId64 ": at most %d", r, kMaxRank);
    return GB_OK;
}

// Rows that are sorted by adapter: from 32 on by each block for itself, more than kHere by a launch before.  4096 x 4096
// of rank 16 with 64 adapters, and 14336 x 4096 of rank 64 with 4, in us (graphs of ten calls):
//     rows                16           31           64           128          200
//     not sorted          8.3  13.4    9.9  19.0
//     by each block      10.7  12.0   11.2  12.8   13.4  16.5   14.0  17.7   18.7  22.6
//     by a launch                                  18.1  17.3   17.7  20.7   16.3  21.0
// The rule goes by rows alone: 16 to 31 of them that share a few adapters with many columns would be faster sorted (16 rows
// 12.0 against 13.4, 31 rows 12.8 against 19.0, in the right columns), with 16 ranks and fewer columns slower.
constexpr int64_t kHereFrom = 32;

struct Plan {
    bool sorted, here;
    int down_tile, cluster, up_tile, parts;
    int64_t down_blocks, up_blocks;
};

int64_t low_columns(int64_t r) { return r <= 16 ? 16 : ceil_div(r, 32) * 32; }

// S's terms; of sorted rows their tiles (a row each at most, and one before them) and their order.
int64_t low_bytes(int64_t M, int64_t r) { return M * low_columns(r) * 4; }
int64_t workspace_of(int64_t M, int64_t r) { return low_bytes(M, r) + (M > kHere ? 16 * (M + 1) + 4 * M : 0); }

// The product down to the rank: X's columns are shared out to a cluster, down to a step for each of its warps, as far as
// clusters for all tiles run at once (at_once[size] of them).  The product up to D: a tile's columns to `parts` blocks,
// as many as run at once.
Plan make_plan(int64_t M, int64_t N, int64_t K, int64_t r, int64_t adapters, int64_t ldx, int64_t ld, int sms, bool shift,
               const int64_t (&at_once)[9]) {
    Plan pl;
    const int64_t slots = 2 * sms, places = (shift || r > 16 ? 2 : 3) * sms;
    const int64_t steps = ceil_div(K, kStep), turns = ceil_div(N, kWarps * kColumns), rows = 8 * turn_units(r <= 16 ? 1 : 2);
    pl.here = M <= kHere;
    // (sorted rows are counted from the matrix's first: its distances are within 32 bits)
    pl.sorted = adapters > 0 && M >= kHereFrom && adapters <= (pl.here ? kMaxHere : kMaxSorted) && M * std::max(ldx, ld) <= kMaxDim;
    if (pl.sorted) {
        pl.down_tile = pl.up_tile = rows;
        // How many tiles there are is known on the GPU only.  Here: as many adapters as would be met if each row chose
        // one at random, and two standard deviations, each with a last tile that is half full, or with one.  (With a
        // tile more than clusters at once the launch takes two turns: 1000 rows in 37 tiles, with clusters of eight, of
        // which 36 run at once, 18 us, of seven 16.5.)
        const int64_t full = ceil_div(M, rows), most = full + std::min(adapters, M) + 1;
        const double none = std::exp(-static_cast<double>(M) / adapters);
        const double met = adapters * (1.0 - none) + 2.0 * std::sqrt(adapters * none * (1.0 - none));
        const int64_t likely = std::min(most, static_cast<int64_t>(std::max(met, full + 0.5 * met)) + 1);
        pl.cluster = static_cast<int>(std::min<int64_t>(8, ceil_div(steps, kWarps)));
        while (pl.cluster > 1 && at_once[pl.cluster] < likely) --pl.cluster;
        pl.down_blocks = std::min(most, at_once[pl.cluster]) * pl.cluster;
        pl.parts = 0;  // (as many as the tiles leave room for, known then)
        pl.up_blocks = std::min(most * turns, places);
        return pl;
    }
    pl.cluster = 1;
    while (pl.cluster < 8 && pl.cluster * kWarps < steps) pl.cluster *= 2;
    while (pl.cluster > 1 && ceil_div(M, slots / pl.cluster) > rows) pl.cluster /= 2;
    pl.down_tile = static_cast<int>(std::min(rows, ceil_div(M, slots / pl.cluster)));
    while (pl.down_tile > 1 && pl.down_tile * ldx > kMaxDim) pl.down_tile /= 2;  // (the kernels' distances within a tile)
    pl.down_blocks = ceil_div(M, pl.down_tile) * pl.cluster;
    // Few rows are requests of a token each, with adapters of their own as a rule: a tile each.
    pl.up_tile = M < kHereFrom ? 1 : kMaxTile;
    while (pl.up_tile > 1 && pl.up_tile * ld > kMaxDim) pl.up_tile /= 2;
    const int64_t up_tiles = ceil_div(M, pl.up_tile);
    pl.parts = static_cast<int>(ceil_div(turns, ceil_div(turns, std::max<int64_t>(1, places / up_tiles))));
    pl.up_blocks = up_tiles * pl.parts;
    return pl;
}

size_t down_smem(int teams) { return static_cast<size_t>(kWarps + 2 * teams) * kSums * 4; }

using UpKernel = void (*)(Params);

template <bool SHIFT>
UpKernel up_kernel_for(int ldlow) {
    return ldlow <= 16 ? up_kernel<16, 1, SHIFT> : ldlow == 32 ? up_kernel<32, 1, SHIFT> : ldlow == 64 ? up_kernel<32, 2, SHIFT>
                                                                                          : up_kernel<32, 0, SHIFT>;
}

}  // namespace

extern "C" {

gb_status_t gb_lora_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t r, size_t* bytes) {
    clear_error();
    if (!bytes) return fail(GB_ERR_INVALID_ARG, "bytes is null");
    *bytes = 0;
    const gb_status_t st = check_sizes(M, N, K, r, 0);
    if (st == GB_OK && M > 0 && N > 0 && K > 0 && r > 0) *bytes = static_cast<size_t>(workspace_of(M, r));
    return st;
}

gb_status_t gb_lora(const void* X, int64_t ldx, const void* A, int64_t lda, int64_t apart_a, const void* B, int64_t ldb,
                    int64_t apart_b, const int32_t* ids, const float* scale, const void* R, int64_t ldr, int act, void* D,
                    int64_t ldd, void* workspace, size_t workspace_bytes, int64_t M, int64_t N, int64_t K, int64_t r,
                    int64_t adapters, void* stream) {
    clear_error();
    gb_status_t st = check_sizes(M, N, K, r, adapters);
    if (st != GB_OK) return st;
    if (act < GB_ACT_NONE || act > GB_ACT_RELU) return fail(GB_ERR_INVALID_ARG, "unknown activation %d", act);
    if (M == 0 || N == 0) {
        note_empty();
        return GB_OK;
    }
    if (!D) return fail(GB_ERR_INVALID_ARG, "D is null");
    if (ldd < N) return fail(GB_ERR_INVALID_ARG, "leading dimension %" PRId64 " of D is below its row length %" PRId64, ldd, N);
    if (R && ldr < N) return fail(GB_ERR_INVALID_ARG, "leading dimension %" PRId64 " of R is below its row length %" PRId64, ldr, N);
    if (!aligned_to(D, 2) || !aligned_to(R, 2)) return fail(GB_ERR_UNSUPPORTED, "D and R must be 2-byte aligned");
    if (!ids) return fail(GB_ERR_INVALID_ARG, "ids is null");
    if (!aligned_to(ids, 4) || !aligned_to(scale, 4)) return fail(GB_ERR_UNSUPPORTED, "ids and scale must be 4-byte aligned");
    const bool any = K > 0 && r > 0 && adapters > 0;  // (else D = act(R))
    if (any) {
        struct {
            const char* name;
            const void* p;
            int64_t ld, rows, cols, apart, count;
        } mats[] = {{"X", X, ldx, M, K, 0, 1}, {"A", A, lda, r, K, apart_a, adapters}, {"B", B, ldb, N, r, apart_b, adapters}};
        for (const auto& m : mats) {
            if (!m.p) return fail(GB_ERR_INVALID_ARG, "%s is null", m.name);
            if (m.ld < m.cols)
                return fail(GB_ERR_INVALID_ARG, "leading dimension %" PRId64 " of %s is below its row length %" PRId64, m.ld,
                            m.name, m.cols);
            if (!aligned_to(m.p, 16) || (m.rows > 1 && m.ld % 8))  // (one row has no next one)
                return fail(GB_ERR_UNSUPPORTED, "%s: base address and rows must be 16-byte aligned (leading dimension %" PRId64
                                                ")", m.name, m.ld);
            if (m.count > 1 && (m.apart % 8 || m.apart < (m.rows - 1) * m.ld + m.cols))
                return fail(m.apart % 8 ? GB_ERR_UNSUPPORTED : GB_ERR_INVALID_ARG,
                            "%s: adapters %" PRId64 " elements apart (a multiple of 8, and at least a matrix)", m.name, m.apart);
        }
    }
    // (the distance of rows says nothing of one row)
    if (M == 1) ldx = K, ldr = N, ldd = N;
    if (r == 1) lda = K;
    if (N == 1) ldb = r;
    if (any && (r - 1) * lda + K > kMaxDim)  // (distances within a matrix are counted in 32 bits)
        return fail(GB_ERR_UNSUPPORTED, "A: %" PRId64 " rows %" PRId64 " elements apart are more than 2^31 elements", r, lda);
    if (any && kColumns * ldb > kMaxDim) return fail(GB_ERR_UNSUPPORTED, "leading dimension %" PRId64 " of B: below 2^26", ldb);
    int dev = 0;
    DeviceInfo info;
    if ((st = device_info(&dev, &info)) != GB_OK) return st;
    const bool wide_r = aligned_to(R, 16) && (M == 1 || ldr % 8 == 0), wide_d = aligned_to(D, 16) && (M == 1 || ldd % 8 == 0);
    const bool shift = !(wide_d && (wide_r || !R));  // rows start anywhere
    // the ranks of a warp in the product down, and the warps that share the rank
    const int tiles = r <= 16 ? 1 : 2;
    int teams = 1;
    while (teams < kWarps && teams * 16 * tiles < r) teams *= 2;
    const auto down = tiles == 1 ? down_kernel<1> : down_kernel<2>;
    int64_t at_once[9] = {};
    if (any) {
        static std::atomic<bool> ready[2][64];
        static ClusterCounts counts[2];
        const size_t most = down_smem(tiles == 1 ? 1 : kWarps);
        if ((st = allow_smem(down, ready[tiles - 1], dev, most)) != GB_OK) return st;
        for (int size = 1; size <= 8; ++size)
            if ((st = counts[tiles - 1].get(down, kThreads, most, dev, size, &at_once[size])) != GB_OK) return st;
    }
    const Plan pl =
        make_plan(M, N, K, r, any ? adapters : 0, any ? ldx : 0, std::max(ldd, R ? ldr : 0), info.sms, shift, at_once);
    if (pl.down_blocks > kMaxDim || pl.up_blocks > kMaxDim)
        return fail(GB_ERR_UNSUPPORTED, "%" PRId64 " rows of %" PRId64 " columns are more than a launch's blocks", M, N);
    const size_t need = any ? static_cast<size_t>(workspace_of(M, r)) : 0;
    if (need && (!workspace || workspace_bytes < need))
        return fail(GB_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace ? workspace_bytes : size_t(0), need);
    if (need && !aligned_to(workspace, 16)) return fail(GB_ERR_INVALID_ARG, "workspace must be 16-byte aligned");

    Params prm{};
    prm.x = static_cast<const uint16_t*>(X);
    prm.a = static_cast<const uint16_t*>(A);
    prm.b = static_cast<const uint16_t*>(B);
    prm.ids = ids;
    prm.scale = scale;
    prm.r = static_cast<const uint16_t*>(R);
    prm.d = static_cast<uint16_t*>(D);
    prm.low = static_cast<uint16_t*>(workspace);
    prm.ldx = ldx;
    prm.lda = lda;
    prm.ldb = ldb;
    prm.ldr = ldr;
    prm.ldd = ldd;
    prm.apart_a = apart_a;
    prm.apart_b = apart_b;
    prm.m = static_cast<int>(M);
    prm.n = static_cast<int>(N);
    prm.k = static_cast<int>(K);
    prm.rank = static_cast<int>(r);
    prm.adapters = any ? static_cast<int>(adapters) : 0;
    prm.ldlow = any ? static_cast<int>(low_columns(r)) : 0;
    prm.act = act;
    prm.cluster = pl.cluster;
    prm.parts = pl.parts;
    prm.up_blocks = static_cast<int>(pl.up_blocks);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    prm.here = pl.sorted && pl.here;
    if (pl.sorted && !pl.here) {
        int4* tiles = reinterpret_cast<int4*>(static_cast<uint8_t*>(workspace) + low_bytes(M, r));
        int32_t* order = reinterpret_cast<int32_t*>(tiles + M + 1);
        prm.tile = pl.down_tile;
        st = Launch(1, kSortThreads, (adapters + 1) * sizeof(int), s)("lora sort launch", sort_kernel, prm, tiles, order);
        if (st != GB_OK) return st;
        prm.tiles = tiles;
        prm.order = order;
    }
    if (any) {
        prm.teams = teams;
        prm.tile = pl.down_tile;
        st = Launch(static_cast<unsigned>(pl.down_blocks), kThreads, down_smem(teams), s, pl.cluster)("lora down launch", down,
                                                                                                     prm);
        if (st != GB_OK) return st;
    }
    prm.tile = pl.up_tile;
    note_plan("kernel=lora sorted=%lld tile=%lld cluster=%lld down_blocks=%lld up_blocks=%lld shifted=%lld", pl.sorted + prm.here,
              pl.down_tile, pl.cluster, any ? pl.down_blocks : 0, pl.up_blocks, shift);
    const UpKernel kernel = shift ? up_kernel_for<true>(prm.ldlow) : up_kernel_for<false>(prm.ldlow);
    if (prm.ldlow > 64) {  // (less is within what any kernel may have)
        static std::atomic<bool> ready[2][64];
        if ((st = allow_smem(kernel, ready[shift], dev, kMaxTile * low_words(kMaxRank) * 4)) != GB_OK) return st;
    }
    const size_t smem = static_cast<size_t>(pl.up_tile) * low_words(prm.ldlow) * 4;
    return Launch(static_cast<unsigned>(pl.up_blocks), kThreads, smem, s)("lora up launch", kernel, prm);
}

}  // extern "C"
