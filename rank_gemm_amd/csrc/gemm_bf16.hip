// Base GEMM of the LoRA linear on gfx950 matrix cores, with the SGMV expand
// fused into its epilogue:
//   y[t_p] = bf16( x[t_p] W^T + scale_s * h[p] B_s^T )   for sorted position p
// where t_p = token_order[p] and s is the slot whose segment holds p. The base
// product is the plain GEMM of "LoRA serving, embeddings, rerankers, pooling"
// (mlinterviewnotes.com, opening section: base GEMM once over the batch, then
// the per-row indexed low-rank correction); doing the correction in the
// epilogue writes y once instead of re-reading it.
//
// Rows are visited in plan (segment) order, so a 16-row block meets few
// slots: each slot met adds one more rank-deep product per block, with h
// (fp32, from the shrink) fed to the matrix cores as bf16 hi + lo halves.
// Rows on slot 0, or on a rank-0 slot, get no product at all, so their bits
// equal those of a run with no adapter row.
//
// Two paths, chosen by (T, d_out) only:
//  * tiled (T above decode sizes, this file): one kernel template with K in
//    stages of 64 through an LDS ring filled by direct-to-LDS loads; the
//    macro tile is the one of 256 x 256 (4 waves), 256 x 128, 128 x 128 and
//    64 x 128 (8 waves) that takes the fewest rounds of 256 tiles times the
//    tile's time. The shrink runs before it as its own kernel.
//  * split-K (decode-sized T, splitk.hip): a K-split GEMM with the shrink in
//    extra workgroups of the same launch, then a kernel that adds the splits
//    and applies the expand.
#include "../../include/lora.h"
#include "gemm_tile.h"
#include "shrink.h"

namespace lora {

template <int BM, int BN, int WM, int WN, int NS, bool EPI, bool KTAIL, bool SPLIT, bool BUF>
__global__ __launch_bounds__(64 * WM * WN, 1) __attribute__((amdgpu_waves_per_eu(WM * WN / 4, WM * WN / 4))) void gemm_tile_kernel(
    const uint16_t* __restrict__ X, const uint16_t* __restrict__ W, uint16_t* __restrict__ Y, int M, int N, int K,
    int tiles_m, int tiles_n, Fuse f, SplitOut so) {
    gemm_tile<BM, BN, WM, WN, NS, EPI, KTAIL, SPLIT, BUF, false>(X, W, Y, M, N, K, tiles_m, tiles_n, f, so);
}

// ------------------------------------------------------------------ plan --
GemmPlan gemm_bf16_plan(int M, int N, int K) {
    GemmPlan g{};
    if (M <= 0 || N <= 0 || K <= 0) return g;  // nothing to launch
    // tiled path: the macro tile with the least (rounds of 256 tiles) x (time
    // of one tile); the relative tile times are measured ones (K = 4096:
    // 256 x 256 96.5 us, 256 x 128 55 us, 128 x 128 39.5 us, 64 x 128 30 us)
    auto n_tiles = [&](int bm, int bn) { return (int64_t)cdiv(M, bm) * cdiv(N, bn); };
    if (n_tiles(256, 256) >= 200 || (M > 256 && n_tiles(64, 128) >= 128)) {
        struct Cand {
            int bm, bn;
            double t;
        };
        constexpr Cand cands[] = {{256, 256, 96.5}, {256, 128, 55.0}, {128, 128, 39.5}, {64, 128, 30.0}};
        double best = 0.0;
        for (const Cand& c : cands) {
            const double cost = (double)((n_tiles(c.bm, c.bn) + 255) / 256) * c.t;
            if (g.bm == 0 || cost < best) {
                best = cost;
                g.bm = c.bm;
                g.bn = c.bn;
            }
        }
        // or 256 x 128 tiles split over K (few tiles, long K): each split's
        // tile time scales with its k range, plus its fp32 partial writes (at
        // 5 TB/s) and ~7 us of fill and drain; then the reduction reads the
        // partials and writes y (at 4.4 TB/s, + 1 us). Measured at T = 512:
        // 14336 -> 4096 split 4 ways 63 + 7 us against ~105 us unsplit;
        // 4096 -> 4096 stays unsplit (33 us).
        const double plain = best * K / 4096.0;
        double best_split = 0.9 * plain;  // taken only when clearly cheaper
        for (int ks = 2; ks <= 8; ks *= 2) {
            const int kc = cdiv(cdiv(K, ks), 64) * 64;
            const int kse = cdiv(K, kc);
            if (kc < 512 || kse < 2) break;
            const double part_bytes = kse * (double)M * N * 4.0;
            const double cost = (double)((n_tiles(256, 128) * kse + 255) / 256) * 55.0 * kc / 4096.0 +
                                part_bytes / 5.0e6 + 7.0 + (part_bytes + (double)M * N * 2.0) / 4.4e6 + 1.0;
            if (cost < best_split) {
                best_split = cost;
                g.tks = kse;
                g.tkc = kc;
            }
        }
        return g;
    }
    // split-K: 64 x 64 tiles, enough K splits for ~256 workgroups
    g.bm = 64; g.bn = 64;
    g.n_mt = cdiv(M, 64);
    g.n_nt = cdiv(N, 64);
    const int tiles = g.n_mt * g.n_nt;
    const int want = tiles >= 256 ? 1 : cdiv(256, tiles);
    const int need = cdiv(cdiv(K, want), 128);  // sub-chunks per split
    int nsub = 1;
    while (nsub < need && nsub < 16) nsub *= 2;
    g.nsub = nsub;
    g.ks = cdiv(K, nsub * 128);
    return g;
}

// Workspace of the split-K pass over all slices together.
static size_t split_workspace(int M, int n_nt_total, const GemmPlan& g, int n_slices, int r_max) {
    const size_t py = (size_t)g.ks * g.n_mt * n_nt_total * 16 * 64 * 16;
    // h planes: the GEMM's ks splits (shrink tiles) or up to 8 shrink splits
    const size_t ph = (size_t)n_slices * max(g.ks, 8) * M * r_max * sizeof(float);
    return ((py + 255) & ~size_t(255)) + ((ph + 255) & ~size_t(255));
}

// tiled path: fp32 h [M][r_max] or bf16 hi / lo [M][2][round_up(r_max, 8)],
// then the K-split shrink's planes (at most kShrinkSplitMaxBlocks x 16 rows)
size_t tiled_workspace(int M, int r_max) {
    const size_t h_final = (size_t)M * ((r_max + 7) & ~7) * sizeof(float);
    const size_t planes = (size_t)kShrinkSplitMaxBlocks * 16 * r_max * sizeof(float);
    return ((h_final + 255) & ~size_t(255)) + planes;
}

// one slice's expand operand (bf16 hi / lo, [M][2][rp]) in the workspace
static size_t ext_stride(int M, int r_max) {
    return ((size_t)M * ((r_max + 7) & ~7) * sizeof(float) + 255) & ~size_t(255);
}

static int total_tiles_n(const int* N, int n_slices) {
    int t = 0;
    for (int i = 0; i < n_slices; ++i) t += cdiv(N[i], 64);
    return t;
}

// Slices share one pass when their concatenated columns take the split-K
// path; otherwise each slice runs on its own (tiled or split-K).
static bool joint_split(int M, const int* N, int n_slices, int K, GemmPlan* out) {
    int n_total = 0;
    for (int i = 0; i < n_slices; ++i) n_total += N[i];
    const GemmPlan g = gemm_bf16_plan(M, n_total, K);
    if (out) *out = g;
    return g.nsub != 0;
}

// tiled path split over K: the partials, then the tiled path's h area
static size_t split_tiled_workspace(int M, int N, const GemmPlan& g, int r_max) {
    const size_t py = ((size_t)g.tks * cdiv(M, 64) * cdiv(N, 64) * 16 * 64 * 16 + 255) & ~size_t(255);
    return py + tiled_workspace(M, r_max);
}

size_t gemm_bf16_workspace(int M, const int* N, int n_slices, int K, int r_max) {
    if (M <= 0 || K <= 0 || n_slices < 1) return 0;
    GemmPlan gj;
    if (n_slices > 1 && joint_split(M, N, n_slices, K, &gj)) {
        // the joint plan's tiles are those of the concatenated columns;
        // count whole 64-column tiles per slice
        GemmPlan g = gj;
        g.n_nt = total_tiles_n(N, n_slices);
        return split_workspace(M, g.n_nt, g, n_slices, r_max);
    }
    // several slices may share one shrink: an expand operand area per slice
    size_t need = n_slices > 1 ? n_slices * ext_stride(M, r_max) : 0;
    for (int i = 0; i < n_slices; ++i) {
        if (N[i] <= 0) continue;
        const GemmPlan g = gemm_bf16_plan(M, N[i], K);
        const size_t b = g.nsub != 0 ? split_workspace(M, g.n_nt, g, 1, r_max)
                         : g.tks > 1 ? split_tiled_workspace(M, N[i], g, r_max)
                                     : tiled_workspace(M, r_max);
        need = b > need ? b : need;
    }
    return need;
}

template <int BM, int BN, int WM, int WN, int NS, bool SPLIT_OK, bool BUF_OK = false>
static hipError_t launch_tile(const uint16_t* X, const uint16_t* W, uint16_t* Y, int M, int N, int K, const Fuse& f,
                            bool epi, hipStream_t st, StageTimer* tm, const SplitOut& so = SplitOut{}, int ks = 1) {
    const int tiles_m = cdiv(M, BM), tiles_n = cdiv(N, BN);
    const bool ktail = K % 64 != 0;
    const dim3 block(64 * WM * WN);
    decltype(&gemm_tile_kernel<BM, BN, WM, WN, NS, false, false, false, false>) ker;
    if constexpr (SPLIT_OK) {
        if (so.part) {
            ker = ktail ? gemm_tile_kernel<BM, BN, WM, WN, NS, false, true, true, false>
                        : gemm_tile_kernel<BM, BN, WM, WN, NS, false, false, true, false>;
            return launch(tm, "gemm_bf16", ker, dim3(tiles_m * tiles_n * ks), block, st, X, W, Y, M, N, K, tiles_m,
                          tiles_n, f, so);
        }
    }
    bool buf = false;
    if constexpr (BUF_OK) buf = tile_buffers_fit(M, N, K, BN, f);
    if (buf) {
        if constexpr (BUF_OK)
            ker = epi ? (ktail ? gemm_tile_kernel<BM, BN, WM, WN, NS, true, true, false, true>
                               : gemm_tile_kernel<BM, BN, WM, WN, NS, true, false, false, true>)
                      : (ktail ? gemm_tile_kernel<BM, BN, WM, WN, NS, false, true, false, true>
                               : gemm_tile_kernel<BM, BN, WM, WN, NS, false, false, false, true>);
    } else {
        ker = epi ? (ktail ? gemm_tile_kernel<BM, BN, WM, WN, NS, true, true, false, false>
                           : gemm_tile_kernel<BM, BN, WM, WN, NS, true, false, false, false>)
                  : (ktail ? gemm_tile_kernel<BM, BN, WM, WN, NS, false, true, false, false>
                           : gemm_tile_kernel<BM, BN, WM, WN, NS, false, false, false, false>);
    }
    return launch(tm, "gemm_bf16", ker, dim3(tiles_m * tiles_n), block, st, X, W, Y, M, N, K, tiles_m, tiles_n, f,
                  SplitOut{});
}

// The shrink of the tiled path, into fp32 h [M][r_max] or, with ext, the
// expand operand of the extra K steps; ws: h_final bytes for h or ext, then
// the K-split shrink's planes.
static hipError_t tiled_shrink(const LinearArgs& L, const SliceArgs& sl, char* ws, float* h, uint16_t* ext,
                               hipStream_t st, StageTimer* tm) {
    const int M = L.M, K = L.K;
    // few items over a long K: split K over more workgroups, then add the splits
    int hs = 1, hkc = K;
    if (L.n_items < kShrinkSplitMaxBlocks / 2) {
        hs = min(8, kShrinkSplitMaxBlocks / max(L.n_items, 1));
        hkc = max(256, (cdiv(K, hs) + 31) / 32 * 32);
        hs = cdiv(K, hkc);
    }
    const size_t h_final = (size_t)M * ((L.r_max + 7) & ~7) * sizeof(float);
    float* part = reinterpret_cast<float*>(ws + ((h_final + 255) & ~size_t(255)));
    return hs > 1 ? sgmv_shrink_split(L.X, sl.A_pool, sl.rank, sl.scale, L.token_order, L.work, L.n_items, hs, hkc,
                                      part, h, ext, K, L.r_max, st, tm)
                  : sgmv_shrink(L.X, sl.A_pool, sl.rank, L.token_order, L.work, L.n_items, h, K, L.r_max, st, tm,
                                sl.scale, ext);
}

// Whether a slice whose plan splits K runs split: where the pool has the
// extra-step form of the expand (r_max % 8 == 0, at most kMetaSlots slots) and
// those steps would add at most 3/8 to a split's. By the sizes and the pool
// alone, not by the batch's plan or adapters: the split is the order in which
// y's sums are taken, and rows without an adapter keep a base-only call's bits.
// Split against unsplit, 769 x 8200 -> 1500: 128 slots of rank 16 (0.22) 69
// against 85 us, 17 of rank 64 (0.26) 74 against 94; 512 x 14336 -> 4096: 64 of
// rank 32 (0.21) 92 against 95, 256 of rank 16 (0.32) 134 against 121 with all in
// use, 78 against 85 with 9; 512 of rank 16 (0.61) 172 against 171.
static bool split_runs(const GemmPlan& g, int M, int S, int r_max) {
    if (g.tks < 2 || r_max % 8 != 0 || S > kMetaSlots) return false;
    // extra steps per 256-row tile, from the work items (16 rows of one slot
    // each) that M rows over S slots can have in 256 rows (64 / (2 rp) slots
    // share a step when 2 rp divides 64)
    const int64_t items_per_tile = ((int64_t)lora_plan_max_items(M, S) * 256 + M - 1) / M;
    const int64_t slots_per_tile = items_per_tile < S ? items_per_tile : S;
    const int r2 = 2 * r_max;
    const int64_t est_extra = 64 % r2 == 0 ? (slots_per_tile * r2 + 63) / 64 : slots_per_tile * cdiv(r2, 64);
    return est_extra * 8 <= (int64_t)g.tks * (g.tkc / 64) * 3;
}

// One slice on the tiled path split over K: the shrink to the expand operand,
// the 256 x 128 kernel writing partials (the extra K steps dealt round the
// splits), then the split-K path's kernel 2 without adapters (adds the
// partials, rounds).
static hipError_t split_tiled_forward(const LinearArgs& L, const SliceArgs& sl, const GemmPlan& g, hipStream_t st,
                                      StageTimer* tm) {
    const int M = L.M, N = sl.N, K = L.K;
    const int n_mt = cdiv(M, 64), n_nt = cdiv(N, 64);
    char* ws = static_cast<char*>(L.workspace);
    const size_t py = ((size_t)g.tks * n_mt * n_nt * 16 * 64 * 16 + 255) & ~size_t(255);
    float* part = reinterpret_cast<float*>(ws);
    uint16_t* ext = reinterpret_cast<uint16_t*>(ws + py);
    if (L.adapters) {
        const hipError_t e = tiled_shrink(L, sl, ws + py, nullptr, ext, st, tm);
        if (e != hipSuccess) return e;
    }
    const Fuse f{L.token_order, L.slot_indptr, nullptr, sl.B_pool, sl.rank, sl.scale, L.S, L.r_max, 1, 0, L.adapters,
                 ext, (L.r_max + 7) & ~7};
    const hipError_t e =
        launch_tile<256, 128, 4, 2, 3, true>(L.X, sl.W, nullptr, M, N, K, f, false, st, tm, SplitOut{part, g.tkc, n_mt, n_nt},
                                     g.tks);
    if (e != hipSuccess) return e;
    LinearArgs base = L;
    base.adapters = 0;
    return splitk_finish_bf16(base, sl, part, g.tks, n_mt, nullptr, 1, st, tm);
}

// One slice on the tiled path: the shrink to final h, then the tiled GEMM
// with the expand fused (r_max % 8 == 0: as extra K steps from scaled h as
// bf16 hi / lo; otherwise in the epilogue from fp32 h). With ext_ready the
// expand operand was already written there (several slices, one shrink).
static hipError_t tiled_forward(const LinearArgs& L, const SliceArgs& sl, const GemmPlan& g, hipStream_t st,
                                StageTimer* tm, uint16_t* ext_ready = nullptr) {
    if (split_runs(g, L.M, L.S, L.r_max)) return split_tiled_forward(L, sl, g, st, tm);
    const int M = L.M, N = sl.N, K = L.K;
    Fuse f{L.token_order, L.slot_indptr, nullptr, sl.B_pool, sl.rank, sl.scale, L.S, L.r_max, 1, 0, L.adapters,
           nullptr, (L.r_max + 7) & ~7};
    char* ws = static_cast<char*>(L.workspace);
    float* hbuf = reinterpret_cast<float*>(ws);
    // the expand as extra K steps needs r_max % 8 == 0 and the slot metadata in LDS
    uint16_t* ext = (L.r_max % 8 == 0 && L.S <= kMetaSlots) ? reinterpret_cast<uint16_t*>(ws) : nullptr;
    if (ext_ready) ext = ext_ready;
    f.h = ext ? nullptr : hbuf;
    f.ext = ext;
    if (L.adapters && !ext_ready) {
        const hipError_t e = tiled_shrink(L, sl, ws, ext ? nullptr : hbuf, ext, st, tm);
        if (e != hipSuccess) return e;
    }
    const bool epi = L.adapters && !f.ext;
    if (g.bm == 256 && g.bn == 256) return launch_tile<256, 256, 2, 2, 2, false, true>(L.X, sl.W, sl.Y, M, N, K, f, epi, st, tm);
    if (g.bm == 256) return launch_tile<256, 128, 4, 2, 3, false>(L.X, sl.W, sl.Y, M, N, K, f, epi, st, tm);
    if (g.bm == 128) return launch_tile<128, 128, 2, 4, 3, false>(L.X, sl.W, sl.Y, M, N, K, f, epi, st, tm);
    return launch_tile<64, 128, 2, 4, 4, false>(L.X, sl.W, sl.Y, M, N, K, f, epi, st, tm);
}

// Several slices that all take the unsplit tiled path with the expand as
// extra K steps share one shrink (x rows read once), each slice's operand in
// its own workspace area; enough items that the single-slice shrink would not
// split K either, so each operand equals that slice's own bit for bit.
static bool slices_share_shrink(const LinearArgs& L, const int* N, GemmPlan* gs) {
    if (L.n_slices < 2 || !L.adapters || L.r_max % 8 != 0 || L.S > kMetaSlots ||
        L.n_items < kShrinkSplitMaxBlocks / 2)
        return false;
    for (int i = 0; i < L.n_slices; ++i) {
        if (N[i] <= 0) return false;
        gs[i] = gemm_bf16_plan(L.M, N[i], L.K);
        if (gs[i].nsub != 0 || gs[i].tks > 1) return false;
    }
    return true;
}

// One slice on the unsplit tiled path (the caller's choice of sizes) whose
// expand operand was already written to ext.
hipError_t tiled_forward_ready(const LinearArgs& L, const SliceArgs& s, uint16_t* ext, hipStream_t st,
                               StageTimer* tm) {
    return tiled_forward(L, s, gemm_bf16_plan(L.M, s.N, L.K), st, tm, ext);
}

hipError_t lora_forward_bf16(const LinearArgs& L, hipStream_t st, StageTimer* tm) {
    const int M = L.M, K = L.K, n = L.n_slices;
    if (M == 0 || n < 1) return hipSuccess;
    int N[kMaxSlices];
    for (int i = 0; i < n; ++i) N[i] = L.slice[i].N;
    GemmPlan gj;
    if (n > 1 && joint_split(M, N, n, K, &gj)) return splitk_forward_bf16(L, gj, st, tm);
    GemmPlan gs[kMaxSlices];
    if (slices_share_shrink(L, N, gs)) {
        ShrinkSlices ss{};
        ss.n = n;
        char* ws = static_cast<char*>(L.workspace);
        for (int i = 0; i < n; ++i) {
            ss.A_pool[i] = L.slice[i].A_pool;
            ss.rank[i] = L.slice[i].rank;
            ss.scale[i] = L.slice[i].scale;
            ss.ext[i] = reinterpret_cast<uint16_t*>(ws + i * ext_stride(M, L.r_max));
        }
        hipError_t e = sgmv_shrink_slices(L.X, ss, L.token_order, L.work, L.n_items, K, L.r_max, st, tm);
        for (int i = 0; i < n && e == hipSuccess; ++i) e = tiled_forward(L, L.slice[i], gs[i], st, tm, ss.ext[i]);
        return e;
    }
    for (int i = 0; i < n; ++i) {
        if (N[i] == 0) continue;
        const GemmPlan g = gemm_bf16_plan(M, N[i], K);
        hipError_t e;
        if (g.nsub == 0) {
            e = tiled_forward(L, L.slice[i], g, st, tm);
        } else {
            LinearArgs one = L;
            one.n_slices = 1;
            one.slice[0] = L.slice[i];
            e = splitk_forward_bf16(one, g, st, tm);
        }
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace lora
