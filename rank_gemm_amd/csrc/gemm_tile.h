// The pipelined tile of the tiled GEMMs: bf16 (gemm_bf16.hip) and MXFP4
// (mx4_gemm.hip) base products, the expand as extra K steps or in the epilogue.
#pragma once

#include "fuse.h"
#include "mx4_format.h"

#include <type_traits>
#include <utility>

namespace lora {

// --------------------------------------------- tiled, direct-to-LDS loads --
// BM x BN macro tiles over WM x WN waves, wave tile (BM / WM) x (BN / WN) of
// 16 x 16 MFMA tiles; K in stages of 64 through NS LDS buffers, filled by
// direct-to-LDS loads (global_load_lds_dwordx4: 16 B per lane, written at the
// instruction's LDS base + 16 * lane). A row of a stage is one 128-byte line
// (8 chunks of 16 B). Rows go in groups of 64; load instruction q (0..7) of a
// group fetches rows q, q + 8, ..., q + 56, the 8 lanes 8 i .. 8 i + 7 one
// whole line of row q + 8 i, so the instruction's 1 KB lands at q * 1024 in
// the group. Lane 8 i + j takes chunk j ^ q of its row (the XOR swizzle of
// the chunk by the row's index within its 8-row stripe): the MFMA fragment
// read of chunk c over 16 consecutive rows then finds their pieces at 16
// distinct 16-byte slots of one aligned 256-byte window modulo 1 KB, which
// this LDS serves in the minimum 4 cycles per ds_read_b128. (Rows merely
// padded apart by 16 bytes spread those pieces over two windows for chunks
// past the first: 8 cycles per read.)
// The fragment reads are issued and waited on by hand: with LDS loads in
// flight the compiler would wait for all of them at the first use.
constexpr int kInstrBytes = 1024;              // 1 KB of 8 rows
constexpr int kGroupBytes = 8 * kInstrBytes;   // 64 rows

// byte offset of the 16-row block starting at row r0 (r0 % 16 == 0)
__host__ __device__ constexpr int block_off(int r0) { return (r0 / 64) * kGroupBytes + (r0 % 64) / 8 * 128; }

// ------------------------------------------------- the pipelined tile --
// Each wave owns a (BM / WM) x (BN / WN) block of 16 x 16 MFMA tiles (fp32
// accumulators in AGPRs) and keeps its matrix core busy by interleaving all
// other work between its MFMAs. A 64-wide step has two 32-wide halves:
//   phase A of step kt: the MFMAs of the first half (fragments F0), one
//     fragment read of the second half (F1) per group of MFMAs;
//   the wave's loads of step kt + 1 landed; barrier;
//   phase B: the MFMAs of F1, one fragment read of step kt + 1's first half
//     per group, and the 1 KB loads of a later step.
// 256 x 256 runs on 4 waves, one per SIMD, with 128 x 128 wave tiles: a step
// reads 2/3 of the LDS bytes of an 8-wave 128 x 64 tiling. The smaller tiles
// run on 8 waves, two per SIMD: with so few MFMAs per phase one wave per SIMD
// hides too little of the fragment reads and barriers (a 4-wave 128 x 128
// took 57.7 us against 47.3 us at T = 1024, 4096 -> 4096).
// The accumulators are tied to AGPRs by issuing these MFMAs as inline asm
// (left to itself the register allocator shuffles accumulators through
// VGPRs at every loop back edge, ~400 copies per stage). The compiler then
// cannot see that those MFMAs read their fragment registers after issue:
// every phase ends by keeping its fragments alive through two s_nop 7, so no
// later instruction writes them while an MFMA may still read them, and 96
// wait states separate the last MFMA from the first read of the accumulators.
__device__ __forceinline__ void mfma_agpr(f32x4& acc, const u32x4& a, const u32x4& b) {
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}
template <int G>
struct Idx {
    static constexpr int v = G;
};
template <class F, int... Gs>
__device__ __forceinline__ void static_for(std::integer_sequence<int, Gs...>, F&& fn) {
    (fn(Idx<Gs>{}), ...);
}
template <int I, int N>
__device__ __forceinline__ void frags_tie(u32x4 (&a)[N]) {
    if constexpr (I < N) {
        asm volatile("" : "+v"(a[I]));
        frags_tie<I + 1, N>(a);
    }
}
template <int I, int N>
__device__ __forceinline__ void frags_use(const u32x4 (&a)[N]) {
    if constexpr (I < N) {
        asm volatile("" ::"v"(a[I]));
        frags_use<I + 1, N>(a);
    }
}
// every LDS read of this wave landed; ties the wait to the fragment
// registers so that no use of them moves above it
template <int N>
__device__ __forceinline__ void frags_landed(u32x4 (&a)[N]) {
    asm volatile("s_waitcnt lgkmcnt(0)" : "+v"(a[0]));
    frags_tie<1, N>(a);
}
// 16 wait states during which the fragment registers stay live: the MFMAs
// issued above may still read them
template <int NA, int NB>
__device__ __forceinline__ void frags_retire(const u32x4 (&a)[NA], const u32x4 (&b)[NB]) {
    asm volatile("s_nop 7\n\ts_nop 7");
    frags_use<0, NA>(a);
    frags_use<0, NB>(b);
}

// The 4-bit product with accumulators in AGPRs, scales in byte SA / SB of sa / sb
template <int SA, int SB>
__device__ __forceinline__ void mfma_mx4_agpr(f32x4& acc, const u32x4& a, const u32x4& b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[%5,%6,0] op_sel_hi:[%7,%8,0] "
                 "cbsz:4 blgp:4"
                 : "+a"(acc)
                 : "v"(a), "v"(b), "v"(sa), "v"(sb), "i"(SA & 1), "i"(SB & 1), "i"(SA >> 1), "i"(SB >> 1));
}
template <int OFF>
__device__ __forceinline__ uint32_t lds_read4(uint32_t addr) {
    uint32_t r;
    asm volatile("ds_read_b32 %0, %1 offset:%2" : "=v"(r) : "v"(addr), "i"(OFF) : "memory");
    return r;
}

// Split over K (mid-sized T): block b takes tile b % n_tiles over the k
// range [kz kc, (kz + 1) kc), kz = b / n_tiles, and writes fp32 partials in
// the layout of the split-K path ([split][64-row tile][64-column tile][16
// blocks of 16 x 16][64 lanes] f32x4, lane l holding rows 4 (l / 16) + e of
// column l % 16). Split 0 also runs the expand's extra K steps, so the
// split-K path's kernel 2 only adds the partials and rounds.
struct SplitOut {
    float* part;     // null: no split
    int kc;          // k per split, a multiple of 64
    int n_mt, n_nt;  // 64 x 64 tile grid of the partials
};

// BM x BN tiles over WM x WN waves with NS stage buffers. With 2 stages, step
// kt + 2 is loaded during step kt into step kt's own buffer, free only in
// phase B. With NS >= 3, step kt + NS - 1 is loaded during step kt into the
// buffer of step kt - 1 (every wave finished reading it before step kt - 1's
// barrier), so its loads are spread over both phases.
// F4: the base product of MXFP4 operands. K counts 16-bit units, as for the
// other loads (a row's bytes / 2: a 64-unit step is 256 codes, 8 blocks), x
// rows are in plan order already, and the 4-bit matrix instruction has the
// operand bytes and the issue time of the bf16 one for four times its
// products, so the pipeline is the same. A step's scales (512 bytes per 64
// rows, mx4_format.h) are one more load of each wave, kept behind the stage's
// rows; the words of a half step are read with its fragments. The expand's
// extra steps stay bf16 products into the same accumulators.
// BUF: loads through buffer resources (x, the tile's W rows, ext, B_pool; the
// host takes this form when each is under 2 GiB): per-lane row offsets set
// once per tile, the base step's k in the uniform offset. Otherwise 64-bit
// addresses, moved by k every step (8192 x 4096 -> 14336: 737-747 us against
// 750-757 us, interleaved on one box, identical outputs).
template <int BM, int BN, int WM, int WN, int NS, bool EPI, bool KTAIL, bool SPLIT, bool BUF, bool F4>
__device__ __forceinline__ void gemm_tile(const uint16_t* __restrict__ X, const uint16_t* __restrict__ W,
                                          uint16_t* __restrict__ Y, int M, int N, int K, int tiles_m, int tiles_n,
                                          const Fuse& f, const SplitOut& so,
                                          const uint8_t* __restrict__ xscales = nullptr,
                                          const uint8_t* __restrict__ wscales = nullptr) {
    static_assert(!(SPLIT && EPI), "a split runs no expand");
    static_assert(!(SPLIT && F4), "4-bit products run unsplit");
    static_assert(!(SPLIT && BUF), "splits take 64-bit addresses");
    constexpr int BK = 64, NW = WM * WN;
    constexpr int FI = BM / WM / 16, FJ = BN / WN / 16;    // MFMA blocks of a wave
    constexpr int DA = BM / 8 / NW, DB = BN / 8 / NW;      // row load instructions of a wave per step
    constexpr int ND = DA + DB + (F4 ? 1 : 0);             // ... and its load of scales
    constexpr int NM = FI * FJ, NR = FI + FJ;              // MFMAs and fragment reads per half step
    constexpr int ABYTES = BM / 64 * kGroupBytes, ROWS16 = (BM + BN) / 64 * kGroupBytes / 16;  // 16-byte units
    constexpr int SG = (BM + BN) / 64, SL = (SG + 1) / 2;  // scales: 64-row groups, loads of two groups
    constexpr int STAGE = ROWS16 + (F4 ? SL * 64 : 0);
    static_assert(BM % 64 == 0 && BN % 64 == 0 && DA * NW * 8 == BM && DB * NW * 8 == BN && NW % 4 == 0, "tile shape");
    constexpr int L = NS >= 3 ? NS - 1 : 2;                // step kt + L is loaded during step kt
    constexpr int NDA = NS >= 3 ? ND / 2 : 0;              // its loads issued in phase A
    constexpr int NDB = ND - NDA;                          // ... and in phase B
    constexpr int VM_MID = (L - 2) * ND + NDA;             // loads younger than step kt + 1's at mid-step
    static_assert(NS >= 2 && VM_MID < 64 && (L - 1) * ND < 64 && NR <= 16, "wait counters");
    __shared__ u32x4 lds[NS * STAGE];
    __shared__ SlotMeta meta;
    __shared__ uint16_t xlist[BM];  // the tile's live slots
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const MetaView mv = stage_meta(f, &meta);
    const int n_tiles = tiles_m * tiles_n;
    const int kz = SPLIT ? (int)blockIdx.x / n_tiles : 0;
    int tm, tn;
    tile_coords(SPLIT ? (int)blockIdx.x - kz * n_tiles : (int)blockIdx.x, tiles_m, tiles_n, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int mend = min(M, m0 + BM);
    const int kb = SPLIT ? kz * so.kc : 0;             // this block's k range [kb, kb + Kr)
    const int Kr = SPLIT ? min(K - kb, so.kc) : K;
    const int nk = (Kr + BK - 1) / BK;
    // load instruction u of the tile fetches rows (u / 8) * 64 + u % 8 + 8 i
    // (rows past M or N are clamped; their outputs are not stored)
    const int rl = lane >> 3, cl = lane & 7;
    int prow[DA], ncol[DB];
    const uint16_t* ap[DA];
    const uint16_t* bp[DB];
#pragma unroll
    for (int b = 0; b < DA; ++b) {
        const int u = wave * DA + b;
        prow[b] = m0 + (u >> 3) * 64 + (u & 7) + 8 * rl;
        const int64_t r = F4 ? min(prow[b], M - 1) : f.token_order[min(prow[b], M - 1)];
        ap[b] = X + r * K + kb + (cl ^ (u & 7)) * 8;
    }
#pragma unroll
    for (int b = 0; b < DB; ++b) {
        const int u = wave * DB + b;
        ncol[b] = n0 + (u >> 3) * 64 + (u & 7) + 8 * rl;
        bp[b] = W + (int64_t)min(ncol[b], N - 1) * K + kb + (cl ^ (u & 7)) * 8;
    }
    // the buffer form's resources and this lane's byte offsets of its rows
    const brsrc rX = make_rsrc(X, (uint32_t)M * (uint32_t)K * 2u);
    const brsrc rW = make_rsrc(W + (int64_t)n0 * K, (uint32_t)(min(N, n0 + BN) - n0) * (uint32_t)K * 2u);
    const brsrc rE = make_rsrc(f.ext, (uint32_t)M * (uint32_t)f.rp * 4u);
    const brsrc rB = make_rsrc(f.B_pool, (uint32_t)f.S * (uint32_t)N * (uint32_t)f.r_max * 2u);
    uint32_t aoff[DA], boff[DB];
    if constexpr (BUF) {
#pragma unroll
        for (int b = 0; b < DA; ++b) {
            const int r = F4 ? min(prow[b], M - 1) : f.token_order[min(prow[b], M - 1)];
            aoff[b] = (uint32_t)(r * K + (cl ^ ((wave * DA + b) & 7)) * 8) * 2u;
        }
#pragma unroll
        for (int b = 0; b < DB; ++b)
            boff[b] = (uint32_t)((min(ncol[b], N - 1) - n0) * K + (cl ^ ((wave * DB + b) & 7)) * 8) * 2u;
    }
    uint32_t vsrc[DA + DB];  // buffer form: per-lane offsets of an extra step, or of a K-tail base step
    uint32_t soff = 0;  // buffer form: the base step's k, in bytes
    __syncthreads();  // slot metadata staged
    // the expand's extra steps; in a split, split kz takes extra steps kz,
    // kz + ks, kz + 2 ks, ... of the tile (the partials carry the correction)
    const int ks = SPLIT ? (int)gridDim.x / n_tiles : 1;
    const lds_meta_ptr lmeta = (lds_meta_ptr)&meta;
    const lds_u16_ptr wlist = (lds_u16_ptr)xlist;
    const ExtraSched xs = extra_schedule(f.adapters && f.ext, lmeta, f.S, m0, mend, f.rp, wlist, wave == 0);
    if (xs.n > 0) __syncthreads();  // the slot list written
    const int ne_all = xs.steps();
    const int ne = __builtin_amdgcn_readfirstlane(SPLIT ? (ne_all > kz ? (ne_all - kz + ks - 1) / ks : 0) : ne_all);
    const int nt = nk + ne;
    // F4: this wave's load of scales, groups 2 u and 2 u + 1 of the stage (x
    // groups, then W groups; waves past the last load repeat one, so that all
    // wait on the same counts), moved by 512 bytes per step
    const int sl = wave % SL;
    const uint8_t* sbase = nullptr;
    gptr<u32x4> ssrc = nullptr;
    uint32_t svoff = 0;  // buffer form: the lane's offset from its operand's first group of the tile
    const bool sx = 2 * sl < BM / 64;  // buffer form: an x load (its groups come in pairs)
    const int sg0 = sx ? m0 / 64 : n0 / 64, sg1 = (sx ? M - 1 : N - 1) / 64;
    const brsrc rS = make_rsrc(F4 ? (sx ? xscales : wscales) + (int64_t)sg0 * nk * kMxTileBytes : nullptr,
                               (uint32_t)(min(sg1 - sg0 + 1, (BM > BN ? BM : BN) / 64) * nk * kMxTileBytes));
    if constexpr (F4) {
        static_assert(!BUF || BM % 128 == 0, "x scale groups in pairs");
        const int g = min(2 * sl + (lane >> 5), SG - 1);
        const int xg = min(m0 / 64 + g, (M - 1) / 64), wg = min(n0 / 64 + g - BM / 64, (N - 1) / 64);
        if constexpr (BUF) {
            svoff = (uint32_t)(((sx ? xg : wg) - sg0) * nk * kMxTileBytes + (lane & 31) * 16);
        } else {
            sbase = (g < BM / 64 ? xscales + (int64_t)xg * nk * kMxTileBytes
                                 : wscales + (int64_t)wg * nk * kMxTileBytes) + (lane & 31) * 16;
            ssrc = as_global<u32x4>(sbase);
        }
    }
    // sources of step kt's load instructions (A 0..DA-1, then B), set once
    // per step
    gptr<u32x4> src[DA + DB];
    // lane cl fetches chunk cl ^ (u % 8) with load instruction u
    auto sources_base = [&](int kt) {
        const int k = (kt - ne) * BK;
        if constexpr (F4 && !BUF) ssrc = as_global<u32x4>(sbase + (int64_t)(kt - ne) * kMxTileBytes);
        if constexpr (BUF) {
            soff = (uint32_t)k * 2u;
            if constexpr (KTAIL) {
#pragma unroll
                for (int b = 0; b < DA; ++b)
                    vsrc[b] = k + (cl ^ ((wave * DA + b) & 7)) * 8 < Kr ? aoff[b] : kOutOfRange;
#pragma unroll
                for (int b = 0; b < DB; ++b)
                    vsrc[DA + b] = k + (cl ^ ((wave * DB + b) & 7)) * 8 < Kr ? boff[b] : kOutOfRange;
            }
            return;
        }
#pragma unroll
        for (int b = 0; b < DA; ++b) {
            const bool kin = !KTAIL || k + (cl ^ ((wave * DA + b) & 7)) * 8 < Kr;
            src[b] = KTAIL ? or_zero(kin, ap[b] + k) : as_global<u32x4>(ap[b] + k);
        }
#pragma unroll
        for (int b = 0; b < DB; ++b) {
            const bool kin = !KTAIL || k + (cl ^ ((wave * DB + b) & 7)) * 8 < Kr;
            src[DA + b] = KTAIL ? or_zero(kin, bp[b] + k) : as_global<u32x4>(bp[b] + k);
        }
    };
    // F4: scale words of a half step, word i for the wave's 16-row blocks
    // 4 i .. 4 i + 3 of x (sA) and W (sB)
    constexpr int GA = (FI + 3) / 4, GB = (FJ + 3) / 4;
    uint32_t sA0[GA], sB0[GB], sA1[GA], sB1[GB];
    const uint32_t sa_off = lds_offset(lds) + ROWS16 * 16 + wm * FI / 4 * kMxTileBytes + lane * 8;
    const uint32_t sb_off = lds_offset(lds) + ROWS16 * 16 + (BM / 64 + wn * FJ / 4) * kMxTileBytes + lane * 8;
    auto read_scales = [&](auto hc, uint32_t (&sa)[GA], uint32_t (&sb)[GB], uint32_t stage) {
        constexpr int h = decltype(hc)::v;
        static_for(std::make_integer_sequence<int, GA>{}, [&](auto ic) {
            sa[decltype(ic)::v] = lds_read4<decltype(ic)::v * kMxTileBytes + 4 * h>(sa_off + stage);
        });
        static_for(std::make_integer_sequence<int, GB>{}, [&](auto ic) {
            sb[decltype(ic)::v] = lds_read4<decltype(ic)::v * kMxTileBytes + 4 * h>(sb_off + stage);
        });
    };
    // after frags_landed: the words' first byte becomes that of the wave's
    // first block (a wave with under four blocks may start inside a group)
    auto scales_landed = [&](uint32_t (&sa)[GA], uint32_t (&sb)[GB]) {
        if constexpr (F4) {
#pragma unroll
            for (int i = 0; i < GA; ++i) asm volatile("" : "+v"(sa[i]));
#pragma unroll
            for (int i = 0; i < GB; ++i) asm volatile("" : "+v"(sb[i]));
            if constexpr (FI < 4) sa[0] >>= 8 * (wm * FI & 3);
            if constexpr (FJ < 4) sb[0] >>= 8 * (wn * FJ & 3);
            // a product issued as asm must not follow the shift at once
            if constexpr (FI < 4 || FJ < 4) asm volatile("s_nop 3" : "+v"(sa[0]), "+v"(sb[0]));
        }
    };
    auto scales_retire = [&](const uint32_t (&sa)[GA], const uint32_t (&sb)[GB]) {
        if constexpr (F4) {
#pragma unroll
            for (int i = 0; i < GA; ++i) asm volatile("" ::"v"(sa[i]));
#pragma unroll
            for (int i = 0; i < GB; ++i) asm volatile("" ::"v"(sb[i]));
        }
    };
    // W is the left operand (acc holds blocks of W x^T, a lane 4 consecutive
    // columns of one row) except in a split, whose partials take the split-K
    // path's orientation (a lane 4 consecutive rows of one column)
    auto mfma = [&](f32x4& c, const u32x4& a, const u32x4& w) {
        if constexpr (SPLIT) mfma_agpr(c, a, w);
        else mfma_agpr(c, w, a);
    };
    // product t of a half step in its tile order; C4: of 4-bit operands
    auto product = [&](auto tc, auto c4, auto& A, auto& B, const uint32_t (&sa)[GA], const uint32_t (&sb)[GB],
                       auto& ac) {
        constexpr int i = decltype(tc)::v / FJ, j = decltype(tc)::v % FJ;
        if constexpr (decltype(c4)::value) mfma_mx4_agpr<j & 3, i & 3>(ac[i][j], B[j], A[i], sb[j / 4], sa[i / 4]);
        else mfma(ac[i][j], A[i], B[j]);
    };
    auto sources_extra = [&](int kt) {
        const ExtraStepMeta xm = extra_step(xs, lmeta, wlist, kz + ks * kt);  // the tile's step of this split
        if constexpr (BUF) {
#pragma unroll
            for (int b = 0; b < DA; ++b) {
                const ExtraChunk c = extra_chunk(xs, xm, cl ^ ((wave * DA + b) & 7), f.rp);
                vsrc[b] = c.ok && prow[b] >= c.sb && prow[b] < c.se ? (uint32_t)(prow[b] * 2 * f.rp + c.k) * 2u
                                                                    : kOutOfRange;
            }
#pragma unroll
            for (int b = 0; b < DB; ++b) {
                const ExtraChunk c = extra_chunk(xs, xm, cl ^ ((wave * DB + b) & 7), f.rp);
                vsrc[DA + b] =
                    c.ok && ncol[b] < N ? (uint32_t)((c.s * N + ncol[b]) * f.r_max + c.q) * 2u : kOutOfRange;
            }
            return;
        }
#pragma unroll
        for (int b = 0; b < DA; ++b) {
            const ExtraChunk c = extra_chunk(xs, xm, cl ^ ((wave * DA + b) & 7), f.rp);
            src[b] = or_zero(c.ok && prow[b] >= c.sb && prow[b] < c.se, f.ext + (int64_t)prow[b] * 2 * f.rp + c.k);
        }
#pragma unroll
        for (int b = 0; b < DB; ++b) {
            const ExtraChunk c = extra_chunk(xs, xm, cl ^ ((wave * DB + b) & 7), f.rp);
            src[DA + b] = or_zero(c.ok && ncol[b] < N, f.B_pool + ((int64_t)c.s * N + ncol[b]) * f.r_max + c.q);
        }
    };
    // XN: the loads are of an extra step (in the buffer form: ext and B_pool
    // with per-lane offsets; else x and W)
    auto load_piece = [&](int g, int buf, auto xn_tag) {
        constexpr bool XN = decltype(xn_tag)::value;
        if constexpr (F4) {
            if (g == DA + DB) {
                // 128 bytes of rows and 512 of scales a step
                if constexpr (BUF) bdma16(rS, svoff, soff * 4u, lds + buf * STAGE + ROWS16 + sl * 64);
                else dma16(ssrc, lds + buf * STAGE + ROWS16 + sl * 64);
                return;
            }
        }
        const int u = g < DA ? wave * DA + g : wave * DB + (g - DA);
        u32x4* dst = lds + buf * STAGE + ((g < DA ? 0 : ABYTES) + (u >> 3) * kGroupBytes + (u & 7) * kInstrBytes) / 16;
        if constexpr (BUF) {
            if constexpr (XN) bdma16(g < DA ? rE : rB, vsrc[g], 0u, dst);
            else bdma16(g < DA ? rX : rW, KTAIL ? vsrc[g] : (g < DA ? aoff[g] : boff[g - DA]), soff, dst);
        } else {
            dma16(src[g], dst);
        }
    };
    using XT = std::true_type;
    using XF = std::false_type;
    const int fr = lane & 15, fc = lane >> 4;
    const uint32_t lane_off = lds_offset(lds) + (fr & 7) * kInstrBytes + (fr >> 3) * 128;
    uint32_t abase[2], bbase[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // chunk h * 4 + fc of row fr sits at slot (h * 4 + fc) ^ (fr % 8)
        abase[h] = lane_off + block_off(wm * FI * 16) + ((h * 4 + fc) ^ (fr & 7)) * 16;
        bbase[h] = lane_off + ABYTES + block_off(wn * FJ * 16) + ((h * 4 + fc) ^ (fr & 7)) * 16;
    }
    u32x4 A0[FI], B0[FJ], A1[FI], B1[FJ];
    f32x4 acc[FI][FJ];
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // steps 0 .. L - 1 in flight, step 0 landed, its first half read
#pragma unroll
    for (int s0 = 0; s0 < L; ++s0) {
        if (s0 < ne) {
            sources_extra(s0);
#pragma unroll
            for (int g = 0; g < ND; ++g) load_piece(g, s0, XT{});
        } else {
            sources_base(min(s0, nt - 1));
#pragma unroll
            for (int g = 0; g < ND; ++g) load_piece(g, s0, XF{});
        }
    }
    vm_landed<(L - 1) * ND>();
    stage_barrier();
    static_for(std::make_integer_sequence<int, (FI > FJ ? FI : FJ)>{}, [&](auto ic) {
        constexpr int i = decltype(ic)::v;
        if constexpr (i < FJ) B0[i] = lds_read16<block_off(16 * i)>(bbase[0]);
        if constexpr (i < FI) A0[i] = lds_read16<block_off(16 * i)>(abase[0]);
    });
    if constexpr (F4) read_scales(Idx<0>{}, sA0, sB0, 0u);
    // fragment read r of a half: B blocks first (the first MFMAs need all of them)
    auto read_half = [&](auto rc, u32x4 (&A)[FI], u32x4 (&B)[FJ], uint32_t ab, uint32_t bb) {
        constexpr int r = decltype(rc)::v;
        if constexpr (r < FJ) B[r] = lds_read16<block_off(16 * r)>(bb);
        else A[r - FJ] = lds_read16<block_off(16 * (r - FJ))>(ab);
    };
    // one step; `next` sets the sources of step kt + L, loaded into buffer bn
    // (step kt's own buffer with 2 stages: only after every wave has read it)
    // bcv: the buffer of step kt (kt % NS), a run-time int or a constant
    // xc_tag: step kt itself is an extra step (F4: bf16 products)
    auto step = [&](int kt, auto&& next, auto xn_tag, auto bcv, auto xc_tag) {
        using C4 = std::integral_constant<bool, F4 && !decltype(xc_tag)::value>;
        int bc;
        if constexpr (std::is_integral_v<decltype(bcv)>) bc = bcv;
        else bc = decltype(bcv)::v;
        const int bn = bc + L >= 2 * NS ? bc + L - 2 * NS : bc + L >= NS ? bc + L - NS : bc + L;  // step kt + L's
        const uint32_t so = bc * STAGE * 16, sn = (bc + 1 == NS ? 0 : bc + 1) * STAGE * 16;
        next(kt + L);
        frags_landed(A0);
        frags_landed(B0);
        scales_landed(sA0, sB0);
        // phase A: MFMAs of the first half, reads of the second half. In a
        // group, the fragment read follows the group's first MFMA and its
        // loads the second, so that each waits in an MFMA's shadow.
        static_for(std::make_integer_sequence<int, NR>{}, [&](auto gc) {
            constexpr int g = decltype(gc)::v;
            constexpr int t0 = (g * NM + NR - 1) / NR, t1 = ((g + 1) * NM + NR - 1) / NR;  // this group's MFMAs
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (t0 < t1) product(Idx<t0>{}, C4{}, A0, B0, sA0, sB0, acc);
            __builtin_amdgcn_sched_barrier(0);
            read_half(gc, A1, B1, abase[1] + so, bbase[1] + so);
            if constexpr (F4 && g == 0) read_scales(Idx<1>{}, sA1, sB1, so);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (t0 + 1 < t1) product(Idx<t0 + 1>{}, C4{}, A0, B0, sA0, sB0, acc);
            __builtin_amdgcn_sched_barrier(0);
            static_for(std::make_integer_sequence<int, ND>{}, [&](auto pc) {  // loads of this group
                constexpr int pi = decltype(pc)::v;
                if constexpr (pi < NDA && pi * NR / NDA == g) load_piece(pi, bn, xn_tag);
            });
            __builtin_amdgcn_sched_barrier(0);
            static_for(std::make_integer_sequence<int, NM>{}, [&](auto tc) {  // the group's other MFMAs
                constexpr int t = decltype(tc)::v;
                if constexpr (t >= t0 + 2 && t < t1) product(tc, C4{}, A0, B0, sA0, sB0, acc);
            });
        });
        __builtin_amdgcn_sched_barrier(0);
        frags_retire(A0, B0);
        scales_retire(sA0, sB0);
        frags_landed(A1);
        frags_landed(B1);
        scales_landed(sA1, sB1);
        vm_landed<VM_MID>();  // step kt + 1 landed (this wave's loads; those of later steps may not)
        stage_barrier();
        // phase B: MFMAs of the second half, reads of step kt + 1's first half, the other loads
        static_for(std::make_integer_sequence<int, NR>{}, [&](auto gc) {
            constexpr int g = decltype(gc)::v;
            constexpr int t0 = (g * NM + NR - 1) / NR, t1 = ((g + 1) * NM + NR - 1) / NR;
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (t0 < t1) product(Idx<t0>{}, C4{}, A1, B1, sA1, sB1, acc);
            __builtin_amdgcn_sched_barrier(0);
            read_half(gc, A0, B0, abase[0] + sn, bbase[0] + sn);
            if constexpr (F4 && g == 0) read_scales(Idx<0>{}, sA0, sB0, sn);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (t0 + 1 < t1) product(Idx<t0 + 1>{}, C4{}, A1, B1, sA1, sB1, acc);
            __builtin_amdgcn_sched_barrier(0);
            static_for(std::make_integer_sequence<int, ND>{}, [&](auto pc) {
                constexpr int pi = decltype(pc)::v;
                if constexpr (pi >= NDA && (pi - NDA) * NR / NDB == g) load_piece(pi, bn, xn_tag);
            });
            __builtin_amdgcn_sched_barrier(0);
            static_for(std::make_integer_sequence<int, NM>{}, [&](auto tc) {
                constexpr int t = decltype(tc)::v;
                if constexpr (t >= t0 + 2 && t < t1) product(tc, C4{}, A1, B1, sA1, sB1, acc);
            });
        });
        __builtin_amdgcn_sched_barrier(0);
        frags_retire(A1, B1);
        scales_retire(sA1, sB1);
    };
    // steps whose step kt + L is an extra step, then the rest (the last L
    // steps reload the last step: the load count per step stays fixed). The
    // base steps run NS to an iteration, so that their buffers, and with them
    // every LDS address of the step, are constants.
    int kt = 0, bcr = 0;  // bcr = kt % NS
    auto adv = [&] { bcr = bcr + 1 == NS ? 0 : bcr + 1; };
    auto base_next = [&](int s) { sources_base(min(s, nt - 1)); };
    for (; kt + L < ne; ++kt, adv()) step(kt, sources_extra, XT{}, bcr, XT{});
    if constexpr (F4)
        for (; kt < ne; ++kt, adv()) step(kt, base_next, XF{}, bcr, XT{});
    for (; kt < nt && bcr != 0; ++kt, adv()) step(kt, base_next, XF{}, bcr, XF{});
    for (; kt + NS <= nt; kt += NS)
        static_for(std::make_integer_sequence<int, NS>{},
                   [&](auto sc) { step(kt + decltype(sc)::v, base_next, XF{}, sc, XF{}); });
    for (; kt < nt; ++kt, adv()) step(kt, base_next, XF{}, bcr, XF{});
    frags_landed(A0);
    frags_landed(B0);
    scales_landed(sA0, sB0);  // the last step's reads are waited on while their registers live
    vm_landed<0>();
#pragma unroll
    for (int i = 0; i < 12; ++i) asm volatile("s_nop 7");  // last MFMA results written
    const int p0 = m0 + wm * FI * 16, nb = n0 + wn * FJ * 16;
    if constexpr (SPLIT) {
        f32x4* out = reinterpret_cast<f32x4*>(so.part) + (int64_t)kz * so.n_mt * so.n_nt * 1024;
#pragma unroll
        for (int i = 0; i < FI; ++i) {
            const int rb = p0 / 16 + i;  // 16-row block
            if ((rb >> 2) >= so.n_mt) continue;
#pragma unroll
            for (int j = 0; j < FJ; ++j) {
                const int cb = nb / 16 + j;
                if ((cb >> 2) >= so.n_nt) continue;
                out[((int64_t)(rb >> 2) * so.n_nt + (cb >> 2)) * 1024 + ((rb & 3) * 4 + (cb & 3)) * 64 + lane] = acc[i][j];
            }
        }
        return;
    }
    if constexpr (EPI) fused_expand<FI, FJ>(acc, f, mv, p0, nb, M, N, lane);
    static_assert(NW * FI * FJ * 16 * 16 * 2 <= NS * STAGE * 16, "output staging");
    __syncthreads();
    store_tile<FI, FJ>(acc, reinterpret_cast<char*>(lds) + wave * (FI * 16) * (FJ * 32), Y, f.token_order, p0, nb, M,
                       N, lane);
}

// Whether every buffer the tile kernel's buffer form reads fits a buffer
// resource (under 2 GiB, so per-lane byte offsets and the out-of-range offset
// stay apart): x, one tile's W rows, ext, B_pool.
inline bool tile_buffers_fit(int M, int N, int K, int BN, const Fuse& f) {
    const int64_t lim = int64_t(1) << 31;
    return (int64_t)M * K * 2 < lim && (int64_t)BN * K * 2 < lim && (int64_t)M * f.rp * 4 < lim &&
           (int64_t)f.S * N * f.r_max * 2 < lim;
}

}  // namespace lora
