// The mixed-adapter linear layer over an MXFP4 base weight:
//   y[t_p] = bf16( act(x[t_p]) What^T + scale_s * h[p] B_s^T ),  h = x A_s^T
// What the values of the 4-bit codes, act the identity (16-bit activations)
// or the MXFP4 rounding of each row of x; the adapters always read x itself.
#include "fuse.h"
#include "mx4_linear.h"
#include "mx4_tile.h"
#include "shrink.h"

namespace lora {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// 16x16x128 product of 4-bit operands: lane l supplies row l % 16 of the left
// operand and column l % 16 of the right one, the 32 codes of k block l / 16
// each, and that block's scale in byte SA / SB of sa / sb; the result is laid
// out as mfma16x16x32's.
template <int SA, int SB>
__device__ __forceinline__ f32x4 mfma_mx4(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
    const i32x8 a8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8 b8{(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, SA, (int)sa, SB, (int)sb);
}

// ------------------------------------------------------------ decode-sized T --
// Kernel 1 of two, as on the bf16 decode path: a workgroup takes 64 columns x
// 16 NT rows over one K split and writes fp32 partials in that path's layout
// ([split][64-row tile][64-column tile][16 blocks][64 lanes], splitk.hip),
// which its kernel 2 adds, applies the expand to and rounds. A wave's unit is
// 64 columns x 256 k: one 8-byte read of scales and eight 16-byte reads of
// codes per lane, all issued at once. The four waves take the split's units
// in turn and add their sums in wave order through LDS. The SGMV shrink runs
// in extra workgroups of the same launch, over K ranges of its own.
// One row, 4096 -> 4096: 4.8 us with its event pair for 9 MB, two dependent
// rounds of memory (token order, then the units) and a launch; 48 rows of 4-bit
// x: 5.8 us. W is loaded without the non-temporal hint, here and below: with 24
// layers of 4096 -> 14336 in turn (744 MB, more than the caches hold) a call of
// 64 rows takes 22.8 us against 24.3 with it, and 20.0 against 23.4 while W
// stays cached.
struct Mx4Split {
    const uint16_t* X;
    const uint8_t *xc, *xs;  // 4-bit activations, in plan order
    const uint8_t *wc, *ws;
    float* part;
    int M, N, K, n_mt, n_nt, ks, upb;  // upb: units per split
    const int32_t* token_order;
    const Item* work;
    const uint16_t* A_pool;
    const int32_t* rank;
    float* part_h;  // [hs][M][r_max]
    int n_items, r_max, hs, hkc;
};

template <bool ACT4, int NT>
__global__ __launch_bounds__(256) void mx4_split_kernel(Mx4Split a) {
    __shared__ f32x4 red[4 * 4 * NT * 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n_shrink = a.n_items * a.hs;
    if ((int)blockIdx.x < n_shrink) {
        const int item = blockIdx.x % a.n_items, hz = blockIdx.x / a.n_items;
        const Item it = a.work[item];
        const int r = a.rank[it.slot];
        if (r == 0) return;
        const int kbeg = hz * a.hkc, kend = min(a.K, kbeg + a.hkc);
        const ShrinkOut out{a.part_h + (int64_t)hz * a.M * a.r_max, nullptr, 0, 0.f};
        shrink_item<4>(a.X, a.A_pool, r, a.token_order, it, out, a.K, kbeg, kend, a.r_max, red);
        return;
    }
    const int b = blockIdx.x - n_shrink, tiles = a.n_mt * a.n_nt;
    const int kz = b / tiles, t = b - kz * tiles, mt = t / a.n_nt, nt = t - mt * a.n_nt;
    const int fr = lane & 15, fc = lane >> 4;
    const int64_t rb = mx4_row_bytes(a.K), kts = mx4_k_tiles(a.K);
    const int u1 = min((int)kts, (kz + 1) * a.upb);
    const uint8_t* wrow[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) wrow[j] = a.wc + (int64_t)min(nt * 64 + 16 * j + fr, a.N - 1) * rb;
    const uint16_t* xrow[NT];
    const uint8_t* xq[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        // rows past M are not read: x comes from memory once per row and column tile
        const int p = mt * 64 + 16 * i + fr, pc = min(p, a.M - 1);
        if constexpr (ACT4) {
            xq[i] = p < a.M ? a.xc + (int64_t)pc * rb : nullptr;
        } else {
            const int tok = a.token_order[pc];  // loaded by every lane: no wait under a branch
            xrow[i] = p < a.M ? a.X + (int64_t)tok * a.K : nullptr;
        }
    }
    f32x4 acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int u = kz * a.upb + wave; u < u1; u += 4) {
        const u32x2 wsc = *as_global<u32x2>(a.ws + ((int64_t)nt * kts + u) * kMxTileBytes + lane * 8);
        u32x4 w[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int blk = u * 8 + h * 4 + fc;
                w[h][j] = *or_zero(blk * 32 < a.K, wrow[j] + blk * 16);
            }
        if constexpr (ACT4) {
            const u32x2 xsc = *as_global<u32x2>(a.xs + ((int64_t)mt * kts + u) * kMxTileBytes + lane * 8);
            u32x4 x[2][NT];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const int blk = u * 8 + h * 4 + fc;
                    x[h][i] = *or_zero(xq[i] && blk * 32 < a.K, xq[i] + blk * 16);
                }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                auto row = [&](auto ic) {
                    constexpr int i = decltype(ic)::value;
                    if constexpr (i < NT) {
                        acc[i][0] = mfma_mx4<i, 0>(x[h][i], w[h][0], acc[i][0], xsc[h], wsc[h]);
                        acc[i][1] = mfma_mx4<i, 1>(x[h][i], w[h][1], acc[i][1], xsc[h], wsc[h]);
                        acc[i][2] = mfma_mx4<i, 2>(x[h][i], w[h][2], acc[i][2], xsc[h], wsc[h]);
                        acc[i][3] = mfma_mx4<i, 3>(x[h][i], w[h][3], acc[i][3], xsc[h], wsc[h]);
                    }
                };
                row(std::integral_constant<int, 0>{});
                row(std::integral_constant<int, 1>{});
                row(std::integral_constant<int, 2>{});
                row(std::integral_constant<int, 3>{});
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4 x[4][NT];
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    u32x4 v[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const int k = u * 256 + h * 128 + 32 * m + 8 * fc;
                        v[m] = *or_zero(xrow[i] && k < a.K, xrow[i] + k);
                    }
                    mx4_transpose(v);
#pragma unroll
                    for (int m = 0; m < 4; ++m) x[m][i] = v[m];
                }
                float sc[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) sc[j] = mx4_scale(wsc[h] >> (8 * j) & 255);
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const u32x4 wf = mx4_bf16x8(w[h][j][m], sc[j]);
#pragma unroll
                        for (int i = 0; i < NT; ++i) acc[i][j] = mfma16x16x32(x[m][i], wf, acc[i][j]);
                    }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) red[((wave * 4 + j) * NT + i) * 64 + lane] = acc[i][j];
    __syncthreads();
    f32x4* out = reinterpret_cast<f32x4*>(a.part) + ((int64_t)(kz * a.n_mt + mt) * a.n_nt + nt) * 1024;
#pragma unroll
    for (int i = 0; i < NT; ++i) {  // wave w: column block w
        f32x4 s = red[(wave * NT + i) * 64 + lane];
#pragma unroll
        for (int v = 1; v < 4; ++v) s += red[((v * 4 + wave) * NT + i) * 64 + lane];
        out[(i * 4 + wave) * 64 + lane] = s;
    }
}

// The 16-bit activations of more than 16 rows: their bytes, read once per
// column tile, outweigh the 4-bit weights' (64 rows x 256 k are 32 KB, 64
// columns of codes 8 KB), and the 64-column kernel above is bound by them. A
// workgroup takes 128 columns over 16 NT rows with 8 waves, wave v columns
// 32 (v % 4) .. + 31 over half v / 4 of every unit (two waves per SIMD: with
// one, fragment reads, conversions and products wait on each other). A
// unit's x goes to LDS by direct loads, once for the eight waves, while its
// codes go to registers. In LDS a row of a unit is 32 chunks of 16 bytes, chunk
// c of row r at slot c ^ ((r + 4) % 16), through the source address. A 16-byte
// read by 64 lanes is served 16 lanes at a time, rows 0 - 3 and 12 - 15 of one
// lane group with rows 4 - 11 of its neighbour, whose chunk differs in bit 2:
// the two sets of slots are then disjoint (with c ^ (r % 16) they are equal,
// and conflicts take 48% of the LDS cycles). 64 rows,
// 4096 -> 14336: 15 us (the 64-column kernel 27), 5.9 and 1.10 a unit of 48 KB
// (44 GB/s a CU, under half of what its feed reaches). No one resource bounds a
// unit: with x's loads answered by zeros it takes 0.92 us, with W's 0.79, without
// the products 0.80, the conversions 1.00, the fragment reads 1.00; they partly
// follow one another. 2, 3 or 4 units in flight, one wave per SIMD or two, and a
// rotated order of units per tile take the same time.
constexpr int kWideCols = 128;
__device__ __forceinline__ int wide_swizzle(int row) { return (row + 4) & 15; }

template <int I, int N>
__device__ __forceinline__ void tie(u32x4 (&a)[N]) {
    if constexpr (I < N) {
        asm volatile("" : "+v"(a[I]));
        tie<I + 1, N>(a);
    }
}
// at most P LDS reads of this wave outstanding; a is read after that
template <int P, int N>
__device__ __forceinline__ void reads_landed(u32x4 (&a)[N]) {
    asm volatile("s_waitcnt lgkmcnt(%1)" : "+v"(a[0]) : "i"(P));
    tie<1, N>(a);
}

// NS buffers: unit u + NS - 1 is loaded, into the buffer of unit u - 1, when
// every wave has passed the barrier of unit u. Loads go through buffer
// resources (x, the tile's code rows, its scales): codes past a row's end are
// the next row's, or zeros past the tile's last row, and meet zeros of x. Only
// the per-lane offset is checked against a resource's end, so a unit's offset
// in the code rows is part of it.
template <int NT, int NS>
__global__ __launch_bounds__(512) void mx4_wide_kernel(Mx4Split a) {
    constexpr int ROWS = 16 * NT, UNIT = ROWS * 32, DMA = ROWS / 2 / 8;  // chunks of a unit; x loads per wave
    constexpr int LOADS = 3 + DMA;                                      // a wave's loads of a unit
    __shared__ u32x4 lds[NS * UNIT];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n_shrink = a.n_items * a.hs;
    static_assert(NS * UNIT >= 8 * 4 * 64 && (NS - 2) * LOADS < 64, "shrink scratch, wait counter");
    if ((int)blockIdx.x < n_shrink) {
        const int item = blockIdx.x % a.n_items, hz = blockIdx.x / a.n_items;
        const Item it = a.work[item];
        const int r = a.rank[it.slot];
        if (r == 0) return;
        const int kbeg = hz * a.hkc, kend = min(a.K, kbeg + a.hkc);
        const ShrinkOut out{a.part_h + (int64_t)hz * a.M * a.r_max, nullptr, 0, 0.f};
        shrink_item<8>(a.X, a.A_pool, r, a.token_order, it, out, a.K, kbeg, kend, a.r_max,
                       reinterpret_cast<f32x4*>(lds));
        return;
    }
    const int n_bt = (a.n_nt + 1) / 2, b = blockIdx.x - n_shrink, tiles = a.n_mt * n_bt;
    const int kz = b / tiles, t = b - kz * tiles, mt = t / n_bt, bt = t - mt * n_bt;
    const int fr = lane & 15, fc = lane >> 4;
    const int64_t rb = mx4_row_bytes(a.K), kts = mx4_k_tiles(a.K);
    const int u0 = kz * a.upb, u1 = min((int)kts, u0 + a.upb);
    const int half = wave >> 2, n0 = bt * kWideCols, c0 = n0 + (wave & 3) * 32, nt = c0 >> 6, cb = c0 >> 4 & 3;
    const int g0 = n0 >> 6, ng = min(a.n_nt - g0, 2);  // scale groups of the tile
    const brsrc rW = make_rsrc(a.wc + n0 * rb, (uint32_t)(min(a.N - n0, kWideCols) * rb));
    const brsrc rS = make_rsrc(a.ws + g0 * kts * kMxTileBytes, (uint32_t)(ng * kts * kMxTileBytes));
    const brsrc rX = make_rsrc(a.X, (uint32_t)a.M * (uint32_t)a.K * 2u);
    uint32_t woff[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
        woff[j] = (uint32_t)((min(c0 + 16 * j + fr, a.N - 1) - n0) * rb) + half * 64 + fc * 16;
    const uint32_t soff = (uint32_t)((min(nt, a.n_nt - 1) - g0) * kts * kMxTileBytes) + lane * 8 + half * 4;
    // x load d of this wave fetches rows 2 (DMA wave + d) + lane / 32 of a unit
    uint32_t xoff[DMA];
    int xk[DMA];
#pragma unroll
    for (int d = 0; d < DMA; ++d) {
        const int r = 2 * (DMA * wave + d) + (lane >> 5), p = mt * 64 + r;
        const int tok = a.token_order[min(p, a.M - 1)];
        const int k = ((lane & 31) ^ wide_swizzle(r)) * 8;
        xk[d] = p < a.M ? k : a.K;  // rows past M: past the row's end, zeros
        xoff[d] = ((uint32_t)tok * (uint32_t)a.K + k) * 2u;
    }
    u32x4 w[NS][2];
    uint32_t s[NS];
    // units past the split's last load zeros of x, so that every unit waits on
    // the same number of loads
    auto load = [&](int u, auto bc) {
        constexpr int buf = decltype(bc)::value;
        const int k = u < u1 ? u * 256 : a.K, uc = min(u, u1 - 1);
        s[buf] = __builtin_amdgcn_raw_buffer_load_b32(rS, soff, uc * kMxTileBytes, 0);
#pragma unroll
        for (int j = 0; j < 2; ++j)
            w[buf][j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rW, woff[j] + uc * 128, 0, 0));
#pragma unroll
        for (int d = 0; d < DMA; ++d)
            bdma16(rX, k + xk[d] < a.K ? xoff[d] : kOutOfRange, (uint32_t)k * 2u,
                   lds + buf * UNIT + (DMA * wave + d) * 64);
        issue_fence();
    };
    f32x4 acc[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto unit = [&](int u, auto bc) {
        constexpr int buf = decltype(bc)::value;
        vm_landed<(NS - 2) * LOADS>();  // this unit's loads landed, later ones may not
        stage_barrier();
        load(u + NS - 1, std::integral_constant<int, (buf + NS - 1) % NS>{});
        // products 0 .. 3 of the wave's half; the next one's fragments are
        // read while a product runs
        const uint32_t row = lds_offset(lds + buf * UNIT) + fr * 512;
        u32x4 x[2][NT];
        auto read = [&](auto mc, u32x4 (&f)[NT]) {
            const uint32_t at = row + (((half * 4 + fc) * 4 + decltype(mc)::value) ^ wide_swizzle(fr)) * 16;
            f[0] = lds_read16<0>(at);
            f[1] = lds_read16<16 * 512>(at);
            if constexpr (NT > 2) {
                f[2] = lds_read16<32 * 512>(at);
                f[3] = lds_read16<48 * 512>(at);
            }
        };
        read(std::integral_constant<int, 0>{}, x[0]);
        float sc[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) sc[j] = mx4_scale(s[buf] >> (8 * (cb + j)) & 255);
        auto product = [&](auto mc) {
            constexpr int m = decltype(mc)::value;
            if constexpr (m < 3) {
                read(std::integral_constant<int, m + 1>{}, x[(m + 1) & 1]);
                reads_landed<NT>(x[m & 1]);
            } else {
                reads_landed<0>(x[m & 1]);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const u32x4 wf = mx4_bf16x8(w[buf][j][m], sc[j]);
#pragma unroll
                for (int i = 0; i < NT; ++i) acc[i][j] = mfma16x16x32(x[m & 1][i], wf, acc[i][j]);
            }
        };
        product(std::integral_constant<int, 0>{});
        product(std::integral_constant<int, 1>{});
        product(std::integral_constant<int, 2>{});
        product(std::integral_constant<int, 3>{});
    };
    load(u0, std::integral_constant<int, 0>{});
    if constexpr (NS > 2) load(u0 + 1, std::integral_constant<int, 1>{});
    if constexpr (NS > 3) load(u0 + 2, std::integral_constant<int, 2>{});
    for (int u = u0; u < u1; u += NS) {
        unit(u, std::integral_constant<int, 0>{});
        if (u + 1 >= u1) break;  // uniform, as the others
        unit(u + 1, std::integral_constant<int, 1>{});
        if constexpr (NS > 2) {
            if (u + 2 >= u1) break;
            unit(u + 2, std::integral_constant<int, 2>{});
        }
        if constexpr (NS > 3) {
            if (u + 3 >= u1) break;
            unit(u + 3, std::integral_constant<int, 3>{});
        }
    }
    // the halves' sums added; no load into LDS is in flight past this
    vm_landed<0>();
    __syncthreads();
    f32x4* red = reinterpret_cast<f32x4*>(lds) + (wave & 3) * 2 * NT * 64;
    static_assert(NS * UNIT >= 4 * 2 * NT * 64, "reduction scratch");
    if (half == 1) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) red[(i * 2 + j) * 64 + lane] = acc[i][j];
    }
    __syncthreads();
    if (half == 1 || nt >= a.n_nt) return;
    f32x4* out = reinterpret_cast<f32x4*>(a.part) + ((int64_t)(kz * a.n_mt + mt) * a.n_nt + nt) * 1024;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) out[(i * 4 + cb + j) * 64 + lane] = acc[i][j] + red[(i * 2 + j) * 64 + lane];
}

// Kernel 2: a wave takes 16 rows x 64 columns, adds the splits in order, runs
// the expand on the matrix cores and stores whole row pieces. The bf16 path's
// kernel 2 (splitk.hip) gives the same 16 x 64 to four waves, each of which
// loads the rows' h and slot metadata again and holds 196 registers: it is
// faster while its blocks fit the chip at once (two a CU; 4.0 against 5.4 us
// at 64 x 4096) and falls behind past that (8.7 against 5.7 us at 64 x 14336,
// 24 against 9.5 us at 256 x 14336; rank 64 at 200 x 14336, 28 against 16 us).
// NC: chunks of 32 ranks (0: no adapters), pools of at most 64 slots (slot s on
// lane s). HALF: rows of B start on 8-byte boundaries (r_max % 8 == 4).
constexpr int kFinishSlots = 64, kFinishRank = 64, kFinishBlocks = 512;

struct Mx4Finish {
    const float* part;  // [ks][n_mt][n_nt][16 blocks][64 lanes] f32x4
    const float* h;     // [hs][M][r_max]
    uint16_t* Y;
    int M, N, ks, n_mt, n_nt, hs, S, r_max;
    const int32_t *token_order, *slot_indptr, *rank;
    const float* scale;
    const uint16_t* B_pool;
};

template <int NC, bool HALF>
__global__ __launch_bounds__(256) void mx4_finish_kernel(Mx4Finish a) {
    constexpr bool ADAPT = NC > 0;
    __shared__ u32x4 stg[4][16 * 9];  // a wave's 16 rows of 64 columns, 16 bytes of padding each
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nt = blockIdx.x, mt = blockIdx.y, p0 = mt * 64 + wave * 16, n0 = nt * 64;
    if (p0 >= a.M) return;  // the waves do not meet
    const int fr = lane & 15, fc = lane >> 4;
    const f32x4* in = reinterpret_cast<const f32x4*>(a.part) + ((int64_t)mt * a.n_nt + nt) * 1024 + wave * 256 + lane;
    const int64_t plane = (int64_t)a.n_mt * a.n_nt * 1024;
    f32x4 acc[4];
    f32x4 p[2][4];
#pragma unroll
    for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int j = 0; j < 4; ++j) p[z][j] = in[min(z, a.ks - 1) * plane + j * 64];
    int tok[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) tok[i] = a.token_order[min(p0 + 8 * i + (lane >> 3), a.M - 1)];
    u32x4 hi[ADAPT ? NC : 1], lo[ADAPT ? NC : 1];
    int slot = 0;        // of row p0 + fr
    uint64_t slots = 0;  // the block's slots
    if constexpr (ADAPT) {
        const int ip = a.slot_indptr[min(lane, a.S)];
        const int rk = a.rank[min(lane, a.S - 1)];
        const float sv = a.scale[min(lane, a.S - 1)];
        // lane (fr, fc): ranks 32 c + 8 fc .. + 7 of row fr, every plane loaded
        f32x4 hv[8][2];
        const float* hp = a.h + (int64_t)min(p0 + fr, a.M - 1) * a.r_max + 8 * fc;
        auto load_h = [&](int c) {
#pragma unroll
            for (int z = 0; z < 8; ++z) {
                const float* q = hp + (int64_t)z * a.M * a.r_max + 32 * c;
#pragma unroll
                for (int g = 0; g < 2; ++g)
                    hv[z][g] = __builtin_bit_cast(
                        f32x4, *or_zero(z < a.hs && 32 * c + 8 * fc + 4 * g < a.r_max, q + 4 * g));
            }
        };
        load_h(0);
        issue_fence();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            // slot of row p0 + j: how many of the slots 1 .. S - 1 start at or before it
            const int s = __popcll(__ballot(lane >= 1 && lane < a.S && ip <= p0 + j));
            if (fr == j) slot = s;
            if (p0 + j < a.M) slots |= 1ull << s;
        }
        slots &= ~1ull;
        int r = __shfl(rk, slot);  // by every lane: slot s is on lane s
        r = slot == 0 ? 0 : r;
        const float sc = __shfl(sv, slot);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (c > 0) load_h(c);
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float x = 0.f;
#pragma unroll
                for (int z = 0; z < 8; ++z) x += hv[z][e >> 2][e & 3];
                // past the rank the planes hold nothing
                v[e] = 32 * c + 8 * fc + e < r ? x * sc : 0.f;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                hi[c][e] = pack_bf16x2(hi_half(v[2 * e]), hi_half(v[2 * e + 1]));
                lo[c][e] = pack_bf16x2(v[2 * e] - __uint_as_float(hi[c][e] << 16),
                                       v[2 * e + 1] - __uint_as_float(hi[c][e] & 0xffff0000u));
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = a.ks > 1 ? p[0][j] + p[1][j] : p[0][j];
    for (int z0 = 2; z0 < a.ks; z0 += 2) {
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
            for (int j = 0; j < 4; ++j) p[z][j] = in[min(z0 + z, a.ks - 1) * plane + j * 64];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            acc[j] += p[0][j];
            if (z0 + 1 < a.ks) acc[j] += p[1][j];
        }
    }
    if constexpr (ADAPT) {
        // two slots at a time: their B rows (lane (fr, fc): column fr of a
        // block, ranks 8 fc ..) loaded together
        while (slots) {
            int s[2], rs[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                s[i] = slots ? (int)__builtin_ctzll(slots) : 0;
                slots &= slots - 1;
                rs[i] = s[i] ? a.rank[s[i]] : 0;  // uniform
            }
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (c > 0 && max(rs[0], rs[1]) <= 32 * c) break;  // uniform
                u32x4 b[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int n = n0 + 16 * j + fr, q = 32 * c + 8 * fc;
                        const uint16_t* row = a.B_pool + ((int64_t)s[i] * a.N + n) * a.r_max + q;
                        if constexpr (HALF) {
                            const u32x2 b0 = *(gptr<u32x2>)or_zero(n < a.N && q < rs[i], row);
                            const u32x2 b1 = *(gptr<u32x2>)or_zero(n < a.N && q + 4 < rs[i], row + 4);
                            b[i][j] = u32x4{b0[0], b0[1], b1[0], b1[1]};
                        } else {
                            b[i][j] = *or_zero(n < a.N && q < rs[i], row);
                        }
                    }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bool on = slot == s[i];
                    u32x4 h1, h2;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        h1[e] = on ? hi[c][e] : 0u;
                        h2[e] = on ? lo[c][e] : 0u;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const f32x4 d = mfma16x16x32(h2, b[i][j], mfma16x16x32(h1, b[i][j], f32x4{0.f, 0.f, 0.f, 0.f}));
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[j][e] += d[e];
                    }
                }
            }
        }
    }
    // lane: rows 4 fc + e, column 16 j + fr -> rows of 128 bytes
    uint16_t* t = reinterpret_cast<uint16_t*>(stg[wave]);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) t[(4 * fc + e) * 72 + 16 * j + fr] = f32_to_bf16(acc[j][e]);
    const int c = lane & 7;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = 8 * i + (lane >> 3), n = n0 + 8 * c;
        const u32x4 v = stg[wave][row * 9 + c];
        if (p0 + row >= a.M || n >= a.N) continue;
        uint16_t* y = a.Y + (int64_t)tok[i] * a.N + n;
        if (a.N % 8 == 0) {
            *reinterpret_cast<u32x4*>(y) = v;
        } else {
            for (int e = 0; e < min(8, a.N - n); ++e) y[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
        }
    }
}

// -------------------------------------------------- before the products --
// What a call does to one operand (x to 4 bits in plan order, or W's values
// to bf16) and the SGMV shrink depend on nothing of each other: one launch,
// the shrink's workgroups (item, K range) first, then a workgroup per tile of
// 64 rows x 256 k.
struct Mx4Prep {
    const uint16_t* X;
    int M, N, K;
    const int32_t* token_order;
    uint8_t *xc, *xs;           // kQuantize
    const uint8_t *wc, *ws;     // kDequantize
    uint16_t* W;
    const Item* work;
    const uint16_t* A_pool;
    const int32_t* rank;
    const float* scale;
    int n_items, r_max, hs, hkc;
    float* h;       // [hs][M][r_max] (ext null)
    uint16_t* ext;  // the expand operand (with hs > 1 h holds the planes before)
};

// 8 waves: 51 us for 2048 x 14336 rows (144 items) beside 4096 x 14336 of W,
// against 63 us with 16; 37 us for 8192 x 4096, against 43 with 16 and 36 with 4.
constexpr int kPrepWaves = 8;
template <bool QUANT>
__global__ __launch_bounds__(64 * kPrepWaves) void mx4_prep_kernel(Mx4Prep a) {
    constexpr int WAVES = kPrepWaves;
    __shared__ f32x4 red[WAVES * 4 * 64];
    static_assert(sizeof(red) >= kMxTileBytes, "scale tile");
    const int n_shrink = a.n_items * a.hs;
    if ((int)blockIdx.x < n_shrink) {
        const int item = blockIdx.x % a.n_items, hz = blockIdx.x / a.n_items;
        const Item it = a.work[item];
        const int r = a.rank[it.slot];
        if (r == 0) return;
        const int kbeg = hz * a.hkc, kend = min(a.K, kbeg + a.hkc);
        const ShrinkOut out{a.h + (int64_t)hz * a.M * a.r_max, a.ext, (a.r_max + 7) & ~7, a.scale[it.slot]};
        shrink_item<WAVES>(a.X, a.A_pool, r, a.token_order, it, out, a.K, kbeg, kend, a.r_max, red);
        return;
    }
    const int kts = (int)mx4_k_tiles(a.K), t = blockIdx.x - n_shrink;
    uint8_t* st = reinterpret_cast<uint8_t*>(red);
    if constexpr (QUANT)
        quantize_tile<uint16_t, 64 * WAVES>(a.X, a.M, a.K, a.token_order, a.xc, a.xs, t % kts, t / kts, st);
    else
        dequantize_tile<uint16_t, 64 * WAVES>(a.wc, a.ws, a.N, a.K, a.W, t % kts, t / kts, st);
}

// The expand operand of an item's rows from hs planes of h, added in order.
__global__ __launch_bounds__(256) void mx4_operand_kernel(Mx4Prep a) {
    const Item it = a.work[blockIdx.x];
    const int r = a.rank[it.slot];
    if (r == 0) return;
    const float sc = a.scale[it.slot];
    const int rp = (a.r_max + 7) & ~7;
    for (int i = threadIdx.x; i < it.count * rp; i += 256) {
        const int m = i / rp, q = i - m * rp;
        const int64_t p = it.begin + m;
        float v = 0.f;
        if (q < r)
            for (int z = 0; z < a.hs; ++z) v += a.h[((int64_t)z * a.M + p) * a.r_max + q];
        v *= sc;
        const uint16_t hi = bf16_hi(v);
        a.ext[(p * 2) * rp + q] = hi;
        a.ext[(p * 2 + 1) * rp + q] = f32_to_bf16(v - bf16_to_f32(hi));
    }
}

// K ranges of the shrink ahead of a tiled product. Over a long K and with few
// items one range per item would outlast the other workgroups (8 waves take
// about 1.3 us per 1024 k: 18 us at 14336), so that it is split and the planes
// joined by one more launch (3 us): 512 x 14336 -> 4096 in 43 us against 65.
// At K = 4096, or with 128 items at 14336, one range is as fast.
static int prep_ranges(int K, int n_items) {
    return K < 8192 ? 1 : max(1, min(min(8, K / 2048), 128 / max(n_items, 1)));
}

template <bool QUANT>
static hipError_t launch_prep(const Mx4Prep& a, hipStream_t st, StageTimer* tm) {
    const int64_t tiles = ((int64_t)(QUANT ? a.M : a.N) + 63) / 64 * mx4_k_tiles(a.K);
    const dim3 grid((uint32_t)(a.n_items * a.hs + tiles));
    const char* name = QUANT ? "mx4_quantize+shrink" : "mx4_dequantize+shrink";
    Mx4Prep k = a;
    if (a.ext && a.hs > 1) k.ext = nullptr;  // planes first
    const hipError_t e = launch(tm, name, mx4_prep_kernel<QUANT>, grid, dim3(64 * kPrepWaves), st, k);
    if (e != hipSuccess || !a.ext || a.hs == 1 || a.n_items == 0) return e;
    return launch(tm, "mx4_operand", mx4_operand_kernel, dim3(a.n_items), dim3(256), st, a);
}

// Rows of any width (x, and with adapters the pool's A up to each slot's rank)
// -> rows of Kp elements, a multiple of 8, zeros behind the row's end: the
// kernels read rows in 16-byte pieces. One launch for both; a wave takes 64
// pieces of a row, loaded off 16-byte boundaries.
struct Mx4Pad {
    const uint16_t *x, *A;
    uint16_t *xp, *Ap;
    int64_t M, rows;  // rows: M + S r_max
    int K, Kp, r_max;
    const int32_t* rank;
};
__global__ __launch_bounds__(256) void pad_rows_kernel(Mx4Pad a) {
    const int64_t r = (blockIdx.y + (int64_t)blockIdx.z * gridDim.y) * 4 + (threadIdx.x >> 6);
    const int k = (blockIdx.x * 64 + (threadIdx.x & 63)) * 8;
    if (r >= a.rows || k >= a.Kp) return;
    const int64_t q = r - a.M;  // row of A
    if (q >= 0 && (int)(q % a.r_max) >= a.rank[q / a.r_max]) return;
    const uint16_t* src = (q < 0 ? a.x + r * a.K : a.A + q * a.K) + k;
    uint16_t* dst = (q < 0 ? a.xp + r * a.Kp : a.Ap + q * a.Kp) + k;
    u32x4 v{0, 0, 0, 0};
    if (k + 8 <= a.K) {
        Raw8<uint16_t> p;
        p.load(src);
        v = p.v;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (k + e < a.K) v[e >> 1] |= (uint32_t)src[e] << (16 * (e & 1));
    }
    *reinterpret_cast<u32x4*>(dst) = v;
}

// B's rows of r_max values (not a multiple of 8) -> rows of rp, zeros behind:
// the tiles' extra steps read them in 16-byte pieces. A thread writes a piece.
__global__ __launch_bounds__(256) void pad_ranks_kernel(const uint16_t* __restrict__ src, int64_t rows, int r_max,
                                                        int rp, u32x4* __restrict__ dst) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = i / (rp / 8);
    if (row >= rows) return;
    const int q = (int)(i - row * (rp / 8)) * 8;
    uint32_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = q + e < r_max ? src[row * r_max + q + e] : 0u;
    dst[i] = u32x4{v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16};
}

// Whether a tiled product pads the pool's B for its extra K steps, rather than
// run the expand in the epilogue of 128 x 128 tiles. The copy (4 to 5 us) moves S
// rp values a column, so it needs rows in proportion; with 4-bit x, where all
// else stays, also a large output: rank 12, 16 adapters, 2048 x 4096 -> 14336 92
// against 123 us, 600 x 4096 -> 14336 57 against 62, 2048 x 4096 -> 4096 43
// against 47, but 600 x 4096 -> 4096 33 against 30. With 16-bit x it also brings
// the shrink into the launch before: 2048 x 4096 -> 4096 78 against 82, 2048 x
// 1024 -> 2048 27 against 33.
static bool tile_pads(int M, int N, int S, int r_max, bool act4) {
    const int rp = (r_max + 7) & ~7;
    return r_max % 8 != 0 && S <= kMetaSlots && (int64_t)M >= (int64_t)2 * S * rp &&
           (!act4 || (int64_t)M * N >= int64_t(1) << 23);
}

// The second kernel of the decode path: mx4_finish past kFinishBlocks blocks
// where it takes the pool, else the bf16 path's.
static bool finish_takes(int S, int r_max) { return S <= kFinishSlots && r_max <= kFinishRank && r_max % 4 == 0; }
static bool finish_few(int M, int N) { return (int64_t)cdiv(N, 64) * cdiv(M, 16) <= kFinishBlocks; }

// The path of a call, by its sizes, the pool's and act alone (a base-only call
// takes the same one).
// 16-bit activations: the wide kernel wherever the bf16 layer splits K, up to
// 768 rows (decoding all of W costs more than it saves there: 320 x 14336 ->
// 4096 71 against 97 us, 320 x 4096 -> 4096 25 against 38, 512 x 4096 -> 4096 35
// against 37, 640 x 4096 -> 28672 198 against 268; 512 x 4096 -> 14336, 88
// against 86, is the worst; from 1024 rows of 4096 columns on it loses, 58
// against 48), and at most 128 of its tiles (1024 x 4096 -> 1024 25 against 33;
// 192 tiles 38 against 33), unless a pool that mx4_finish does not take would
// leave many blocks to the bf16 path's kernel 2.
// 4-bit activations: split K while its 64 x 64 tiles are few (kernels, split
// against the 4-bit tile: 64 x 4096 -> 4096 15.5 against 22 us, 128 x 4096 ->
// 4096 21 against 22, 256 x 4096 -> 2048 21 against 22, 512 x 4096 -> 1024 equal
// at 22, 128 x 14336 -> 4096 39 against 35; past 128 tiles 65 x 4096 -> 8200 31
// against 23, 96 x 4096 -> 14336 35 against 24), and for one tile of rows at any
// width (64 x 4096 -> 14336 25 against 24).
enum class Mx4Path { kSplit, kTile4, kDequant };
static Mx4Path mx4_path(int M, int N, int K, int S, int r_max, bool act4) {
    if (act4) return M <= 64 || (int64_t)cdiv(M, 64) * cdiv(N, 64) <= 128 ? Mx4Path::kSplit : Mx4Path::kTile4;
    const bool few = (M <= 768 || (int64_t)cdiv(M, 64) * cdiv(N, kWideCols) <= 128) &&
                     (finish_takes(S, r_max) || finish_few(M, N));
    return (few || gemm_bf16_plan(M, N, K).nsub != 0) && (int64_t)M * K * 2 < int64_t(1) << 31 ? Mx4Path::kSplit
                                                                                              : Mx4Path::kDequant;
}

static bool mx4_wide(int M, bool act4) { return !act4 && M > 16; }

// K splits of the decode path. The shrink's work items count as tiles, as many
// as M rows over S slots can give, so that a base-only call splits alike: an
// item moves about the bytes of a unit per 256 k. The wide kernel takes the
// splits of the least estimated time: 1.5 us per unit and workgroup of a CU
// (two on one CU take about twice as long), and each split's partials,
// written and read at 5 TB/s. The 64-column kernel goes for 512 workgroups (4-bit
// x, kernels at 256 / 512 / 1024: 48 x 4096 -> 4096 18.5 / 15 / 15 us, 64 x 14336
// -> 4096 32 / 28 / 26, 64 x 4096 -> 14336 29 / 25 / 28; 16-bit x: 1 x 4096 ->
// 4096 9.6 / 8.7 / 8.7, 16 x 14336 -> 4096 18.9 / 16.7 / 18.2). The shrink takes
// K ranges of a split's length, 8 at most.
struct Mx4SplitPlan {
    int n_mt, n_nt, ks, upb, hs, hkc;
};
static Mx4SplitPlan mx4_split_plan(int M, int N, int K, int S, bool act4) {
    Mx4SplitPlan p{};
    p.n_mt = cdiv(M, 64);
    p.n_nt = cdiv(N, 64);
    const int kts = (int)mx4_k_tiles(K), items = M / 16 + min(S - 1, M);
    if (mx4_wide(M, act4)) {
        const int64_t tiles = (int64_t)p.n_mt * cdiv(N, kWideCols) + items;
        double best = 0.0;
        for (int ks = 1; ks <= 16 && ks <= kts; ++ks) {
            const int upb = cdiv(kts, ks);
            const int64_t rounds = (tiles * cdiv(kts, upb) + 255) / 256;  // workgroups per CU
            const double cost = upb * 1.5 * rounds + ks * (M * 8e-6 / 5.0) * N;
            if (p.upb == 0 || cost < best) {
                best = cost;
                p.upb = upb;
            }
        }
    } else {  // a unit for every wave
        const int tiles = p.n_mt * p.n_nt;
        p.upb = (cdiv(kts, max(1, 512 / (tiles + items))) + 3) / 4 * 4;
    }
    p.ks = cdiv(kts, p.upb);
    p.hkc = max(p.upb * 256, (cdiv(K, 8) + 31) / 32 * 32);
    p.hs = cdiv(K, p.hkc);
    return p;
}

// Workspace: padded rows of x and A (d_in not a multiple of 8), the 4-bit
// activations, then the path's own (partials and h planes; h or the expand
// operand; W in bf16 and the bf16 layer's workspace).
struct Mx4Space {
    size_t xpad, apad, bpad, codes, scales, own, h, planes, total;
};
static Mx4Space mx4_space(int M, int N, int d_in, int S, int r_max, bool act4) {
    const int K = (d_in + 7) / 8 * 8;  // padded rows, which the path and its kernels see too
    Mx4Space s{};
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += (bytes + 255) & ~size_t(255);
        return at;
    };
    s.xpad = take(d_in % 8 ? (size_t)M * K * 2 : 0);
    s.apad = take(d_in % 8 ? (size_t)S * r_max * K * 2 : 0);
    const bool pads = mx4_path(M, N, K, S, r_max, act4) != Mx4Path::kSplit && tile_pads(M, N, S, r_max, act4);
    s.bpad = take(pads ? (size_t)S * N * ((r_max + 7) & ~7) * 2 : 0);
    s.codes = take(act4 ? (size_t)M * mx4_row_bytes(K) : 0);
    s.scales = take(act4 ? (size_t)mx4_scale_bytes(M, K) : 0);
    switch (mx4_path(M, N, K, S, r_max, act4)) {
        case Mx4Path::kSplit: {
            const Mx4SplitPlan p = mx4_split_plan(M, N, K, S, act4);
            s.own = take((size_t)p.ks * p.n_mt * p.n_nt * 64 * 64 * sizeof(float));
            s.h = take((size_t)p.hs * M * r_max * sizeof(float));
            break;
        }
        case Mx4Path::kTile4:
            s.own = take(tiled_workspace(M, r_max));
            s.planes = take((size_t)8 * M * r_max * sizeof(float));
            break;
        case Mx4Path::kDequant:
            s.own = take((size_t)N * K * 2);
            s.h = take(gemm_bf16_workspace(M, &N, 1, K, r_max));
            s.planes = take((size_t)8 * M * r_max * sizeof(float));
    }
    s.total = o;
    return s;
}

size_t mx4_linear_workspace(int M, int N, int K, int S, int r_max, bool act4) {
    return M > 0 ? mx4_space(M, N, K, S, r_max, act4).total : 0;
}

static hipError_t pad_rows(const Mx4Pad& a, hipStream_t st, StageTimer* tm) {
    const int64_t blocks = (a.rows + 3) / 4;
    const uint32_t gy = (uint32_t)(blocks < 65535 ? blocks : 65535);
    return launch(tm, "pad_rows", pad_rows_kernel, dim3((a.Kp + 511) / 512, gy, (uint32_t)((blocks + gy - 1) / gy)),
                  dim3(256), st, a);
}

static hipError_t launch_split(const Mx4Split& a, bool act4, hipStream_t st, StageTimer* tm) {
    if (mx4_wide(a.M, act4))
        return launch(tm, "mx4_wide", a.M <= 32 ? mx4_wide_kernel<2, 3> : mx4_wide_kernel<4, 3>,
                      dim3(a.n_items * a.hs + a.n_mt * cdiv(a.N, kWideCols) * a.ks), dim3(512), st, a);
    auto ker = !act4       ? mx4_split_kernel<false, 1>
               : a.M <= 16 ? mx4_split_kernel<true, 1>
               : a.M <= 32 ? mx4_split_kernel<true, 2>
                           : mx4_split_kernel<true, 4>;
    return launch(tm, "mx4_split", ker, dim3(a.n_items * a.hs + a.n_mt * a.n_nt * a.ks), dim3(256), st, a);
}

hipError_t mx4_linear(const LinearArgs& L0, const uint8_t* codes, const uint8_t* scales, bool act4, hipStream_t st,
                      StageTimer* tm) {
    LinearArgs L = L0;
    SliceArgs& sl = L.slice[0];
    const int M = L.M, N = sl.N;
    char* ws = static_cast<char*>(L.workspace);
    const Mx4Space sp = mx4_space(M, N, L.K, L.S, L.r_max, act4);
    hipError_t e = hipSuccess;
    Mx4Prep pr{};
    pr.X = L.X;
    pr.M = M;
    pr.N = N;
    pr.K = L.K;
    pr.token_order = L.token_order;
    pr.xc = reinterpret_cast<uint8_t*>(ws + sp.codes);
    pr.xs = reinterpret_cast<uint8_t*>(ws + sp.scales);
    if (L.K % 8) {
        const int Kp = (L.K + 7) / 8 * 8;
        uint16_t* xp = reinterpret_cast<uint16_t*>(ws + sp.xpad);
        uint16_t* ap = reinterpret_cast<uint16_t*>(ws + sp.apad);
        const Mx4Pad pad{L.X, sl.A_pool, xp, ap, M, M + (L.adapters ? (int64_t)L.S * L.r_max : 0), L.K, Kp, L.r_max,
                         sl.rank};
        e = pad_rows(pad, st, tm);
        if (e != hipSuccess) return e;
        L.X = xp;
        sl.A_pool = ap;
        L.K = Kp;  // as many blocks and scale tiles; zeros quantise to zeros
        pr.X = xp;
        pr.K = Kp;
    }
    pr.work = reinterpret_cast<const Item*>(L.work);
    pr.A_pool = sl.A_pool;
    pr.rank = sl.rank;
    pr.scale = sl.scale;
    pr.n_items = L.adapters ? L.n_items : 0;
    pr.r_max = L.r_max;
    pr.hs = 1;
    pr.hkc = L.K;
    // the expand as extra K steps of a tiled product, where its form allows
    const bool pads = tile_pads(M, N, L.S, L.r_max, act4), ext_ok = pads || (L.r_max % 8 == 0 && L.S <= kMetaSlots);
    auto pad_ranks = [&] {  // after it L describes a pool of padded ranks (pr's A is the pool's)
        const int rp = (L.r_max + 7) & ~7;
        const int64_t rows = (int64_t)L.S * N;
        u32x4* bp = reinterpret_cast<u32x4*>(ws + sp.bpad);
        const hipError_t pe = !L.adapters ? hipSuccess
                                          : launch(tm, "pad_ranks", pad_ranks_kernel,
                                                   dim3((uint32_t)((rows * (rp / 8) + 255) / 256)), dim3(256), st,
                                                   sl.B_pool, rows, L.r_max, rp, bp);
        sl.B_pool = reinterpret_cast<const uint16_t*>(bp);
        L.r_max = rp;
        return pe;
    };
    switch (mx4_path(M, N, L.K, L.S, L.r_max, act4)) {
        case Mx4Path::kSplit: {
            const Mx4SplitPlan p = mx4_split_plan(M, N, L.K, L.S, act4);
            Mx4Split a{L.X, pr.xc, pr.xs, codes, scales, reinterpret_cast<float*>(ws + sp.own), M, N, L.K, p.n_mt,
                       p.n_nt, p.ks, p.upb, L.token_order, pr.work, sl.A_pool, sl.rank,
                       reinterpret_cast<float*>(ws + sp.h), pr.n_items, L.r_max, p.hs, p.hkc};
            if (act4) {  // the shrink beside the quantisation
                pr.hs = p.hs;
                pr.hkc = p.hkc;
                pr.h = a.part_h;
                a.n_items = 0;
                e = launch_prep<true>(pr, st, tm);
                if (e != hipSuccess) return e;
            }
            e = launch_split(a, act4, st, tm);
            if (e != hipSuccess) return e;
            if (!finish_takes(L.S, L.r_max) || finish_few(M, N))
                return splitk_finish_bf16(L, sl, a.part, p.ks, p.n_mt, a.part_h, p.hs, st, tm);
            const Mx4Finish fin{a.part, a.part_h, sl.Y, M, N, p.ks, p.n_mt, p.n_nt, p.hs, L.S, L.r_max, L.token_order,
                                L.slot_indptr, sl.rank, sl.scale, sl.B_pool};
            const bool half = L.r_max % 8 != 0;
            auto ker = !L.adapters     ? mx4_finish_kernel<0, false>
                       : L.r_max <= 32 ? (half ? mx4_finish_kernel<1, true> : mx4_finish_kernel<1, false>)
                                       : (half ? mx4_finish_kernel<2, true> : mx4_finish_kernel<2, false>);
            return launch(tm, "mx4_finish", ker, dim3(p.n_nt, p.n_mt), dim3(256), st, fin);
        }
        case Mx4Path::kTile4: {
            float* h = reinterpret_cast<float*>(ws + sp.own);
            if (pads) e = pad_ranks();
            if (e != hipSuccess) return e;
            Fuse f{L.token_order, L.slot_indptr, h, sl.B_pool, sl.rank, sl.scale, L.S, L.r_max, 1, 0, L.adapters,
                   nullptr, (L.r_max + 7) & ~7};
            pr.h = h;
            if (ext_ok) {
                pr.ext = reinterpret_cast<uint16_t*>(h);
                pr.h = reinterpret_cast<float*>(ws + sp.planes);
                pr.hs = prep_ranges(L.K, pr.n_items);
                pr.hkc = (cdiv(L.K, pr.hs) + 31) / 32 * 32;
                f.ext = pr.ext;
                f.h = nullptr;
            }
            e = launch_prep<true>(pr, st, tm);
            if (e != hipSuccess) return e;
            return mx4_gemm(pr.xc, pr.xs, codes, scales, sl.Y, M, N, L.K, f, st, tm);
        }
        case Mx4Path::kDequant: break;
    }
    // W's values are exact in bf16: the bf16 layer on them
    pr.wc = codes;
    pr.ws = scales;
    pr.W = reinterpret_cast<uint16_t*>(ws + sp.own);
    sl.W = pr.W;
    L.workspace = ws + sp.h;
    const bool beside = ext_ok && gemm_bf16_plan(M, N, L.K).tks < 2;
    if (beside) {
        if (pads) e = pad_ranks();
        if (e != hipSuccess) return e;
        pr.ext = reinterpret_cast<uint16_t*>(ws + sp.h);
        pr.h = reinterpret_cast<float*>(ws + sp.planes);
        pr.hs = prep_ranges(L.K, pr.n_items);
        pr.hkc = (cdiv(L.K, pr.hs) + 31) / 32 * 32;
    } else {
        pr.n_items = 0;
    }
    e = launch_prep<false>(pr, st, tm);
    if (e != hipSuccess) return e;
    return beside ? tiled_forward_ready(L, sl, pr.ext, st, tm) : lora_forward_bf16(L, st, tm);
}

}  // namespace lora
