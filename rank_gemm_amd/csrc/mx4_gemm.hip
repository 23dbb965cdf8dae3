// The tiled GEMM of MXFP4 operands (x rounded to 4 bits in plan order, W in 4
// bits): gemm_tile.h's pipeline with the scaled 16x16x128 product. 8192 x 4096
// -> 14336 takes 255 to 290 us by box and clock (median of event times 262, 3.7
// PFLOP/s), base-only 230 to 240. A step of 256 k takes 1.55 to 1.60 us (slopes of
// 8192 x 4096 .. 16384 -> 14336) for 0.97 us of matrix time (2048 cycles at 2.1
// GHz; the matrix cores are busy 49% of the kernel's cycles). It is not memory: a
// step that loads the same lines again and again takes 1.51. With every load
// answered by zeros it takes 1.03, but zeros also spare the matrix cores power;
// what the rest is has not been established. The stores are 8 us of the kernel,
// 16 base-only.
#include "gemm_tile.h"
#include "mx4_linear.h"

namespace lora {

template <int BM, int BN, int WM, int WN, int NS, bool EPI, bool KTAIL, bool BUF>
__global__ __launch_bounds__(64 * WM * WN, 1)
__attribute__((amdgpu_waves_per_eu(WM * WN / 4, WM * WN / 4))) void mx4_tile_kernel(
    const uint16_t* __restrict__ xc, const uint8_t* __restrict__ xs, const uint16_t* __restrict__ wc,
    const uint8_t* __restrict__ wsc, uint16_t* __restrict__ Y, int M, int N, int K16, int tiles_m, int tiles_n,
    Fuse f) {
    gemm_tile<BM, BN, WM, WN, NS, EPI, KTAIL, false, BUF, true>(xc, wc, Y, M, N, K16, tiles_m, tiles_n, f,
                                                                SplitOut{}, xs, wsc);
}

// BUF: loads through buffer resources. The expand runs as extra K steps, in
// the 128-row tile also in the epilogue.
template <int BM, int BN, int WM, int WN, int NS, bool BUF>
static hipError_t launch_mx4(const uint8_t* xc, const uint8_t* xs, const uint8_t* wc, const uint8_t* wsc, uint16_t* Y,
                             int M, int N, int K16, const Fuse& f, hipStream_t st, StageTimer* tm) {
    const int tiles_m = cdiv(M, BM), tiles_n = cdiv(N, BN);
    const bool ktail = K16 % 64 != 0;
    auto ker = ktail ? mx4_tile_kernel<BM, BN, WM, WN, NS, false, true, BUF>
                     : mx4_tile_kernel<BM, BN, WM, WN, NS, false, false, BUF>;
    if constexpr (BM == 128) {
        if (f.adapters && !f.ext)
            ker = ktail ? mx4_tile_kernel<BM, BN, WM, WN, NS, true, true, BUF>
                        : mx4_tile_kernel<BM, BN, WM, WN, NS, true, false, BUF>;
    }
    return launch(tm, "mx4_gemm", ker, dim3(tiles_m * tiles_n), dim3(64 * WM * WN), st, (const uint16_t*)xc, xs,
                  (const uint16_t*)wc, wsc, Y, M, N, K16, tiles_m, tiles_n, f);
}

hipError_t mx4_gemm(const uint8_t* xc, const uint8_t* xs, const uint8_t* wc, const uint8_t* wsc, uint16_t* Y, int M,
                    int N, int K, const Fuse& f, hipStream_t st, StageTimer* tm) {
    const int K16 = (int)(mx4_row_bytes(K) / 2);  // a row's bytes in the 16-bit units the tile counts in
    const bool extra = !f.adapters || f.ext;
    // the macro tile with the least (rounds of 256 tiles) x (time of one
    // tile); relative times measured at K = 4096 with every CU busy (a tile
    // alone: 64 x 128 8 us, 128 x 128 11 us, 256 x 128 17 us)
    struct Cand {
        int bm, bn;
        double t;
    };
    constexpr Cand cands[] = {{256, 256, 38.0}, {256, 128, 22.0}, {128, 128, 13.5}, {64, 128, 9.0}};
    int best = 2;  // 128 x 128 has the epilogue form of the expand
    double cost = 0.0;
    for (int c = 0; c < 4 && extra; ++c) {
        if (c == 0 && !tile_buffers_fit(M, N, K16, 256, f)) continue;
        const int64_t n = (int64_t)cdiv(M, cands[c].bm) * cdiv(N, cands[c].bn);
        const double t = (double)((n + 255) / 256) * cands[c].t;
        if (cost == 0.0 || t < cost) {
            cost = t;
            best = c;
        }
    }
    switch (best) {
        case 0: return launch_mx4<256, 256, 2, 2, 2, true>(xc, xs, wc, wsc, Y, M, N, K16, f, st, tm);
        case 1: return launch_mx4<256, 128, 4, 2, 2, false>(xc, xs, wc, wsc, Y, M, N, K16, f, st, tm);
        case 2: return launch_mx4<128, 128, 2, 4, 3, false>(xc, xs, wc, wsc, Y, M, N, K16, f, st, tm);
        default: return launch_mx4<64, 128, 2, 4, 4, false>(xc, xs, wc, wsc, Y, M, N, K16, f, st, tm);
    }
}

}  // namespace lora
