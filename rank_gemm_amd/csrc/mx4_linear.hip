// The mixed-adapter linear layer over an MXFP4 base weight:
//   y[t_p] = bf16( act(x[t_p]) What^T + scale_s * h[p] B_s^T ),  h = x A_s^T
// What the values of the 4-bit codes, act the identity (16-bit activations)
// or the MXFP4 rounding of each row of x; the adapters always read x itself.
#include "fuse.h"
#include "mx4.h"
#include "mx4_linear.h"
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

// 64 sorted rows x 64 columns per workgroup, a wave 16 rows x 64 columns over
// all of K, operands straight from memory.
template <bool ACT4>
__global__ __launch_bounds__(256) void mx4_rows_kernel(const uint16_t* __restrict__ X,
                                                       const uint8_t* __restrict__ xc,
                                                       const uint8_t* __restrict__ xs,
                                                       const uint8_t* __restrict__ wc,
                                                       const uint8_t* __restrict__ wsc, uint16_t* __restrict__ Y,
                                                       int M, int N, int K, Fuse f) {
    __shared__ SlotMeta meta;
    __shared__ u32x4 stg[4 * 128];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int fr = lane & 15, fc = lane >> 4;
    const MetaView mv = stage_meta(f, &meta);
    __syncthreads();
    const int n0 = blockIdx.x * 64, m0 = blockIdx.y * 64, p0 = m0 + 16 * wave;
    const int64_t rb = mx4_row_bytes(K), kts = mx4_k_tiles(K);
    const int nb = (K + 31) / 32;
    const int p = min(p0 + fr, M - 1);
    const uint16_t* xrow = X + (int64_t)f.token_order[p] * K;
    const uint8_t* xq = xc + (int64_t)p * rb;
    f32x4 acc[1][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[0][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int kt = 0; kt < kts; ++kt) {
        const u32x2 ws = *reinterpret_cast<const u32x2*>(wsc + ((int64_t)blockIdx.x * kts + kt) * kMxTileBytes + lane * 8);
        u32x2 xsc{0, 0};
        if constexpr (ACT4) {
            xsc = *reinterpret_cast<const u32x2*>(xs + ((int64_t)blockIdx.y * kts + kt) * kMxTileBytes + lane * 8);
            xsc[0] >>= 8 * wave;
            xsc[1] >>= 8 * wave;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int blk = kt * 8 + h * 4 + fc;
            u32x4 w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = *or_zero(blk < nb, wc + (int64_t)min(n0 + 16 * j + fr, N - 1) * rb + blk * 16);
            if constexpr (ACT4) {
                const u32x4 x = *or_zero(blk < nb, xq + blk * 16);
                acc[0][0] = mfma_mx4<0, 0>(w[0], x, acc[0][0], ws[h], xsc[h]);
                acc[0][1] = mfma_mx4<1, 0>(w[1], x, acc[0][1], ws[h], xsc[h]);
                acc[0][2] = mfma_mx4<2, 0>(w[2], x, acc[0][2], ws[h], xsc[h]);
                acc[0][3] = mfma_mx4<3, 0>(w[3], x, acc[0][3], ws[h], xsc[h]);
            } else {
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int k = blk * 32 + 8 * m;
                    const u32x4 x = *or_zero(k < K, xrow + k);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[0][j] = mfma16x16x32(mx4_bf16x8(w[j][m], mx4_scale(ws[h] >> (8 * j) & 255)), x, acc[0][j]);
                }
            }
        }
    }
    fused_expand<1, 4>(acc, f, mv, p0, n0, M, N, lane);
    store_tile<1, 4>(acc, reinterpret_cast<char*>(stg) + wave * 2048, Y, f.token_order, p0, n0, M, N, lane);
}

// rows of any width -> rows of Kp elements (a multiple of 8), zeros behind
// the row's end: the kernels read rows in 16-byte pieces
__global__ __launch_bounds__(256) void pad_rows_kernel(const uint16_t* __restrict__ src, int64_t rows, int K, int Kp,
                                                       uint16_t* __restrict__ dst) {
    const int64_t r = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    const int k = blockIdx.x * 256 + threadIdx.x;
    if (r < rows && k < Kp) dst[r * Kp + k] = k < K ? src[r * K + k] : uint16_t(0);
}

static inline size_t a256(size_t n) { return (n + 255) & ~size_t(255); }

// Workspace: padded rows of x and A (d_in not a multiple of 8), the 4-bit
// activations, then the shrink's h and planes.
struct Mx4Space {
    size_t xpad, apad, codes, scales, shrink, total;
};
static Mx4Space mx4_space(int M, int K, int S, int r_max, bool act4) {
    const size_t Kp = (K + 7) / 8 * 8;
    Mx4Space s{};
    size_t o = 0;
    s.xpad = o;
    if (K % 8) o += a256((size_t)M * Kp * 2);
    s.apad = o;
    if (K % 8) o += a256((size_t)S * r_max * Kp * 2);
    s.codes = o;
    if (act4) o += a256((size_t)M * mx4_row_bytes(K));
    s.scales = o;
    if (act4) o += a256((size_t)mx4_scale_bytes(M, K));
    s.shrink = o;
    o += tiled_workspace(M, r_max);
    s.total = o;
    return s;
}

size_t mx4_linear_workspace(int M, int N, int K, int S, int r_max, bool act4) {
    (void)N;
    return M > 0 ? mx4_space(M, K, S, r_max, act4).total : 0;
}

static hipError_t pad_rows(const uint16_t* src, int64_t rows, int K, int Kp, uint16_t* dst, hipStream_t st,
                           StageTimer* tm) {
    const uint32_t gy = (uint32_t)(rows < 65535 ? rows : 65535);
    return launch(tm, "pad_rows", pad_rows_kernel, dim3((Kp + 255) / 256, gy, (uint32_t)((rows + gy - 1) / gy)),
                  dim3(256), st, src, rows, K, Kp, dst);
}

hipError_t mx4_linear(const LinearArgs& L0, const uint8_t* codes, const uint8_t* scales, bool act4, hipStream_t st,
                      StageTimer* tm) {
    LinearArgs L = L0;
    SliceArgs sl = L.slice[0];
    const int M = L.M, N = sl.N;
    char* ws = static_cast<char*>(L.workspace);
    const Mx4Space sp = mx4_space(M, L.K, L.S, L.r_max, act4);
    hipError_t e = hipSuccess;
    const uint8_t *xc = nullptr, *xs = nullptr;
    if (act4) {
        xc = reinterpret_cast<uint8_t*>(ws + sp.codes);
        xs = reinterpret_cast<uint8_t*>(ws + sp.scales);
        e = mx4_quantize(1, L.X, 1, M, L.K, L.token_order, const_cast<uint8_t*>(xc), const_cast<uint8_t*>(xs), st, tm);
        if (e != hipSuccess) return e;
    }
    if (L.K % 8) {
        const int Kp = (L.K + 7) / 8 * 8;
        uint16_t* xp = reinterpret_cast<uint16_t*>(ws + sp.xpad);
        uint16_t* ap = reinterpret_cast<uint16_t*>(ws + sp.apad);
        e = pad_rows(L.X, M, L.K, Kp, xp, st, tm);
        if (e == hipSuccess && L.adapters) e = pad_rows(sl.A_pool, (int64_t)L.S * L.r_max, L.K, Kp, ap, st, tm);
        if (e != hipSuccess) return e;
        L.X = xp;
        sl.A_pool = ap;
        L.K = Kp;
    }
    float* h = reinterpret_cast<float*>(ws + sp.shrink);
    Fuse f{L.token_order, L.slot_indptr, h, sl.B_pool, sl.rank, sl.scale, L.S, L.r_max, 1, 0, L.adapters,
           nullptr, (L.r_max + 7) & ~7};
    const bool tiled = act4 && M > 64;
    if (tiled && L.r_max % 8 == 0 && L.S <= kMetaSlots) {
        f.ext = reinterpret_cast<uint16_t*>(h);
        f.h = nullptr;
    }
    if (L.adapters) {
        e = tiled_shrink(L, sl, ws + sp.shrink, f.ext ? nullptr : h, const_cast<uint16_t*>(f.ext), st, tm);
        if (e != hipSuccess) return e;
    }
    if (tiled) return mx4_gemm(xc, xs, codes, scales, sl.Y, M, N, L.K, f, st, tm);
    return launch(tm, "mx4_rows", act4 ? mx4_rows_kernel<true> : mx4_rows_kernel<false>,
                  dim3(cdiv(N, 64), cdiv(M, 64)), dim3(256), st, L.X, xc, xs, codes, scales, sl.Y, M, N, L.K, f);
}

}  // namespace lora
