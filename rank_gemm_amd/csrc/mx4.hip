// MXFP4 rows to and from values, and scale bytes in row order to the tiles
// the products read (format: mx4_format.h). Memory-bound: each value is read and
// each code written once; the arithmetic is a maximum over 32 values and the
// hardware's scaled conversion.
#include "kernels.h"
#include "mx4.h"

namespace lora {

// One workgroup per scale tile (64 rows x 256 k): a row's piece of 256
// values is taken by 32 lanes of 8 values, so a wave's loads and code stores
// are whole 128-byte lines of two rows. Four lanes hold a block; its largest
// magnitude is taken across them on the bit patterns (an integer maximum of
// non-negative floats orders NaN last, so one non-finite value marks the
// block). The tile's scales gather in LDS and go out as words.
template <class T, bool VEC>
__device__ __forceinline__ void load8(const T* __restrict__ p, int n, float (&v)[8]) {
    if constexpr (sizeof(T) == 2) {
        if constexpr (VEC) {
            const u32x4 w = *as_global<u32x4>(p);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[2 * e] = __uint_as_float(w[e] << 16);
                v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
            }
            return;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < n ? bf16_to_f32(p[e]) : 0.f;
    } else {
        if constexpr (VEC) {
            const f32x4 a = as_global<f32x4>(p)[0], b = as_global<f32x4>(p)[1];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = a[e];
                v[4 + e] = b[e];
            }
            return;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < n ? p[e] : 0.f;
    }
}

template <class T, bool VEC>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(const T* __restrict__ src, int64_t rows, int64_t K,
                                                           const int32_t* __restrict__ order,
                                                           uint8_t* __restrict__ codes,
                                                           uint8_t* __restrict__ scales) {
    __shared__ uint8_t st[kMxTileBytes];
    const int tid = threadIdx.x, ln = tid & 31;
    const int64_t k0 = (int64_t)blockIdx.x * 256, r0 = (int64_t)blockIdx.y * 64, mat = blockIdx.z;
    const int64_t rb = mx4_row_bytes(K);
    src += mat * rows * K;
    codes += mat * rows * rb;
    const int64_t k = k0 + ln * 8;
    const int n = (int)max(int64_t(0), min(int64_t(8), K - k));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + i * 8 + (tid >> 5);
        const bool ok = r < rows && n > 0;
        float v[8];
        if (ok) load8<T, VEC>(src + (order ? order[r] : r) * K + k, n, v);
        else
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.f;
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
        m = max(m, (uint32_t)__shfl_xor((int)m, 1));
        m = max(m, (uint32_t)__shfl_xor((int)m, 2));
        const uint32_t b = mx4_scale_byte(m);
        // k / 2 bytes into the row: inside it, as a row is whole blocks
        if (r < rows && k < rb * 2) *reinterpret_cast<uint32_t*>(codes + r * rb + k / 2) = mx4_codes8(v, b);
        if ((ln & 3) == 0) st[mx4_tile_off(i * 8 + (tid >> 5), ln >> 2)] = (uint8_t)b;
    }
    __syncthreads();
    if (tid < kMxTileBytes / 4) {
        uint8_t* tile = scales + mat * mx4_scale_bytes(rows, K) + (blockIdx.y * mx4_k_tiles(K) + blockIdx.x) * kMxTileBytes;
        reinterpret_cast<uint32_t*>(tile)[tid] = reinterpret_cast<const uint32_t*>(st)[tid];
    }
}

template <class T, bool VEC>
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ scales, int64_t rows,
                                                             int64_t K, T* __restrict__ dst) {
    __shared__ uint8_t st[kMxTileBytes];
    const int tid = threadIdx.x, ln = tid & 31;
    const int64_t k0 = (int64_t)blockIdx.x * 256, r0 = (int64_t)blockIdx.y * 64, mat = blockIdx.z;
    const int64_t rb = mx4_row_bytes(K);
    codes += mat * rows * rb;
    dst += mat * rows * K;
    if (tid < kMxTileBytes / 4) {
        const uint8_t* tile = scales + mat * mx4_scale_bytes(rows, K) + (blockIdx.y * mx4_k_tiles(K) + blockIdx.x) * kMxTileBytes;
        reinterpret_cast<uint32_t*>(st)[tid] = reinterpret_cast<const uint32_t*>(tile)[tid];
    }
    const int64_t k = k0 + ln * 8;
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + i * 8 + (tid >> 5);
        c[i] = r < rows && k < K ? *reinterpret_cast<const uint32_t*>(codes + r * rb + k / 2) : 0u;
    }
    __syncthreads();
    const int n = (int)max(int64_t(0), min(int64_t(8), K - k));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + i * 8 + (tid >> 5);
        if (r >= rows || n == 0) continue;
        float v[8];
        mx4_f32x8(c[i], mx4_scale(st[mx4_tile_off(i * 8 + (tid >> 5), ln >> 2)]), v);
        T* p = dst + r * K + k;
        if constexpr (sizeof(T) == 2) {
            const u32x4 w{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                          pack_bf16x2(v[6], v[7])};
            if constexpr (VEC) {
                *reinterpret_cast<u32x4*>(p) = w;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < n) p[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
            }
        } else {
            if constexpr (VEC) {
                reinterpret_cast<f32x4*>(p)[0] = f32x4{v[0], v[1], v[2], v[3]};
                reinterpret_cast<f32x4*>(p)[1] = f32x4{v[4], v[5], v[6], v[7]};
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < n) p[e] = v[e];
            }
        }
    }
}

// scale bytes [rows][ceil(K / 32)] -> tiles; a thread writes one word
__global__ __launch_bounds__(128) void mx4_pack_kernel(const uint8_t* __restrict__ plain, int64_t rows, int64_t K,
                                                       uint8_t* __restrict__ scales) {
    const int64_t nb = (K + 31) / 32, mat = blockIdx.z;
    plain += mat * rows * nb;
    const int w = threadIdx.x, fr = (w >> 1) & 15, b = (w >> 5) + 4 * (w & 1);
    const int64_t blk = (int64_t)blockIdx.x * 8 + b, r0 = (int64_t)blockIdx.y * 64 + fr;
    uint32_t v = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (r0 + 16 * j < rows && blk < nb) v |= (uint32_t)plain[(r0 + 16 * j) * nb + blk] << (8 * j);
    uint8_t* tile = scales + mat * mx4_scale_bytes(rows, K) + (blockIdx.y * mx4_k_tiles(K) + blockIdx.x) * kMxTileBytes;
    reinterpret_cast<uint32_t*>(tile)[w] = v;
}

static dim3 mx4_grid(int64_t batch, int64_t rows, int64_t K) {
    return dim3((uint32_t)mx4_k_tiles(K), (uint32_t)((rows + 63) / 64), (uint32_t)batch);
}

template <class T>
static hipError_t quantize(const void* src, int64_t batch, int64_t rows, int64_t K, const int32_t* order,
                           uint8_t* codes, uint8_t* scales, hipStream_t st, StageTimer* tm) {
    const bool vec = K % 8 == 0 && (uintptr_t)src % 16 == 0;
    return launch(tm, "mx4_quantize", vec ? mx4_quantize_kernel<T, true> : mx4_quantize_kernel<T, false>,
                  mx4_grid(batch, rows, K), dim3(256), st, (const T*)src, rows, K, order, codes, scales);
}

hipError_t mx4_quantize(int dtype, const void* src, int64_t batch, int64_t rows, int64_t K, const int32_t* order,
                        uint8_t* codes, uint8_t* scales, hipStream_t st, StageTimer* tm) {
    return dtype == 1 ? quantize<uint16_t>(src, batch, rows, K, order, codes, scales, st, tm)
                      : quantize<float>(src, batch, rows, K, order, codes, scales, st, tm);
}

template <class T>
static hipError_t dequantize(const uint8_t* codes, const uint8_t* scales, int64_t batch, int64_t rows, int64_t K,
                             void* dst, hipStream_t st, StageTimer* tm) {
    const bool vec = K % 8 == 0 && (uintptr_t)dst % 16 == 0;
    return launch(tm, "mx4_dequantize", vec ? mx4_dequantize_kernel<T, true> : mx4_dequantize_kernel<T, false>,
                  mx4_grid(batch, rows, K), dim3(256), st, codes, scales, rows, K, (T*)dst);
}

hipError_t mx4_dequantize(int dtype, const uint8_t* codes, const uint8_t* scales, int64_t batch, int64_t rows,
                          int64_t K, void* dst, hipStream_t st, StageTimer* tm) {
    return dtype == 1 ? dequantize<uint16_t>(codes, scales, batch, rows, K, dst, st, tm)
                      : dequantize<float>(codes, scales, batch, rows, K, dst, st, tm);
}

hipError_t mx4_pack_scales(const uint8_t* plain, int64_t batch, int64_t rows, int64_t K, uint8_t* scales,
                           hipStream_t st) {
    return launch(nullptr, "mx4_pack", mx4_pack_kernel, mx4_grid(batch, rows, K), dim3(128), st, plain, rows, K,
                  scales);
}

}  // namespace lora
