// MXFP4 rows to and from values, and scale bytes in row order to the tiles
// the products read (format: mx4_format.h). Memory-bound: each value is read and
// each code written once; the arithmetic is a maximum over 32 values and the
// hardware's scaled conversion. 14336 x 4096 bf16: 24.8 us to codes and 30.1 us
// back, 6.0 and 4.9 TB/s of what each moves (149 MB; part of it stays in the
// memory-side cache between calls), where a 1 GiB copy reaches 5.1 TB/s; 16 rows
// are a launch (4 us with its event pair).
#include "kernels.h"
#include "mx4_tile.h"

namespace lora {

template <class T>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(const T* __restrict__ src, int64_t rows, int64_t K,
                                                           uint8_t* __restrict__ codes,
                                                           uint8_t* __restrict__ scales) {
    __shared__ uint8_t st[kMxTileBytes];
    const int64_t mat = blockIdx.z;
    quantize_tile<T, 256>(src + mat * rows * K, rows, K, nullptr, codes + mat * rows * mx4_row_bytes(K),
                          scales + mat * mx4_scale_bytes(rows, K), blockIdx.x, blockIdx.y, st);
}

template <class T>
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ scales, int64_t rows,
                                                             int64_t K, T* __restrict__ dst) {
    __shared__ uint8_t st[kMxTileBytes];
    const int64_t mat = blockIdx.z;
    dequantize_tile<T, 256>(codes + mat * rows * mx4_row_bytes(K), scales + mat * mx4_scale_bytes(rows, K), rows, K,
                            dst + mat * rows * K, blockIdx.x, blockIdx.y, st);
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
static hipError_t quantize(const void* src, int64_t batch, int64_t rows, int64_t K, uint8_t* codes, uint8_t* scales,
                           hipStream_t st, StageTimer* tm) {
    return launch(tm, "mx4_quantize", mx4_quantize_kernel<T>, mx4_grid(batch, rows, K), dim3(256), st,
                  (const T*)src, rows, K, codes, scales);
}

hipError_t mx4_quantize(int dtype, const void* src, int64_t batch, int64_t rows, int64_t K, uint8_t* codes,
                        uint8_t* scales, hipStream_t st, StageTimer* tm) {
    return dtype == 1 ? quantize<uint16_t>(src, batch, rows, K, codes, scales, st, tm)
                      : quantize<float>(src, batch, rows, K, codes, scales, st, tm);
}

template <class T>
static hipError_t dequantize(const uint8_t* codes, const uint8_t* scales, int64_t batch, int64_t rows, int64_t K,
                             void* dst, hipStream_t st, StageTimer* tm) {
    return launch(tm, "mx4_dequantize", mx4_dequantize_kernel<T>, mx4_grid(batch, rows, K), dim3(256), st, codes,
                  scales, rows, K, (T*)dst);
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
