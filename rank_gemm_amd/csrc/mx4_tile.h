// A tile of MXFP4 rows (64 rows x 256 k, one scale tile) from and to values,
// by one workgroup.
#pragma once

#include "mx4.h"

namespace lora {

// Eight consecutive values of a row, as loaded. Rows of any width start on
// the element's own boundary only; global memory takes 16-byte accesses at
// any such address, so one form serves every width.
template <class T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
    typedef u32x4 V __attribute__((aligned(2)));
    u32x4 v;
    __device__ __forceinline__ void load(const void* p) { v = *(gptr<V>)p; }
    __device__ __forceinline__ void to(float (&f)[8]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[2 * e] = __uint_as_float(v[e] << 16);
            f[2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void put(uint16_t* p, const float (&f)[8]) {
        *reinterpret_cast<V*>(p) = V{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                     pack_bf16x2(f[6], f[7])};
    }
    static __device__ __forceinline__ float one(uint16_t b) { return bf16_to_f32(b); }
    static __device__ __forceinline__ uint16_t back(float f) { return f32_to_bf16(f); }
};
template <>
struct Raw8<float> {
    typedef f32x4 V __attribute__((aligned(4)));
    f32x4 v[2];
    __device__ __forceinline__ void load(const void* p) {
        v[0] = ((gptr<V>)p)[0];
        v[1] = ((gptr<V>)p)[1];
    }
    __device__ __forceinline__ void to(float (&f)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = v[e >> 2][e & 3];
    }
    static __device__ __forceinline__ void put(float* p, const float (&f)[8]) {
        reinterpret_cast<V*>(p)[0] = V{f[0], f[1], f[2], f[3]};
        reinterpret_cast<V*>(p)[1] = V{f[4], f[5], f[6], f[7]};
    }
    static __device__ __forceinline__ float one(float f) { return f; }
    static __device__ __forceinline__ float back(float f) { return f; }
};
static __device__ const u32x4 kZeros32[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};

// One workgroup per scale tile (64 rows x 256 k): a row's piece of 256
// values is taken by 32 lanes of 8 values, so a wave's loads and code stores
// are whole 128-byte lines of two rows, all loads issued before the first is
// used. Four lanes hold a block; its largest magnitude is taken across them on
// the bit patterns (an integer maximum of non-negative floats orders NaN
// last, so one non-finite value marks the block). The tile's scales gather in
// LDS and go out as words.
// With order, row r of the result is source row order[r]. st: LDS of a tile.
template <class T, int THREADS>
__device__ __forceinline__ void quantize_tile(const T* __restrict__ src, int64_t rows, int64_t K,
                                              const int32_t* __restrict__ order, uint8_t* __restrict__ codes,
                                              uint8_t* __restrict__ scales, int bx, int by, uint8_t* st) {
    constexpr int STEP = THREADS / 32, N = 64 / STEP;  // rows at once, rows per thread
    const int tid = threadIdx.x, ln = tid & 31;
    const int64_t k = (int64_t)bx * 256 + ln * 8, r0 = (int64_t)by * 64 + (tid >> 5);
    const int64_t rb = mx4_row_bytes(K);
    const int n = (int)max(int64_t(0), min(int64_t(8), K - k));
    const T* row[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t r = min(r0 + i * STEP, rows - 1);
        row[i] = src + (order ? order[r] : r) * K + k;
    }
    Raw8<T> raw[N];
#pragma unroll
    for (int i = 0; i < N; ++i)  // rows past the end and partial pieces load zeros
        raw[i].load(n == 8 && r0 + i * STEP < rows ? (const void*)row[i] : (const void*)kZeros32);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t r = r0 + i * STEP;
        float v[8];
        raw[i].to(v);
        if (n > 0 && n < 8 && r < rows)  // the row's last piece
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < n ? Raw8<T>::one(row[i][e]) : 0.f;
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
        m = max(m, (uint32_t)__shfl_xor((int)m, 1));
        m = max(m, (uint32_t)__shfl_xor((int)m, 2));
        const uint32_t b = mx4_scale_byte(m);
        // k / 2 bytes into the row: inside it, as a row is whole blocks
        if (r < rows && k < rb * 2) *reinterpret_cast<uint32_t*>(codes + r * rb + k / 2) = mx4_codes8(v, b);
        if ((ln & 3) == 0) st[mx4_tile_off(i * STEP + (tid >> 5), ln >> 2)] = (uint8_t)b;
    }
    __syncthreads();
    if (tid < kMxTileBytes / 4) {
        uint8_t* tile = scales + (by * mx4_k_tiles(K) + bx) * kMxTileBytes;
        reinterpret_cast<uint32_t*>(tile)[tid] = reinterpret_cast<const uint32_t*>(st)[tid];
    }
}

// The reverse, a tile of codes and scales to values.
template <class T, int THREADS>
__device__ __forceinline__ void dequantize_tile(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                int64_t rows, int64_t K, T* __restrict__ dst, int bx, int by,
                                                uint8_t* st) {
    constexpr int STEP = THREADS / 32, N = 64 / STEP;
    const int tid = threadIdx.x, ln = tid & 31;
    const int64_t k = (int64_t)bx * 256 + ln * 8, r0 = (int64_t)by * 64 + (tid >> 5);
    const int64_t rb = mx4_row_bytes(K);
    if (tid < kMxTileBytes / 4) {
        const uint8_t* tile = scales + (by * mx4_k_tiles(K) + bx) * kMxTileBytes;
        reinterpret_cast<uint32_t*>(st)[tid] = reinterpret_cast<const uint32_t*>(tile)[tid];
    }
    uint32_t c[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {  // clamped: the extra values are not stored
        const int64_t r = min(r0 + i * STEP, rows - 1);
        c[i] = *as_global<uint32_t>(codes + r * rb + min(k, rb * 2 - 8) / 2);
    }
    __syncthreads();
    const int n = (int)max(int64_t(0), min(int64_t(8), K - k));
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t r = r0 + i * STEP;
        if (r >= rows || n == 0) continue;
        float v[8];
        mx4_f32x8(c[i], mx4_scale(st[mx4_tile_off(i * STEP + (tid >> 5), ln >> 2)]), v);
        T* p = dst + r * K + k;
        if (n == 8) {
            Raw8<T>::put(p, v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) p[e] = Raw8<T>::back(v[e]);
        }
    }
}

}  // namespace lora
