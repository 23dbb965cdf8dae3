// A tile of MXFP4 rows (64 rows x 256 k, one scale tile) from and to values,
// by one workgroup.
#pragma once

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

// With order, row r of the result is source row order[r]. st: LDS of a tile.
template <class T, bool VEC, int THREADS>
__device__ __forceinline__ void quantize_tile(const T* __restrict__ src, int64_t rows, int64_t K,
                                              const int32_t* __restrict__ order, uint8_t* __restrict__ codes,
                                              uint8_t* __restrict__ scales, int bx, int by, uint8_t* st) {
    constexpr int STEP = THREADS / 32;  // rows at once
    const int tid = threadIdx.x, ln = tid & 31;
    const int64_t k0 = (int64_t)bx * 256, r0 = (int64_t)by * 64;
    const int64_t rb = mx4_row_bytes(K);
    const int64_t k = k0 + ln * 8;
    const int n = (int)max(int64_t(0), min(int64_t(8), K - k));
#pragma unroll
    for (int i = 0; i < 64 / STEP; ++i) {
        const int64_t r = r0 + i * STEP + (tid >> 5);
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
        if ((ln & 3) == 0) st[mx4_tile_off(i * STEP + (tid >> 5), ln >> 2)] = (uint8_t)b;
    }
    __syncthreads();
    if (tid < kMxTileBytes / 4) {
        uint8_t* tile = scales + (by * mx4_k_tiles(K) + bx) * kMxTileBytes;
        reinterpret_cast<uint32_t*>(tile)[tid] = reinterpret_cast<const uint32_t*>(st)[tid];
    }
}

// The reverse, a tile of codes and scales to values.
template <class T, bool VEC, int THREADS>
__device__ __forceinline__ void dequantize_tile(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                int64_t rows, int64_t K, T* __restrict__ dst, int bx, int by,
                                                uint8_t* st) {
    constexpr int STEP = THREADS / 32;
    const int tid = threadIdx.x, ln = tid & 31;
    const int64_t k0 = (int64_t)bx * 256, r0 = (int64_t)by * 64;
    const int64_t rb = mx4_row_bytes(K);
    if (tid < kMxTileBytes / 4) {
        const uint8_t* tile = scales + (by * mx4_k_tiles(K) + bx) * kMxTileBytes;
        reinterpret_cast<uint32_t*>(st)[tid] = reinterpret_cast<const uint32_t*>(tile)[tid];
    }
    const int64_t k = k0 + ln * 8;
    uint32_t c[64 / STEP];
#pragma unroll
    for (int i = 0; i < 64 / STEP; ++i) {
        const int64_t r = r0 + i * STEP + (tid >> 5);
        c[i] = r < rows && k < K ? *reinterpret_cast<const uint32_t*>(codes + r * rb + k / 2) : 0u;
    }
    __syncthreads();
    const int n = (int)max(int64_t(0), min(int64_t(8), K - k));
#pragma unroll
    for (int i = 0; i < 64 / STEP; ++i) {
        const int64_t r = r0 + i * STEP + (tid >> 5);
        if (r >= rows || n == 0) continue;
        float v[8];
        mx4_f32x8(c[i], mx4_scale(st[mx4_tile_off(i * STEP + (tid >> 5), ln >> 2)]), v);
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

}  // namespace lora
