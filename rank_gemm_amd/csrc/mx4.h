// Device helpers on MXFP4 operands (their layout: mx4_format.h).
#pragma once

#include "common.h"
#include "mx4_format.h"

namespace lora {

// offset inside its tile of the scale of row r, block b (both taken in the tile)
__host__ __device__ constexpr int mx4_tile_off(int r, int b) {
    return ((((b & 3) * 16 + (r & 15)) * 2 + (b >> 2 & 1)) << 2) + (r >> 4 & 3);
}
__host__ __device__ inline int64_t mx4_scale_off(int64_t r, int64_t b, int64_t k_tiles) {
    return ((r >> 6) * k_tiles + (b >> 3)) * kMxTileBytes + mx4_tile_off((int)(r & 63), (int)(b & 7));
}

// 2^(b - 127) as fp32 (b = 0: the subnormal 2^-127; b = 255: NaN)
__device__ __forceinline__ float mx4_scale(uint32_t b) {
    const uint32_t bits = b == 255 ? 0x7fc00000u : b == 0 ? 0x00400000u : b << 23;
    return __uint_as_float(bits);
}

// The shared scale's byte for a block whose largest magnitude has these fp32
// bits: floor(log2) - 2 (the largest E2M1 exponent), from the exponent field;
// a block with an infinity or a NaN has no scale (255).
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t max_bits) {
    const uint32_t e = max_bits >> 23;
    return e == 255 ? 255u : e > 2 ? e - 2 : 0u;
}

// Eight fp32 values -> eight codes of scale 2^(b - 127), nearest, ties to the
// even mantissa, at most 6. The hardware conversion divides by the scale and
// rounds so. Scale 2^-127 is a subnormal fp32 operand: there (the block's
// largest magnitude under 2^-124) the values are first multiplied by 2^64,
// exactly, and the scale with them.
__device__ __forceinline__ uint32_t mx4_codes8(const float (&v)[8], uint32_t b) {
    if (b == 255) return 0;
    const bool tiny = b < 64;
    const float up = tiny ? 0x1p64f : 1.f;
    const float sc = __uint_as_float((tiny ? b + 64 : b) << 23);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0] * up, v[1] * up, sc, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2] * up, v[3] * up, sc, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4] * up, v[5] * up, sc, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6] * up, v[7] * up, sc, 3);
    return c;
}

// Eight codes -> eight bf16 values (a matrix-core fragment). Exact while
// 2^(b - 127) keeps 0.5 times it representable; a product with a scale under
// 2^-125 or over 2^125 may round or overflow as bf16 does.
__device__ __forceinline__ u32x4 mx4_bf16x8(uint32_t c, float sc) {
    u32x4 r;
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 0));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 1));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 2));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 3));
    return r;
}

// The other operand of products of 16-bit values with decoded 4-bit rows. A
// lane (fr, fc) of the 4-bit side holds block fc of a 128-wide half tile, so
// product m of the half (8 of each block's codes) needs k = 32 fc + 8 m of
// the 16-bit row. Loaded in that order, a lane group's pieces lie 64 bytes
// apart; so load i takes k = 32 i + 8 fc (64 consecutive bytes of a row) and
// the four pieces are transposed across the four lane groups in registers.
__device__ __forceinline__ void mx4_transpose(u32x4 (&x)[4]) {
    auto swap32 = [](uint32_t& a, uint32_t& b) {  // a's upper half lanes <-> b's lower
        const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(a, b, false, false));
        a = r[0];
        b = r[1];
    };
    auto swap16 = [](uint32_t& a, uint32_t& b) {  // a's odd groups of 16 <-> b's even ones
        const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a, b, false, false));
        a = r[0];
        b = r[1];
    };
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        uint32_t a = x[0][d], b = x[1][d], c = x[2][d], e = x[3][d];
        swap32(a, c);
        swap32(b, e);
        swap16(a, b);
        swap16(c, e);
        x[0][d] = a;
        x[1][d] = b;
        x[2][d] = c;
        x[3][d] = e;
    }
}

// Eight codes -> eight fp32 values of scale 1, times sc in fp32 (exact but
// for results under 2^-149 or over the fp32 range).
__device__ __forceinline__ void mx4_f32x8(uint32_t c, float sc, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t q = c >> (4 * e), m = q & 7;
        // m < 2: 0 or 0.5; else (1 + (m & 1) / 2) 2^(m / 2 - 1)
        const uint32_t bits = m < 2 ? (m ? 0x3f000000u : 0u) : ((126 + (m >> 1)) << 23) | (m & 1) << 22;
        v[e] = __uint_as_float(bits | (q & 8) << 28) * sc;
    }
}

}  // namespace lora
