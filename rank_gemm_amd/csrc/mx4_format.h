// MXFP4 operands of liblora (OCP Microscaling Formats 1.0): 32 consecutive
// values of a row share one scale 2^(b - 127), b a byte (255: not a number);
// each value is an E2M1 code (sign, 2 exponent bits, 1 mantissa bit).
//
// Codes: rows of mx4_row_bytes(K) = 16 ceil(K / 32) bytes, two codes a byte,
// the earlier value in the low four bits; a block is one 16-byte piece, and
// the codes past K in a row's last block are 0.
//
// Scales: tiles of 64 rows x 8 blocks (256 k), 512 bytes each, row groups
// first, then along K. Inside a tile the 16x16x128 matrix-core product's
// lane (fr, fc) = (row % 16, block % 4) finds its scales as the two
// consecutive words 2 (16 fc + fr) + h, h = block / 4 % 2, whose byte j
// belongs to row 16 j + fr of the group: one 8-byte read per lane covers 64
// rows x 256 k, and the instruction picks the byte of its 16-row block
// itself. Bytes of rows and blocks past the matrix are 0.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lora {

constexpr int kMxBlock = 32;
constexpr int kMxTileBytes = 512;  // scales of 64 rows x 256 k

__host__ __device__ inline int64_t mx4_row_bytes(int64_t K) { return (K + 31) / 32 * 16; }
__host__ __device__ inline int64_t mx4_k_tiles(int64_t K) { return (K + 255) / 256; }
__host__ __device__ inline int64_t mx4_scale_bytes(int64_t rows, int64_t K) {
    return (rows + 63) / 64 * mx4_k_tiles(K) * kMxTileBytes;
}

}  // namespace lora
