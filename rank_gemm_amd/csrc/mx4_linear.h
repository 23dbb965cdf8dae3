// Pieces of the MXFP4 linear layer (internal interface).
#pragma once

#include "fuse.h"
#include "mx4_format.h"

namespace lora {

// y = xhat What^T with the expand of f: x's codes and scales in plan order,
// tile rows of T of any size; f.ext (extra K steps) or f.h (epilogue).
hipError_t mx4_gemm(const uint8_t* xc, const uint8_t* xs, const uint8_t* wc, const uint8_t* wsc, uint16_t* Y, int M,
                    int N, int K, const Fuse& f, hipStream_t st, StageTimer* tm);

}  // namespace lora
