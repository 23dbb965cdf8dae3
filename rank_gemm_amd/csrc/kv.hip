// New keys and values into a paged cache: row rows[t] of the cache = k[t], v[t]
// (8-bit caches: the nearest E4M3 value of k / scale of the head, at most 448).
// Bound by memory: 8192 tokens of 8 heads of 128, bf16 (67 MB), 12.4 us, 5.4 TB/s;
// 64 tokens into 8 bits 3 us, a launch.
#include "common.h"
#include "kernels.h"

namespace lora {

// Nearest E4M3 value (ties to the even mantissa), at most 448 in magnitude;
// NaN stays NaN.
__device__ __forceinline__ float f8_range(float v) { return v != v ? v : __builtin_amdgcn_fmed3f(v, -448.f, 448.f); }
__device__ __forceinline__ uint32_t pack_f8x4(float a, float b, float c, float d) {
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(f8_range(a), f8_range(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f8_range(c), f8_range(d), r, true);
}

// A thread takes 8 values of a head's row: of k (blockIdx.y 0) or of v.
template <bool F8>
__global__ __launch_bounds__(256) void kv_append_kernel(KvCache c, const uint16_t* __restrict__ K,
                                                        const uint16_t* __restrict__ V, int64_t k_stride,
                                                        int64_t v_stride, const int64_t* __restrict__ rows, int T) {
    const int pieces = c.kv_heads * (c.dim / 8);
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t t = i / pieces;
    if (t >= T) return;
    const int piece = (int)(i - t * pieces), h = piece / (c.dim / 8), d = piece % (c.dim / 8) * 8;
    const int64_t row = rows[t];
    if (row < 0 || row >= (int64_t)c.n_pages * c.page_rows) return;
    const bool is_v = blockIdx.y != 0;
    const uint16_t* src = (is_v ? V + t * v_stride : K + t * k_stride) + h * c.dim + d;
    const u32x4 x = *as_global<u32x4>(src);
    const int64_t page = row / c.page_rows;
    const int64_t at = page * c.page_stride + (row - page * c.page_rows) * c.row_stride + h * c.head_stride + d;
    if constexpr (!F8) {
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(is_v ? c.v : c.k) + at) = x;
    } else {
        const float s = (is_v ? c.v_scale : c.k_scale)[h];
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = __uint_as_float(x[j] << 16) / s;
            f[2 * j + 1] = __uint_as_float(x[j] & 0xffff0000u) / s;
        }
        const u32x2 o = {pack_f8x4(f[0], f[1], f[2], f[3]), pack_f8x4(f[4], f[5], f[6], f[7])};
        *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(is_v ? c.v : c.k) + at) = o;
    }
}

hipError_t kv_append(const KvCache& c, bool f8, const uint16_t* k, const uint16_t* v, int64_t k_stride,
                     int64_t v_stride, const int64_t* rows, int T, hipStream_t st, StageTimer* tm) {
    const int64_t n = (int64_t)T * c.kv_heads * (c.dim / 8);
    return launch(tm, "kv_append", f8 ? kv_append_kernel<true> : kv_append_kernel<false>,
                  dim3((uint32_t)((n + 255) / 256), 2), dim3(256), st, c, k, v, k_stride, v_stride, rows, T);
}

}  // namespace lora
