// The paged key-value cache of a decode step and the attention that reads it:
//   append: rows[t] of the cache = k[t], v[t] (8-bit caches: the nearest E4M3
//           value of k / scale of the head, at most 448)
//   decode: out[b][h] = sum_j p_j v_j,  p = softmax_j(scale q . k_j) over the
//           request's positions j, read through its row of the page table.
// A request's position j lies in row j % page_rows of page table[b][j /
// page_rows]. Positions whose page is outside the cache are left out, so no
// table makes a kernel read past it.
#include "common.h"
#include "kernels.h"

namespace lora {

// ----------------------------------------------------------------- append --
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

// ----------------------------------------------------------------- decode --
// The positions [lo, hi) a request attends to.
__device__ __forceinline__ void attn_range(const AttnArgs& a, int b, int* lo, int* hi) {
    const int n = min(max(a.lengths[b], 0), a.width * a.c.page_rows);
    *lo = a.window > 0 ? max(n - a.window, 0) : 0;
    *hi = n;
}

// One workgroup per request and head, its waves taking positions in turn: a
// running maximum m, sum l and output o a wave (base 2), joined at the end.
// Lane i of a wave holds dimensions i, i + 64, ...
template <bool F8>
__global__ __launch_bounds__(256) void attn_decode_kernel(AttnArgs a) {
    constexpr int N = kAttnMaxDim / 64;
    __shared__ float sm[4], sl[4], so[4][kAttnMaxDim];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = blockIdx.x, b = blockIdx.y;
    const int D = a.c.dim, hk = h / (a.heads / a.c.kv_heads);
    const float ks = F8 ? a.c.k_scale[hk] : 1.f, vs = F8 ? a.c.v_scale[hk] : 1.f;
    float q[N], o[N], m = -3.402823466e38f, l = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int d = lane + 64 * i;
        q[i] = d < D ? bf16_to_f32(a.q[b * a.q_stride + (int64_t)h * D + d]) : 0.f;
        o[i] = 0.f;
    }
    auto value = [&](const void* base, int64_t at, int d) {
        if (d >= D) return 0.f;
        if constexpr (F8)
            return __builtin_amdgcn_cvt_f32_fp8(static_cast<const uint8_t*>(base)[at + d], 0);
        else
            return bf16_to_f32(static_cast<const uint16_t*>(base)[at + d]);
    };
    int lo, hi;
    attn_range(a, b, &lo, &hi);
    for (int j = lo + wave; j < hi; j += 4) {
        const int pi = j / a.c.page_rows, page = a.table[b * a.table_stride + pi];
        if (page < 0 || page >= a.c.n_pages) continue;
        const int64_t at = page * a.c.page_stride + (int64_t)(j - pi * a.c.page_rows) * a.c.row_stride +
                           hk * a.c.head_stride;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) s += q[i] * value(a.c.k, at, lane + 64 * i);
#pragma unroll
        for (int w = 32; w > 0; w >>= 1) s += __shfl_xor(s, w);
        s *= a.scale_log2 * ks;
        const float mn = fmaxf(m, s), f = exp2f(m - mn), p = exp2f(s - mn);
        m = mn;
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = o[i] * f + p * value(a.c.v, at, lane + 64 * i);
    }
    if (lane == 0) {
        sm[wave] = m;
        sl[wave] = l;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) so[wave][lane + 64 * i] = o[i];
    __syncthreads();
    float top = sm[0], f[4], den = 0.f;
    for (int w = 1; w < 4; ++w) top = fmaxf(top, sm[w]);
    for (int w = 0; w < 4; ++w) {
        f[w] = exp2f(sm[w] - top);
        den += f[w] * sl[w];
    }
    const int64_t row = (int64_t)b * a.heads + h;
    for (int d = threadIdx.x; d < D; d += 256) {
        float x = 0.f;
        for (int w = 0; w < 4; ++w) x += f[w] * so[w][d];
        a.out[row * D + d] = f32_to_bf16(den == 0.f ? 0.f : x / den * vs);
    }
    if (a.lse && threadIdx.x == 0) a.lse[row] = den == 0.f ? -INFINITY : (top + log2f(den)) * 0.6931471805599453f;
}

size_t attn_decode_workspace(int, int, int, int, int, int) { return 0; }

hipError_t attn_decode(const AttnArgs& a, bool f8, hipStream_t st, StageTimer* tm) {
    return launch(tm, "attn_decode", f8 ? attn_decode_kernel<true> : attn_decode_kernel<false>, dim3(a.heads, a.B),
                  dim3(256), st, a);
}

}  // namespace lora
