// The next token of each request, from its logits and one random number:
//   w_i = exp((l_i - max l) / temperature), in the order of falling l (equal
//   logits by index): the first top_k, of these the shortest prefix with at
//   least top_p of their sum, of these the ones with w >= min_p; then the
//   first token, by index, at which the running sum of the kept w passes u
//   times their whole sum.
// Both prefixes are found without sorting, by descending through the digits
// of the logits' keys (their order as unsigned integers): a histogram of a
// digit says in which bin the border lies. Weights are 64-bit exponentials
// held as whole numbers of 2^-shift, so that sums do not depend on the order
// in which they are made: equal inputs give equal tokens.
#include "common.h"
#include "kernels.h"

namespace lora {

// Keys: 0 for NaN, otherwise rising with the value; -0 counts as 0.
constexpr uint32_t kKeyNone = 0x007fffffu;  // of -infinity: never drawn, like NaN
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);
    return v != v ? 0u : b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k >> 31 ? k ^ 0x80000000u : ~k); }

// 2^y for y <= 0 (0 below -1000): y = n + r, |r| <= 1/2, and the series of
// 2^r = e^(r ln 2) to the eleventh power (the next term is under 1e-14).
__device__ __forceinline__ double exp2_neg(double y) {
    constexpr double L = 0.693147180559945309417;
    constexpr double c2 = L * L / 2, c3 = c2 * L / 3, c4 = c3 * L / 4, c5 = c4 * L / 5, c6 = c5 * L / 6,
                     c7 = c6 * L / 7, c8 = c7 * L / 8, c9 = c8 * L / 9, c10 = c9 * L / 10, c11 = c10 * L / 11;
    const double n = __builtin_rint(y), r = y - n;
    double s = c11;
    s = __builtin_fma(s, r, c10);
    s = __builtin_fma(s, r, c9);
    s = __builtin_fma(s, r, c8);
    s = __builtin_fma(s, r, c7);
    s = __builtin_fma(s, r, c6);
    s = __builtin_fma(s, r, c5);
    s = __builtin_fma(s, r, c4);
    s = __builtin_fma(s, r, c3);
    s = __builtin_fma(s, r, c2);
    s = __builtin_fma(s, r, L);
    s = __builtin_fma(s, r, 1.0);
    return y < -1000.0 ? 0.0 : __builtin_ldexp(s, (int)n);
}

// The weights of one request: w of a key, and w as a whole number of 2^-shift.
struct Weights {
    float top;         // the largest logit
    double per;        // log2(e) / temperature
    int shift;
    __device__ __forceinline__ double of(uint32_t key) const {
        const float v = of_key(key);
        if (key <= kKeyNone) return 0.0;
        if (top == INFINITY) return v == top ? 1.0 : 0.0;
        return exp2_neg(((double)v - (double)top) * per);
    }
    // w + 2^(52 - shift) has 2^-shift as the last place of its mantissa
    __device__ __forceinline__ uint64_t whole(double w) const {
        const double c = __builtin_ldexp(1.0, 52 - shift);
        return __builtin_bit_cast(uint64_t, w + c) - __builtin_bit_cast(uint64_t, c);
    }
};

constexpr int kSampleThreads = 1024, kSampleWaves = kSampleThreads / 64;
constexpr int kDigitBins = 2048;
struct SampleLds {
    uint64_t mass[kDigitBins];
    uint32_t count[kDigitBins];
    uint64_t part[kSampleWaves];
    uint64_t found[4];
};

__device__ __forceinline__ uint64_t shfl64(uint64_t v, int src) {
    return (uint64_t)(uint32_t)__shfl((int)(uint32_t)v, src) |
           (uint64_t)(uint32_t)__shfl((int)(uint32_t)(v >> 32), src) << 32;
}
__device__ __forceinline__ uint64_t wave_scan(uint64_t v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint64_t p = shfl64(v, lane - o < 0 ? lane : lane - o);
        if (lane >= o) v += p;
    }
    return v;
}
// the sum of a value over the threads before this one; *all: over all of them
__device__ __forceinline__ uint64_t block_before(uint64_t v, SampleLds& L, uint64_t* all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t in = wave_scan(v, lane);
    __syncthreads();
    if (lane == 63) L.part[wave] = in;
    __syncthreads();
    uint64_t before = in - v, sum = 0;
    for (int w = 0; w < kSampleWaves; ++w) {
        if (w < wave) before += L.part[w];
        sum += L.part[w];
    }
    *all = sum;
    return before;
}

// A prefix of a request's tokens in falling order: every key above `key`, and
// of the equal ones those at an index up to `last`.
struct Prefix {
    uint32_t key;
    int last;
    __device__ __forceinline__ bool holds(uint32_t k, int i) const { return k > key || (k == key && i <= last); }
};

template <bool BF16>
__device__ __forceinline__ uint32_t key_at(const void* row, int i) {
    if constexpr (BF16)
        return key_of(bf16_to_f32(static_cast<const uint16_t*>(row)[i]));
    else
        return key_of(static_cast<const float*>(row)[i]);
}

// The index of the n-th (from 1) of the tokens with this key; V if there are
// no more than n of them... the last one then needs no border.
template <bool BF16>
__device__ __forceinline__ int nth_equal(const void* row, int V, uint32_t key, uint64_t n, SampleLds& L) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, per = (V + kSampleWaves - 1) / kSampleWaves;
    const int lo = min(wave * per, V), hi = min(lo + per, V);
    uint64_t mine = 0;
    for (int i0 = lo; i0 < hi; i0 += 64)
        mine += __popcll(__ballot(i0 + lane < hi && key_at<BF16>(row, i0 + lane) == key));
    uint64_t all;
    const uint64_t before = shfl64(block_before(lane == 0 ? mine : 0, L, &all), 0);
    if (threadIdx.x == 0) L.found[0] = V;
    __syncthreads();
    if (before < n && n <= before + mine) {
        uint64_t left = n - before;
        for (int i0 = lo; i0 < hi; i0 += 64) {
            const uint64_t m = __ballot(i0 + lane < hi && key_at<BF16>(row, i0 + lane) == key);
            const int c = __popcll(m);
            if (left <= (uint64_t)c) {
                if ((m >> lane) & 1 && __popcll(m & ((2ull << lane) - 1)) == (int)left) L.found[0] = i0 + lane;
                break;
            }
            left -= c;
        }
    }
    __syncthreads();
    return (int)L.found[0];
}

// The shortest prefix of `in` with at least `want` of its tokens (MASS false)
// or of its whole weights (MASS true); *sum: the weights of the prefix.
// `want` is at least 1 and at most the whole. Returns in.key 0 tokens short
// of nothing: where all are wanted the result is `in` itself.
template <bool BF16, bool MASS>
__device__ __forceinline__ Prefix descend(const void* row, int V, const Weights& W, Prefix in, uint64_t want,
                                          SampleLds& L) {
    const int tid = threadIdx.x;
    uint32_t prefix = 0;
    uint64_t above = 0;
    for (int level = 0; level < 3; ++level) {
        const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
        for (int i = tid; i < kDigitBins; i += kSampleThreads) L.mass[i] = 0;
        __syncthreads();
        for (int i = tid; i < V; i += kSampleThreads) {
            const uint32_t k = key_at<BF16>(row, i);
            if (k > kKeyNone && in.holds(k, i) && (level == 0 || k >> (shift + bits) == prefix))
                atomicAdd((unsigned long long*)&L.mass[(k >> shift) & ((1u << bits) - 1)],
                          (unsigned long long)(MASS ? W.whole(W.of(k)) : 1));
        }
        __syncthreads();
        // from the top bin down, two bins a thread
        const int b = kDigitBins - 2 - 2 * tid;
        const uint64_t hi = L.mass[b + 1], lo = L.mass[b];
        uint64_t all;
        const uint64_t before = above + block_before(hi + lo, L, &all);
        if (before < want && want <= before + hi + lo) {
            const bool first = want <= before + hi;
            L.found[0] = first ? b + 1 : b;
            L.found[1] = first ? before : before + hi;
        }
        __syncthreads();
        prefix = prefix << bits | (uint32_t)L.found[0];
        above = L.found[1];
        __syncthreads();
    }
    const uint64_t one = MASS ? W.whole(W.of(prefix)) : 1;
    const uint64_t n = (want - above + one - 1) / one;  // of the tokens with this key
    return Prefix{prefix, nth_equal<BF16>(row, V, prefix, n, L)};
}

// One workgroup a request.
template <bool BF16>
__global__ __launch_bounds__(kSampleThreads) void sample_kernel(SampleArgs a, int shift) {
    __shared__ SampleLds L;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, b = blockIdx.x, V = a.V;
    const void* row = static_cast<const char*>(a.logits) + (int64_t)b * a.stride * (BF16 ? 2 : 4);
    // the first token in the order: the largest key, of equal ones the lowest index
    uint64_t best = 0;
    for (int i = tid; i < V; i += kSampleThreads) {
        const uint64_t k = (uint64_t)key_at<BF16>(row, i) << 32 | (uint32_t)~i;
        best = k > best ? k : best;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const uint64_t p = shfl64(best, lane ^ o);
        best = p > best ? p : best;
    }
    if (lane == 0) L.part[wave] = best;
    __syncthreads();
    for (int w = 0; w < kSampleWaves; ++w) best = L.part[w] > best ? L.part[w] : best;
    __syncthreads();
    const uint32_t top = (uint32_t)(best >> 32);
    const int first = (int)~(uint32_t)best;
    const float t = a.temperature ? a.temperature[b] : 1.f;
    if (top <= kKeyNone || !(t > 0.f)) {
        if (tid == 0) {
            a.ids[b] = top <= kKeyNone ? -1 : first;
            a.probs[b] = top <= kKeyNone ? 0.f : 1.f;
        }
        return;
    }
    const Weights W{of_key(top), 1.4426950408889634 / (double)t, shift};
    Prefix kept{kKeyNone, -1};  // all but NaN and -infinity
    uint64_t all;
    const int k = a.top_k ? a.top_k[b] : 0;
    if (k > 0 && k < V) {
        uint64_t n = 0;
        for (int i = tid; i < V; i += kSampleThreads) n += key_at<BF16>(row, i) > kKeyNone;
        block_before(n, L, &all);
        if ((uint64_t)k < all) kept = descend<BF16, false>(row, V, W, kept, (uint64_t)k, L);
    }
    const float p = a.top_p ? a.top_p[b] : 1.f;
    if (p < 1.f) {
        uint64_t n = 0;
        for (int i = tid; i < V; i += kSampleThreads) {
            const uint32_t x = key_at<BF16>(row, i);
            if (kept.holds(x, i)) n += W.whole(W.of(x));
        }
        block_before(n, L, &all);
        const double want = __builtin_ceil((double)p * (double)all);
        const uint64_t w = want < 1.0 ? 1 : want >= (double)all ? all : (uint64_t)want;
        kept = descend<BF16, true>(row, V, W, kept, w, L);
    }
    const double least = a.min_p ? (double)a.min_p[b] : 0.0;
    // the draw: a wave sums its stretch of the vocabulary, the one with the border walks it again
    auto weight = [&](int i) -> uint64_t {
        const uint32_t x = key_at<BF16>(row, i);
        if (!kept.holds(x, i)) return 0;
        const double w = W.of(x);
        return w < least && i != first ? 0 : W.whole(w);
    };
    const int per = (V + kSampleWaves - 1) / kSampleWaves, lo = min(wave * per, V), hi = min(lo + per, V);
    uint64_t mine = 0;
    for (int i = lo + lane; i < hi; i += 64) mine += weight(i);
    const uint64_t before_lane = block_before(mine, L, &all);
    const uint64_t before = shfl64(before_lane, 0), whole = shfl64(before_lane + mine, 63) - before;
    const double u = fmin(fmax(a.u[b], 0.0), 1.0);
    // the first running sum above u * all: a whole number, so above its floor, and at most all
    const uint64_t pass = min((uint64_t)(u * (double)all), all - 1);
    if (before <= pass && pass < before + whole) {
        uint64_t run = before;
        for (int i0 = lo; i0 < hi; i0 += 64) {
            const uint64_t w = i0 + lane < hi ? weight(i0 + lane) : 0;
            const uint64_t in = run + wave_scan(w, lane);
            const uint64_t m = __ballot(in > pass);
            if (m) {
                if (lane == __builtin_ctzll(m)) {
                    a.ids[b] = i0 + lane;
                    a.probs[b] = (float)(W.of(key_at<BF16>(row, i0 + lane)) * __builtin_ldexp(1.0, shift) / (double)all);
                }
                break;
            }
            run = shfl64(in, 63);
        }
    }
}

size_t sample_workspace(int, int) { return 0; }

hipError_t sample(const SampleArgs& a, bool bf16, hipStream_t st, StageTimer* tm) {
    // V weights of at most 2^shift add up to less than 2^63
    int bits = 0;
    while ((int64_t)1 << bits < a.V) ++bits;
    return launch(tm, "sample", bf16 ? sample_kernel<true> : sample_kernel<false>, dim3(a.B), dim3(kSampleThreads), st,
                  a, min(46, 62 - bits));
}

}  // namespace lora
