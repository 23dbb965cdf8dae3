// The next token of each request, from its logits and one random number:
//   w_i = exp((l_i - max l) / temperature), in the order of falling l (equal
//   logits by index): the first top_k, of these the shortest prefix with at
//   least top_p of their sum, of these the ones with w >= min_p; then the
//   first token, by index, at which the running sum of the kept w passes u
//   times their whole sum.
//
// Nothing is sorted. A first kernel reads every logit once and leaves, for each
// tile of 512, the largest and (where the request draws from all of them, or
// by top_p alone) the sum of the weights. A second one, a workgroup a request,
// finds the border of each prefix: a histogram over the tokens that can lie
// above it says in which bin it is, the tokens of that bin are ranked. Tiles
// whose largest logit is below the border found so far are not read again, so
// that a few likely tokens cost a few tiles. The draw goes by the tiles' sums
// and then through one tile.
//
// Weights are 64-bit exponentials held as whole numbers of 2^-shift, so that
// sums do not depend on the order in which they are made: equal inputs give
// equal tokens.
#include <algorithm>

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

// Weights relative to a largest logit: w of a key, and w as a whole number of
// 2^-shift: w + 2^(52 - shift) has 2^-shift as the last place of its mantissa.
struct Weights {
    float top;
    double per;  // log2(e) / temperature
    double lift;  // 2^(52 - shift)
    __device__ __forceinline__ double of(uint32_t key) const {
        const float v = of_key(key);
        const double w = exp2_neg(((double)v - (double)top) * per);
        // among infinite logits all weigh the same; -infinity and NaN nothing
        return key <= kKeyNone ? 0.0 : top == INFINITY ? (v == top ? 1.0 : 0.0) : w;
    }
    __device__ __forceinline__ uint64_t whole(double w) const {
        return __builtin_bit_cast(uint64_t, w + lift) - __builtin_bit_cast(uint64_t, lift);
    }
};

__device__ __forceinline__ uint64_t shfl64(uint64_t v, int src) {
    return (uint64_t)(uint32_t)__shfl((int)(uint32_t)v, src) |
           (uint64_t)(uint32_t)__shfl((int)(uint32_t)(v >> 32), src) << 32;
}
__device__ __forceinline__ uint64_t shfl64_xor(uint64_t v, int o) {
    return (uint64_t)(uint32_t)__shfl_xor((int)(uint32_t)v, o) |
           (uint64_t)(uint32_t)__shfl_xor((int)(uint32_t)(v >> 32), o) << 32;
}
__device__ __forceinline__ uint64_t wave_total(uint64_t v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += shfl64_xor(v, o);
    return v;
}
__device__ __forceinline__ uint32_t wave_top(uint32_t v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
    return v;
}
__device__ __forceinline__ uint64_t wave_scan(uint64_t v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint64_t p = shfl64(v, lane - o < 0 ? lane : lane - o);
        if (lane >= o) v += p;
    }
    return v;
}

// ------------------------------------------------------------------- tiles --
// A request's logits in tiles of 512, 8 a lane, read in the 16-byte pieces that
// hold them: rows may begin anywhere, values before and behind the row count
// as NaN. Element e of a lane's piece i of tile t has index
// 512 t + 512 i / pieces + 16 / size lane + e - skip.
constexpr int kTile = 512;
template <bool BF16>
struct Row {
    static constexpr int E = BF16 ? 8 : 4, P = 8 / E;
    const u32x4* base;
    int skip, V, pieces, tiles;
    __device__ __forceinline__ Row(const SampleArgs& a, int b) : V(a.V) {
        const uintptr_t at = (uintptr_t)a.logits + (uintptr_t)(b * a.stride) * (BF16 ? 2 : 4);
        base = reinterpret_cast<const u32x4*>(at & ~(uintptr_t)15);
        skip = (int)(at & 15) / (BF16 ? 2 : 4);
        pieces = (skip + V + E - 1) / E;
        tiles = (pieces + 64 * P - 1) / (64 * P);
    }
    __device__ __forceinline__ void load(u32x4 (&x)[P], int t, bool on, int lane) const {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int at = (t * P + i) * 64 + lane;
            x[i] = *or_zero(on && at < pieces, base + at);
        }
    }
    __device__ __forceinline__ int index(int t, int j, int lane) const {
        return t * kTile + (j / E) * 64 * E + lane * E + j % E - skip;
    }
    __device__ __forceinline__ uint32_t key(const u32x4 (&x)[P], int t, int j, int lane) const {
        const int i = index(t, j, lane);
        float v;
        if constexpr (BF16) {
            const uint32_t w = x[0][j >> 1];
            v = __uint_as_float(j & 1 ? w & 0xffff0000u : w << 16);
        } else {
            v = __uint_as_float(x[j >> 2][j & 3]);
        }
        return (uint32_t)i < (uint32_t)V ? key_of(v) : 0u;
    }
};

// Tiles of a row at most, whatever its alignment; the workspace's layout.
__host__ __device__ inline int sample_tiles(int V) { return (V + 7 + kTile - 1) / kTile; }

// What a request asks for.
struct Ask {
    bool greedy;
    int k;        // 0: all
    float p;      // 1: all
    float least;  // 0: all
};
__device__ __forceinline__ Ask ask_of(const SampleArgs& a, int b, float* t) {
    Ask r;
    *t = a.temperature ? a.temperature[b] : 1.f;
    const int k = a.top_k ? a.top_k[b] : 0;
    const float p = a.top_p ? a.top_p[b] : 1.f, least = a.min_p ? a.min_p[b] : 0.f;
    r.greedy = !(*t > 0.f);
    r.k = k > 0 && k < a.V ? k : 0;
    r.p = p < 1.f ? p : 1.f;
    r.least = least > 0.f ? least : 0.f;
    return r;
}
// Whether the tiles' sums over all tokens are used: the draw is from all of
// them, or top_p is the first filter.
__device__ __forceinline__ bool needs_sums(const Ask& r) {
    return !r.greedy && r.k == 0 && (r.p < 1.f || r.least == 0.f);
}

// The largest key of each tile, and the sum of its weights relative to that. A
// wave takes 4 tiles.
template <bool BF16>
__global__ __launch_bounds__(256) void sample_tiles_kernel(SampleArgs a, double lift, uint32_t* __restrict__ tops,
                                                           uint64_t* __restrict__ sums) {
    const int lane = threadIdx.x & 63, b = blockIdx.y, nt = sample_tiles(a.V);
    const int t0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * 4;
    const Row<BF16> row(a, b);
    u32x4 x[4][Row<BF16>::P];
#pragma unroll
    for (int j = 0; j < 4; ++j) row.load(x[j], t0 + j, true, lane);
    float t;
    const Ask ask = ask_of(a, b, &t);
    const bool sum = needs_sums(ask);
    issue_fence();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (t0 + j >= nt) break;  // uniform
        uint32_t k[8], top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            k[e] = row.key(x[j], t0 + j, e, lane);
            top = max(top, k[e]);
        }
        top = wave_top(top);
        uint64_t s = 0;
        if (sum) {
            const Weights W{of_key(top), 1.4426950408889634 / (double)t, lift};
#pragma unroll
            for (int e = 0; e < 8; ++e) s += W.whole(W.of(k[e]));
            s = wave_total(s);
        }
        if (lane == 0) {
            tops[(int64_t)b * nt + t0 + j] = top;
            sums[(int64_t)b * nt + t0 + j] = s;
        }
    }
}

// ------------------------------------------------------------------ borders --
constexpr int kSampleThreads = 1024, kSampleWaves = kSampleThreads / 64;
constexpr int kBins = 2048, kList = kSampleThreads;
struct SampleLds {
    uint64_t bin[kBins];
    uint64_t list[kList];   // tokens of the border's bin: key, then ~index
    uint64_t part[kSampleWaves];
    uint64_t found[4];
    uint32_t count, low, high;
};
__device__ __forceinline__ uint64_t token(uint32_t key, int i) { return (uint64_t)key << 32 | (uint32_t)~i; }

// the sum of a value over the threads before this one; *all: over all of them
__device__ __forceinline__ uint64_t block_before(uint64_t v, SampleLds& L, uint64_t* all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t in = wave_scan(v, lane);
    __syncthreads();
    if (lane == 63) L.part[wave] = in;
    __syncthreads();
    uint64_t before = in - v, sum = 0;
#pragma unroll
    for (int w = 0; w < kSampleWaves; ++w) {
        const uint64_t x = L.part[w];
        if (w < wave) before += x;
        sum += x;
    }
    *all = sum;
    return before;
}

// A prefix of a request's tokens in falling order: all up to token `last`
// (tokens compare as their order: a larger key, then a lower index).
typedef uint64_t Prefix;
__device__ __forceinline__ bool holds(Prefix p, uint64_t t) { return t >= p; }
constexpr Prefix kAll = (uint64_t)(kKeyNone + 1) << 32;  // every token but NaN and -infinity

// Whole rows, tile by tile: f(tile, logits) for the tiles that on(tile) says, 4
// of a wave's in flight.
template <bool BF16, class On, class F>
__device__ __forceinline__ void each_tile(const Row<BF16>& row, On on, F f) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int t0 = wave * 4; t0 < row.tiles; t0 += kSampleWaves * 4) {
        u32x4 x[4][Row<BF16>::P];
        uint32_t is = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (t0 + j < row.tiles && __builtin_amdgcn_readfirstlane(on(t0 + j))) is |= 1u << j;
        if (!is) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) row.load(x[j], t0 + j, (is >> j) & 1, lane);
        issue_fence();
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if ((is >> j) & 1) f(t0 + j, x[j]);
    }
}

// The bin at which the sum of the bins from the first on reaches `want`
// (found[0], kBins if none), and the sum before it (found[1]). *all: the whole.
__device__ __forceinline__ void find_bin(uint64_t above, uint64_t want, SampleLds& L, uint64_t* all) {
    const int tid = threadIdx.x;
    const uint64_t x = L.bin[2 * tid], y = L.bin[2 * tid + 1];
    const uint64_t before = above + block_before(x + y, L, all);
    if (tid == 0) L.found[0] = kBins;
    __syncthreads();
    if (before < want && want <= before + x + y) {
        const bool first = want <= before + x;
        L.found[0] = first ? 2 * tid : 2 * tid + 1;
        L.found[1] = first ? before : before + x;
    }
    __syncthreads();
}
__device__ __forceinline__ void clear_bins(SampleLds& L) {
    L.bin[threadIdx.x] = 0;
    L.bin[threadIdx.x + kSampleThreads] = 0;
    __syncthreads();
}

// The n-th (from 1) of the tokens with this key that `in` holds; there are at
// least n.
template <bool BF16>
__device__ __forceinline__ Prefix nth_equal(const Row<BF16>& row, const uint32_t* tops, uint32_t key, uint64_t n,
                                            SampleLds& L) {
    const int lane = threadIdx.x & 63;
    // tokens of each stretch of tiles, a bin each; then the tile by tile and lane by lane walk of one wave
    int sh = 0;
    while (((row.tiles - 1) >> sh) >= kBins) ++sh;
    clear_bins(L);
    auto same = [&](int t) { return tops[t] >= key; };
    each_tile(row, same, [&](int t, const u32x4(&x)[Row<BF16>::P]) {
        int c = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) c += __popcll(__ballot(row.key(x, t, e, lane) == key));
        if (lane == 0 && c) atomicAdd((unsigned long long*)&L.bin[t >> sh], (unsigned long long)c);
    });
    __syncthreads();
    uint64_t all;
    find_bin(0, n, L, &all);
    const int t0 = (int)L.found[0] << sh;
    uint64_t left = n - L.found[1];
    if (threadIdx.x < 64)
        for (int t = t0; t < min(t0 + (1 << sh), row.tiles); ++t) {
            u32x4 x[Row<BF16>::P];
            row.load(x, t, true, lane);
            uint64_t done = 0;
#pragma unroll
            for (int i = 0; i < Row<BF16>::P; ++i) {
                uint32_t c = 0;
#pragma unroll
                for (int e = 0; e < Row<BF16>::E; ++e) c += row.key(x, t, i * Row<BF16>::E + e, lane) == key;
                const uint64_t in = wave_scan(c, lane);
                if (left > done + in - c && left <= done + in) {
                    uint64_t at = done + in - c;
#pragma unroll
                    for (int e = 0; e < Row<BF16>::E; ++e) {
                        const int j = i * Row<BF16>::E + e;
                        if (row.key(x, t, j, lane) == key && ++at == left) L.found[2] = token(key, row.index(t, j, lane));
                    }
                }
                done += shfl64(in, 63);
            }
            if (left <= done) break;  // uniform
            left -= done;
        }
    __syncthreads();
    return L.found[2];
}

// Where a token falls: bins of equal width below the largest logit, monotone
// in the key (each step of the arithmetic is).
struct Scale {
    float top, per;
    __device__ __forceinline__ int bin(uint32_t key) const {
        return (int)fminf((top - of_key(key)) * per, (float)(kBins - 1));
    }
};

// The shortest prefix of `in` with at least `want` of its tokens (MASS false)
// or of its whole weights (MASS true); in where even that has less. `last` is
// a bin that no border lies behind; tokens behind it are not looked at.
template <bool BF16, bool MASS>
__device__ __forceinline__ Prefix border(const Row<BF16>& row, const uint32_t* tops, const Weights& W, Prefix in,
                                         uint64_t want, double part, const Scale& S, int last, SampleLds& L) {
    const int tid = threadIdx.x, lane = tid & 63;
    const uint32_t floor_key = (uint32_t)(in >> 32);
    auto weight = [&](uint32_t k) -> uint64_t { return MASS ? W.whole(W.of(k)) : 1; };
    clear_bins(L);
    each_tile(
        row, [&](int t) { return tops[t] >= floor_key && S.bin(tops[t]) <= last; },
        [&](int t, const u32x4(&x)[Row<BF16>::P]) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t k = row.key(x, t, e, lane);
                if (holds(in, token(k, row.index(t, e, lane)))) {
                    const int n = S.bin(k);
                    if (n <= last) atomicAdd((unsigned long long*)&L.bin[n], (unsigned long long)weight(k));
                }
            }
        });
    __syncthreads();
    uint64_t all;
    if (MASS && want == 0) {  // the share of what the bins hold
        block_before(L.bin[2 * tid] + L.bin[2 * tid + 1], L, &all);
        const double x = __builtin_ceil(part * (double)all);
        want = x < 1.0 ? 1 : x >= (double)all ? all : (uint64_t)x;
    }
    find_bin(0, want, L, &all);
    const int b = (int)L.found[0];
    if (b == kBins) return in;
    uint64_t above = L.found[1];
    // the tokens of the border's bin
    if (tid == 0) {
        L.count = 0;
        L.low = ~0u;
        L.high = 0;
    }
    __syncthreads();
    each_tile(
        row, [&](int t) { return tops[t] >= floor_key && S.bin(tops[t]) <= b; },
        [&](int t, const u32x4(&x)[Row<BF16>::P]) {
            uint32_t low = ~0u, high = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t k = row.key(x, t, e, lane);
                const uint64_t tk = token(k, row.index(t, e, lane));
                if (holds(in, tk) && S.bin(k) == b) {
                    const uint32_t at = atomicAdd(&L.count, 1u);
                    if (at < kList) L.list[at] = tk;
                    low = min(low, k);
                    high = max(high, k);
                }
            }
            if (high) {
                atomicMin(&L.low, low);
                atomicMax(&L.high, high);
            }
        });
    __syncthreads();
    const int n = (int)L.count;
    uint32_t low = L.low, high = L.high;
    if (low != high && n <= kList) {
        // ranks: what of the bin comes before each token
        const uint64_t mine = tid < n ? L.list[tid] : 0;
        const uint64_t w = tid < n ? weight((uint32_t)(mine >> 32)) : 0;
        __syncthreads();
        if (MASS) L.bin[tid] = w;
        __syncthreads();
        if (tid < n) {
            uint64_t before = above;
            for (int j = 0; j < n; ++j)
                if (L.list[j] > mine) before += MASS ? L.bin[j] : 1;
            if (before < want && want <= before + w) L.found[2] = mine;
        }
        __syncthreads();
        return L.found[2];
    }
    while (low != high) {  // more tokens than the list holds: by the digits of their keys
        int sh = 0;
        while ((high - low) >> sh >= kBins) ++sh;
        clear_bins(L);
        each_tile(
            row, [&](int t) { return tops[t] >= low; },
            [&](int t, const u32x4(&x)[Row<BF16>::P]) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t k = row.key(x, t, e, lane);
                    if (k >= low && k <= high && holds(in, token(k, row.index(t, e, lane))))
                        atomicAdd((unsigned long long*)&L.bin[(high - k) >> sh], (unsigned long long)weight(k));
                }
            });
        __syncthreads();
        find_bin(above, want, L, &all);
        const uint32_t at = (uint32_t)L.found[0];
        above = L.found[1];
        const uint32_t top = high - (at << sh);
        low = max(low, top - ((1u << sh) - 1));
        high = top;
        __syncthreads();
    }
    const uint64_t one = weight(high);
    return nth_equal(row, tops, high, (want - above + one - 1) / one, L);
}

// One workgroup a request, over what the first kernel left.
template <bool BF16>
__global__ __launch_bounds__(kSampleThreads) void sample_kernel(SampleArgs a, double lift,
                                                                const uint32_t* __restrict__ all_tops,
                                                                const uint64_t* __restrict__ all_sums) {
    extern __shared__ uint64_t tile_sum[];  // [tiles], then the largest keys
    __shared__ SampleLds L;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, b = blockIdx.x, nt = sample_tiles(a.V);
    uint32_t* tops = reinterpret_cast<uint32_t*>(tile_sum + nt);
    const Row<BF16> row(a, b);
    float t;
    const Ask ask = ask_of(a, b, &t);
    // the largest key, and the first tile that has it
    uint64_t best = 0;
    uint32_t least_top = ~0u;  // of the tiles with a token that can be drawn
    int live = 0;              // their number
    for (int i = tid; i < nt; i += kSampleThreads) {
        const uint32_t k = all_tops[(int64_t)b * nt + i];
        tops[i] = k;
        best = max(best, token(k, i));
        if (k > kKeyNone) {
            least_top = min(least_top, k);
            ++live;
        }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        best = max(best, shfl64_xor(best, o));
        least_top = min(least_top, (uint32_t)__shfl_xor((int)least_top, o));
        live += __shfl_xor(live, o);
    }
    if (lane == 0) {
        L.part[wave] = best;
        L.list[wave] = (uint64_t)least_top << 32 | (uint32_t)live;
    }
    __syncthreads();
    live = 0;
    least_top = ~0u;
    for (int w = 0; w < kSampleWaves; ++w) {
        best = max(best, L.part[w]);
        least_top = min(least_top, (uint32_t)(L.list[w] >> 32));
        live += (int)(uint32_t)L.list[w];
    }
    const uint32_t top = (uint32_t)(best >> 32);
    if (top <= kKeyNone) {
        if (tid == 0) {
            a.ids[b] = -1;
            a.probs[b] = 0.f;
        }
        return;
    }
    // the first token in the order
    if (tid < 64) {
        const int at = (int)~(uint32_t)best;
        u32x4 x[Row<BF16>::P];
        row.load(x, at, true, lane);
        uint64_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, token(row.key(x, at, e, lane), row.index(at, e, lane)));
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) m = max(m, shfl64_xor(m, o));
        if (lane == 0) L.found[3] = m;
    }
    __syncthreads();
    const uint64_t first = L.found[3];
    if (ask.greedy) {
        if (tid == 0) {
            a.ids[b] = (int)~(uint32_t)first;
            a.probs[b] = 1.f;
        }
        return;
    }
    const Weights W{of_key(top), 1.4426950408889634 / (double)t, lift};
    Prefix kept = kAll;
    uint64_t all;
    bool filtered = false;
    if (ask.k) {
        // at least k tokens lie at or above the k-th largest tile's top: bins down
        // to the lowest one hold the border then, otherwise twice as far
        const bool sure = ask.k <= live;
        const float reach = (W.top - of_key(least_top)) * (sure ? 1.f : 2.f);
        const Scale S{W.top, W.top == INFINITY ? 0.f : fminf((kBins - 2) / fmaxf(reach, 1e-30f), 1e30f)};
        int last = kBins - 1;
        if (sure) {
            clear_bins(L);
            for (int i = tid; i < nt; i += kSampleThreads)
                if (tops[i] > kKeyNone) atomicAdd((unsigned long long*)&L.bin[S.bin(tops[i])], 1ull);
            __syncthreads();
            find_bin(0, (uint64_t)ask.k, L, &all);
            last = min((int)L.found[0], kBins - 1);
            __syncthreads();
        }
        kept = border<BF16, false>(row, tops, W, kept, (uint64_t)ask.k, 0.0, S, last, L);
        filtered = true;
    }
    if (ask.p < 1.f) {
        // the tokens behind the border weigh at most (1 - p) of the whole, which is
        // at least 1, and are fewer than V: the first of them weighs at least ...
        const double reach = log2((double)a.V / (1.0 - (double)fmaxf(ask.p, 0.f))) + 1.0;
        const double per = W.per * (kBins - 2) / reach;
        const Scale S{W.top, W.top == INFINITY ? 0.f : (float)fmin(per, 1e30)};
        uint64_t want = 0;
        int last = kBins - 1;
        if (!filtered) {
            // where the largest tokens of the tiles alone make up the share, the border is among them
            clear_bins(L);
            uint64_t sum = 0;
            for (int i = tid; i < nt; i += kSampleThreads) {
                const double f = W.of(tops[i]);
                sum += (uint64_t)((double)all_sums[(int64_t)b * nt + i] * f);
                if (tops[i] > kKeyNone)
                    atomicAdd((unsigned long long*)&L.bin[S.bin(tops[i])], (unsigned long long)W.whole(f));
            }
            block_before(sum, L, &all);
            const double x = __builtin_ceil((double)ask.p * (double)all);
            const uint64_t share = x < 1.0 ? 1 : (uint64_t)x;
            uint64_t of_tops;
            find_bin(0, share, L, &of_tops);
            if ((int)L.found[0] < kBins) {
                last = (int)L.found[0];
                want = share;
            }
            __syncthreads();
        }
        kept = border<BF16, true>(row, tops, W, kept, want, (double)ask.p, S, last, L);
        filtered = true;
    }
    // the sums of the kept tokens, tile by tile
    const double least = (double)ask.least;
    auto weight = [&](uint32_t k, int i) -> uint64_t {
        const uint64_t tk = token(k, i);
        if (!holds(kept, tk)) return 0;
        const double w = W.of(k);
        return w < least && tk != first ? 0 : W.whole(w);
    };
    const bool whole = !filtered && ask.least == 0.f;
    const uint32_t floor_key = (uint32_t)(kept >> 32);
    __syncthreads();
    if (whole) {
        for (int i = tid; i < nt; i += kSampleThreads)
            tile_sum[i] = (uint64_t)((double)all_sums[(int64_t)b * nt + i] * W.of(tops[i]));
    } else {
        for (int i = tid; i < nt; i += kSampleThreads) tile_sum[i] = 0;
        __syncthreads();
        each_tile(
            row, [&](int i) { return tops[i] >= floor_key && (W.of(tops[i]) >= least || tops[i] == top); },
            [&](int i, const u32x4(&x)[Row<BF16>::P]) {
                uint64_t s = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) s += weight(row.key(x, i, e, lane), row.index(i, e, lane));
                s = wave_total(s);
                if (lane == 0) tile_sum[i] = s;
            });
    }
    __syncthreads();
    // the tile with the border of u: a stretch of tiles a thread
    const int per = (nt + kSampleThreads - 1) / kSampleThreads, t0 = min(tid * per, nt), t1 = min(t0 + per, nt);
    uint64_t mine = 0;
    for (int i = t0; i < t1; ++i) mine += tile_sum[i];
    uint64_t before = block_before(mine, L, &all);
    const double u = fmin(fmax(a.u[b], 0.0), 1.0);
    // the first running sum above u * all: a whole number, so above its floor, and at most all
    const uint64_t pass = min((uint64_t)(u * (double)all), all - 1);
    if (before <= pass && pass < before + mine) {
        int i = t0;
        for (; before + tile_sum[i] <= pass; ++i) before += tile_sum[i];
        L.found[0] = i;
        L.found[1] = pass - before;
    }
    __syncthreads();
    if (tid >= 64) return;
    const int at = (int)L.found[0];
    const uint64_t left = L.found[1];
    u32x4 x[Row<BF16>::P];
    row.load(x, at, true, lane);
    // sums of all tokens are relative to the tile's own largest: f takes them to
    // the row's as tile_sum has it, a step that keeps their order
    const double f = whole ? W.of(tops[at]) : 1.0;
    const Weights T{of_key(tops[at]), W.per, lift};
    uint64_t run = 0;
#pragma unroll
    for (int i = 0; i < Row<BF16>::P; ++i) {
        uint64_t w[Row<BF16>::E], s = 0;
#pragma unroll
        for (int e = 0; e < Row<BF16>::E; ++e) {
            const int j = i * Row<BF16>::E + e;
            const uint32_t k = row.key(x, at, j, lane);
            w[e] = whole ? T.whole(T.of(k)) : weight(k, row.index(at, j, lane));
            s += w[e];
        }
        const uint64_t in = run + wave_scan(s, lane);
        auto passes = [&](uint64_t v) { return (whole ? (uint64_t)((double)v * f) : v) > left; };
        const uint64_t m = __ballot(passes(in));
        if (m) {
            if (lane == __builtin_ctzll(m)) {
                uint64_t v = in - s;
                int e = 0;
#pragma unroll
                for (int n = 0; n < Row<BF16>::E; ++n) {
                    if (!passes(v + w[n]) && e == n) {
                        v += w[n];
                        e = n + 1;
                    }
                }
#pragma unroll
                for (int n = 0; n < Row<BF16>::E; ++n)
                    if (n == e) {
                        const int j = i * Row<BF16>::E + n;
                        a.ids[b] = row.index(at, j, lane);
                        a.probs[b] = (float)(W.of(row.key(x, at, j, lane)) * (4503599627370496.0 / lift) / (double)all);
                    }
            }
            return;
        }
        run = shfl64(in, 63);
    }
}

// -------------------------------------------------------------------- host --
static size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

size_t sample_workspace(int B, int V) {
    const size_t n = (size_t)B * sample_tiles(V);
    return align256(n * sizeof(uint64_t)) + align256(n * sizeof(uint32_t));
}

hipError_t sample(const SampleArgs& a, bool bf16, hipStream_t st, StageTimer* tm) {
    // V weights of at most 2^shift add up to less than 2^63
    int bits = 0;
    while ((int64_t)1 << bits < a.V) ++bits;
    const double lift = (double)((int64_t)1 << (52 - std::min(46, 62 - bits)));
    const int nt = sample_tiles(a.V);
    uint64_t* sums = static_cast<uint64_t*>(a.workspace);
    uint32_t* tops = reinterpret_cast<uint32_t*>(static_cast<char*>(a.workspace) + align256((size_t)a.B * nt * 8));
    hipError_t e = launch(tm, "sample_tiles", bf16 ? sample_tiles_kernel<true> : sample_tiles_kernel<false>,
                          dim3((nt + 15) / 16, a.B), dim3(256), st, a, lift, tops, sums);
    if (e != hipSuccess) return e;
    return launch_shm(tm, "sample", bf16 ? sample_kernel<true> : sample_kernel<false>, dim3(a.B), dim3(kSampleThreads),
                      nt * 12, st, a, lift, (const uint32_t*)tops, (const uint64_t*)sums);
}

}  // namespace lora
