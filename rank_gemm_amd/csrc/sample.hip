// The next token of each request, from its logits and one random number:
//   w_i = exp((l_i - max l) / temperature), in the order of falling l (equal
//   logits by index): the first top_k, of these the shortest prefix with at
//   least top_p of their sum, of these the ones with w >= min_p; then the
//   first token, by index, at which the running sum of the kept w passes u
//   times their whole sum.
//
// No long row is sorted. The border of a prefix is found by a histogram of the
// tokens over bins of equal width below the largest logit, and by ranking the
// tokens of the one bin that holds it; the draw goes by sums over tiles of 512
// tokens and then through one tile. Short rows are a workgroup's each from end
// to end, in one launch. Every pass over others is spread over the chip, tile by
// tile:
//   tops     the largest logit of each tile
//   bins     the histogram (top_p, or a top_k past the number of tiles); rows
//            without those filters: the tiles' sums at once
//   gather   the tokens of the border's bin; where there are few down to there
//            for sure, all of them
//   border   a workgroup a request: ranks that bin; or, where all tokens that
//            can be kept are at hand, sorts them and draws. A top_k up to the
//            number of tiles is done here from first to last: its tokens are in
//            tiles whose largest logit is among the k largest, few of which are
//            read
//   sums     the tiles' sums of the kept tokens
//   draw     a workgroup a request
// Bound by that chain: of one row of 131072 with top_k 50 and top_p 0.9 (20 us)
// the border's workgroup takes 10 and each of the others, busy or not, 1.3 to
// 3.2; the one launch over 32000 takes 14. Of 256 rows of 131072 fp32 (134 MB) with
// filters of every kind (97 us) tops reads at 6.5 TB/s (20 us), and bins takes 30:
// half of the rows pass over all of their tokens there, which is 38 vector
// instructions a weighed token (20 of them the 64-bit exponential's), and vector
// instructions issue in 71 % of the cycles that a CU has a wave, which are 73 %;
// conflicts of the histogram's adds are 7 %. With no filter bins is 48 of 74, and
// they issue in 82 % of the cycles.
//
// Weights are 64-bit exponentials held as whole numbers of 2^-shift, so that
// sums do not depend on the order in which they are made: equal inputs give
// equal tokens.
#include <algorithm>

#include "common.h"
#include "kernels.h"

namespace lora {

// ------------------------------------------------------------------ weights --
// a b + c with c in scalar registers (the compiler would copy every c to vector
// registers first).
__device__ __forceinline__ double fma_s(double a, double b, double c) {
    double d;
    asm("v_fma_f64 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "s"(c));
    return d;
}
// 2^y of N numbers -1000 <= y <= 0: y = n + r, |r| <= 1/2, and the series of 2^r
// = e^(r ln 2) to the eleventh power (the next term is under 1e-14). n is the
// low word of y + 1.5 2^52, and goes into the exponent as it is.
template <int N>
__device__ __forceinline__ void exp2_neg(double (&y)[N]) {
    constexpr double L = 0.693147180559945309417;
    constexpr double c2 = L * L / 2, c3 = c2 * L / 3, c4 = c3 * L / 4, c5 = c4 * L / 5, c6 = c5 * L / 6,
                     c7 = c6 * L / 7, c8 = c7 * L / 8, c9 = c8 * L / 9, c10 = c9 * L / 10, c11 = c10 * L / 11;
    constexpr double c[11] = {c10, c9, c8, c7, c6, c5, c4, c3, c2, L, 1.0};
    constexpr double kRound = 6755399441055744.0;
    double r[N];
    uint32_t n[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const double m = y[i] + kRound;
        n[i] = __builtin_bit_cast(u32x2, m)[0];
        r[i] = y[i] - (m - kRound);
        y[i] = c11;
    }
#pragma unroll
    for (int k = 0; k < 11; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = fma_s(y[i], r[i], c[k]);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const u32x2 b = __builtin_bit_cast(u32x2, y[i]);
        y[i] = __builtin_bit_cast(double, u32x2{b[0], b[1] + (n[i] << 20)});
    }
}

// The weights of a request: w of a logit (at least 2^-1000, also of -infinity
// and NaN), and w as a whole number of 2^-shift, 0 for those: w + 2^(52 - shift)
// has 2^-shift as the last place of its mantissa.
struct Weights {
    float top;    // the largest logit
    double per;   // log2(e) / temperature
    double lift;  // 2^(52 - shift)
    template <int N>
    __device__ __forceinline__ void of(double (&w)[N], const float (&v)[N]) const {
        if (top == INFINITY) {  // uniform; among infinite logits all weigh the same
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = v[i] == top ? 1.0 : 0.0;
            return;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = __builtin_fmax(((double)v[i] - (double)top) * per, -1000.0);
        exp2_neg<N>(w);
    }
    __device__ __forceinline__ double of(float v) const {
        double w[1];
        const float x[1] = {v};
        of<1>(w, x);
        return w[0];
    }
    __device__ __forceinline__ uint64_t whole(double w) const {
        return __builtin_bit_cast(uint64_t, w + lift) - __builtin_bit_cast(uint64_t, lift);
    }
};

// A token as a number that rises with its place in the order: its logit's bits
// made to rise with the value (-0 counts as 0), then its index inverted.
__device__ __forceinline__ uint64_t token(float v, int i) {
    const uint32_t b = __float_as_uint(v + 0.f);
    return (uint64_t)(b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u)) << 32 | (uint32_t)~i;
}
__device__ __forceinline__ float token_logit(uint64_t t) {
    const uint32_t k = (uint32_t)(t >> 32);
    return __uint_as_float(k >> 31 ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ int token_index(uint64_t t) { return (int)~(uint32_t)t; }

// A prefix of a request's tokens in the order: all logits above v, and of the
// equal ones those at an index up to `last`. NaN is in none.
struct Prefix {
    float v;
    int last;
    __device__ __forceinline__ bool holds(float x, int i) const { return x > v || (x == v && i <= last); }
};
__device__ __forceinline__ Prefix up_to(uint64_t t) { return Prefix{token_logit(t), token_index(t)}; }

__device__ __forceinline__ uint64_t shfl64(uint64_t v, int src) {
    return (uint64_t)(uint32_t)__shfl((int)(uint32_t)v, src) |
           (uint64_t)(uint32_t)__shfl((int)(uint32_t)(v >> 32), src) << 32;
}
// f over all lanes of a wave (f of two values, in any order).
template <class T, class F>
__device__ __forceinline__ T wave_all(T v, F f) {
    v = f(v, lane_xor<32>(v));
    v = f(v, lane_xor<16>(v));
    v = f(v, lane_xor<8>(v));
    v = f(v, lane_xor<4>(v));
    v = f(v, lane_xor<2>(v));
    return f(v, lane_xor<1>(v));
}
__device__ __forceinline__ float wave_max(float v) {
    return wave_all(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float wave_min(float v) {
    return wave_all(v, [](float a, float b) { return fminf(a, b); });
}
__device__ __forceinline__ uint64_t wave_total(uint64_t v) {
    return wave_all(v, [](uint64_t a, uint64_t b) { return a + b; });
}
// v of the lane a DPP move names, 0 where it names none or the row is not in ROWS.
template <int MOVE, int ROWS>
__device__ __forceinline__ uint64_t dpp64(uint64_t v) {
    const u32x2 x = __builtin_bit_cast(u32x2, v);
    return __builtin_bit_cast(uint64_t, u32x2{(uint32_t)__builtin_amdgcn_update_dpp(0, (int)x[0], MOVE, ROWS, 0xf, false),
                                              (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x[1], MOVE, ROWS, 0xf, false)});
}
// The sum over the lanes up to this one: within rows of 16, then with the last
// lane of the row before, then with lane 31.
__device__ __forceinline__ uint64_t wave_scan(uint64_t v) {
    v += dpp64<0x111, 0xf>(v);
    v += dpp64<0x112, 0xf>(v);
    v += dpp64<0x114, 0xf>(v);
    v += dpp64<0x118, 0xf>(v);
    v += dpp64<0x142, 0xa>(v);
    return v + dpp64<0x143, 0xc>(v);
}

// -------------------------------------------------------------------- rows --
// A request's logits in tiles of 512, 8 a lane, read in the 16-byte pieces that
// hold them: rows may begin anywhere, values before and behind the row count
// as NaN. Value j of a lane of tile t has index(t, j, lane).
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
    __device__ __forceinline__ void values(float (&v)[8], const u32x4 (&x)[P], int t, int lane) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (BF16) {
                const uint32_t w = x[0][j >> 1];
                v[j] = __uint_as_float(j & 1 ? w & 0xffff0000u : w << 16);
            } else {
                v[j] = __uint_as_float(x[j >> 2][j & 3]);
            }
        }
        if (t == 0 || t == tiles - 1) {  // uniform
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if ((uint32_t)index(t, j, lane) >= (uint32_t)V) v[j] = __builtin_nanf("");
        }
    }
};

// Tiles of a row at most, whatever its alignment.
__host__ __device__ inline int sample_tiles(int V) { return (V + 7 + kTile - 1) / kTile; }

constexpr int kBins = 2048;
constexpr int kList = 2048;  // tokens of a border's bin that are ranked, or of a list that is sorted

// What the kernels leave for one another, in the workspace.
struct RowState {
    uint32_t count;  // tokens gathered
    int drawn;       // the border kernel did it
    Prefix kept;
    int way, live;  // what the bins kernel found (Ask)
    float top, under;
};
struct SampleSpace {
    SampleArgs a;
    double lift;
    int nt, per_wg;    // tiles of a row, of a workgroup
    uint64_t* bins;    // [B][kBins]
    uint64_t* sums;    // [B][nt]
    uint64_t* list;    // [B][kList]
    float* tops;       // [B][nt]
    RowState* state;   // [B]
};

// What a request asks for, and the way it takes.
enum Way { kDone, kSums, kFew, kCount, kMass };
struct Ask {
    float t, p, least;  // p 1, least 0: all
    int k;              // 0: all
    Way way;
    float top;   // the largest logit, the least of the tiles' largest
    float under;
    int live;    // tiles with a token that can be drawn
};
template <int NT>
struct BlockLds {
    uint64_t part[NT / 64];
    float part_top[NT / 64], part_under[NT / 64];
    int part_live[NT / 64];
    uint64_t found[4];
    uint32_t count;
};
__device__ __forceinline__ Ask asked(const SampleArgs& a, int b) {
    Ask r;
    r.t = a.temperature ? a.temperature[b] : 1.f;
    const int k = a.top_k ? a.top_k[b] : 0;
    const float p = a.top_p ? a.top_p[b] : 1.f, least = a.min_p ? a.min_p[b] : 0.f;
    r.k = k > 0 && k < a.V ? k : 0;
    r.p = p < 1.f ? fmaxf(p, 0.f) : 1.f;
    r.least = least > 0.f ? least : 0.f;
    return r;
}
// From the tiles' largest logits, by a workgroup.
template <int NT>
__device__ __forceinline__ Ask find_way(const SampleSpace& s, int b, const float* tops, BlockLds<NT>& L) {
    Ask r = asked(s.a, b);
    float top = -INFINITY, under = INFINITY;
    int live = 0;
    for (int i = threadIdx.x; i < s.nt; i += NT) {
        const float v = tops[i];
        if (v > -INFINITY) {
            top = fmaxf(top, v);
            under = fminf(under, v);
            ++live;
        }
    }
    top = wave_max(top);
    under = wave_min(under);
    live = (int)wave_all((uint32_t)live, [](uint32_t a, uint32_t b) { return a + b; });
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
        L.part_top[wave] = top;
        L.part_under[wave] = under;
        L.part_live[wave] = live;
    }
    __syncthreads();
    r.top = top, r.under = under, r.live = 0;
    for (int w = 0; w < NT / 64; ++w) {
        r.top = fmaxf(r.top, L.part_top[w]);
        r.under = fminf(r.under, L.part_under[w]);
        r.live += L.part_live[w];
    }
    r.top = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(r.top)));
    r.way = !(r.t > 0.f) || r.top == -INFINITY ? kDone
            : r.k                              ? (r.k <= r.live ? kFew : kCount)
            : r.p < 1.f                        ? kMass
                                               : kSums;
    return r;
}
// As the bins kernel left it.
__device__ __forceinline__ Ask known_way(const SampleSpace& s, int b) {
    Ask r = asked(s.a, b);
    const RowState& st = s.state[b];
    r.way = (Way)st.way, r.live = st.live, r.top = st.top, r.under = st.under;
    return r;
}
__device__ __forceinline__ Weights weights_of(const SampleSpace& s, const Ask& r) {
    return Weights{r.top, 1.4426950408889634 / (double)r.t, s.lift};
}

// Bins of equal width below the largest logit, monotone in it (each step of
// the arithmetic is); what lies past the last, and NaN, is in the last.
struct Scale {
    float top, per;
    __device__ __forceinline__ int bin(float v) const { return (int)fminf((top - v) * per, (float)(kBins - 1)); }
};
// Of top_k: down to the lowest tile's largest logit, which the border is not
// below where there are at least k tiles; otherwise twice as far, or 24 (logits
// of a vocabulary spread over some tens; a border past the last bin is found
// too, by one workgroup: 5 rows of 3001, top_k 50, 66 us where reach falls short
// of it, 25 us where not).
__device__ __forceinline__ Scale scale_of_count(const Ask& r) {
    const float reach = r.k <= r.live ? r.top - r.under : fmaxf(2.f * (r.top - r.under), 24.f);
    return Scale{r.top, r.top == INFINITY ? 0.f : fminf((kBins - 2) / fmaxf(reach, 1e-30f), 1e30f)};
}
// Of top_p: the tokens behind the border weigh at least 1 - p of the whole,
// which is at least 1, with the border's own; fewer than V of them, so that one
// weighs at least (1 - p) / V.
__device__ __forceinline__ Scale scale_of_mass(const Ask& r, const Weights& W, int V) {
    const float reach = log2f((float)V / (1.f - r.p)) + 1.f;
    return Scale{r.top, r.top == INFINITY ? 0.f : fminf((float)W.per * ((kBins - 2) / reach), 1e30f)};
}

// the sum of a value over the threads before this one; *all: over all of them
template <int NT>
__device__ __forceinline__ uint64_t block_before(uint64_t v, BlockLds<NT>& L, uint64_t* all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t in = wave_scan(v);
    __syncthreads();
    if (lane == 63) L.part[wave] = in;
    __syncthreads();
    uint64_t before = in - v, sum = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        const uint64_t x = L.part[w];
        if (w < wave) before += x;
        sum += x;
    }
    *all = sum;
    return before;
}
// The bin at which above + the sum of the bins from the first on reaches what
// is wanted (found[0], kBins if none), and the sum before it (found[1]).
// want_of(sum of all bins) says what that is, and is its result.
template <int NT, class Want>
__device__ __forceinline__ uint64_t find_bin(const uint64_t* bins, uint64_t above, Want want_of, BlockLds<NT>& L) {
    constexpr int N = kBins / NT;
    uint64_t x[N], sum = 0, all;
#pragma unroll
    for (int i = 0; i < N; ++i) sum += x[i] = bins[N * threadIdx.x + i];
    uint64_t before = above + block_before<NT>(sum, L, &all);
    const uint64_t want = want_of(all);
    if (threadIdx.x == 0) L.found[0] = kBins;
    __syncthreads();
    if (before < want && want <= before + sum) {
        int i = 0;
#pragma unroll
        for (int j = 0; j < N - 1; ++j)
            if (i == j && before + x[j] < want) {
                before += x[j];
                ++i;
            }
        L.found[0] = N * threadIdx.x + i;
        L.found[1] = before;
    }
    __syncthreads();
    return want;
}
// What a draw from sums of `all` looks for: the first running sum above u all,
// a whole number, so above its floor, and at most all.
__device__ __forceinline__ uint64_t draw_at(const SampleSpace& s, int b, uint64_t all) {
    const double u = fmin(fmax(s.a.u[b], 0.0), 1.0);
    return min((uint64_t)(u * (double)all), all - 1);
}
__device__ __forceinline__ float probability(const SampleSpace& s, const Weights& W, float v, uint64_t all) {
    return (float)(W.of(v) * (4503599627370496.0 / s.lift) / (double)all);  // 2^52 / lift: units of 1
}
// at least one unit: the first token stays
__device__ __forceinline__ uint64_t share(float p, uint64_t all) {
    const double x = __builtin_ceil((double)p * (double)all);
    return x < 1.0 ? 1 : x >= (double)all ? all : (uint64_t)x;
}
__device__ __forceinline__ void add(uint64_t* at, uint64_t v) {
    atomicAdd((unsigned long long*)at, (unsigned long long)v);
}
// To a bin, but what falls in the last one (often most of a row, and adds to
// one address take turns) is summed by each lane for itself: 61 -> 35 us for
// 256 rows of 128k with mixed filters. add_rest brings it there in the end.
__device__ __forceinline__ void add_bin(uint64_t* bins, int n, uint64_t v, uint64_t& rest) {
    if (n == kBins - 1)
        rest += v;
    else
        add(&bins[n], v);
}
__device__ __forceinline__ void add_rest(uint64_t* bins, uint64_t rest) {
    rest = wave_total(rest);
    if ((threadIdx.x & 63) == 0 && rest) add(&bins[kBins - 1], rest);
}

// Tiles [t0, t1) of a row, a wave 4 at a time: f(tile, values) for those that
// on(tile) says, then end(first of the 4, which of them).
struct Nothing {
    __device__ __forceinline__ void operator()(int, uint32_t) const {}
};
template <int NT, bool BF16, class On, class F, class End = Nothing>
__device__ __forceinline__ void each_tile(const Row<BF16>& row, int t0, int t1, On on, F f, End end = End()) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    t1 = min(t1, row.tiles);
    for (int t = t0 + wave * 4; t < t1; t += NT / 64 * 4) {
        u32x4 x[4][Row<BF16>::P];
        uint32_t is = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (t + j < t1 && __builtin_amdgcn_readfirstlane(on(t + j))) is |= 1u << j;
        if (!is) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) row.load(x[j], t + j, (is >> j) & 1, lane);
        issue_fence();
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if ((is >> j) & 1) {
                float v[8];
                row.values(v, x[j], t + j, lane);
                f(t + j, v);
            }
        end(t, is);
    }
}
// The same for the tiles of a list.
template <int NT, bool BF16, class F>
__device__ __forceinline__ void each_listed(const Row<BF16>& row, const int* tiles, int n, F f) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int i = wave * 4; i < n; i += NT / 64 * 4) {
        u32x4 x[4][Row<BF16>::P];
        int t[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) t[j] = __builtin_amdgcn_readfirstlane(tiles[min(i + j, n - 1)]);
#pragma unroll
        for (int j = 0; j < 4; ++j) row.load(x[j], t[j], true, lane);
        issue_fence();
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < n) {
                float v[8];
                row.values(v, x[j], t[j], lane);
                f(t[j], v);
            }
    }
}
// The sums of 4 values over a wave: of value i in the lanes 16 i to 16 i + 15.
__device__ __forceinline__ uint64_t wave_totals(const uint64_t (&x)[4], int lane) {
    const bool h = lane & 32, q = lane & 16;
    const uint64_t a = (h ? x[2] : x[0]) + lane_xor<32>(h ? x[0] : x[2]);
    const uint64_t b = (h ? x[3] : x[1]) + lane_xor<32>(h ? x[1] : x[3]);
    uint64_t v = (q ? b : a) + lane_xor<16>(q ? a : b);
    v += lane_xor<8>(v);
    v += lane_xor<4>(v);
    v += lane_xor<2>(v);
    return v + lane_xor<1>(v);
}

// ------------------------------------------------------------- row by tiles --
constexpr int kTilesNT = 256;

__device__ __forceinline__ void tile_top(float* tops, int t, const float (&v)[8], int lane) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, v[j]);  // of a number and NaN the number
    m = wave_max(m);
    if (lane == 0) tops[t] = m;
}

template <bool BF16>
__global__ __launch_bounds__(kTilesNT) void sample_tops_kernel(SampleSpace s) {
    const int b = blockIdx.y, lane = threadIdx.x & 63, t0 = blockIdx.x * s.per_wg;
    const Row<BF16> row(s.a, b);
    each_tile<kTilesNT>(
        row, t0, t0 + s.per_wg, [](int) { return true; },
        [&](int t, const float(&v)[8]) {
            tile_top(s.tops + (int64_t)b * s.nt, t, v, lane);
        });
    // what the others add to
    for (int i = blockIdx.x * kTilesNT + threadIdx.x; i < kBins; i += gridDim.x * kTilesNT)
        s.bins[(int64_t)b * kBins + i] = 0;
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) s.state[b].count = 0, s.state[b].drawn = 0;
        // the tile that only rows of another alignment have
        for (int t = row.tiles + threadIdx.x; t < s.nt; t += kTilesNT) s.tops[(int64_t)b * s.nt + t] = -INFINITY;
    }
}

// The tiles' sums of the tokens that a prefix and min_p leave.
template <int NT, bool BF16>
__device__ __forceinline__ void tile_sums(const SampleSpace& s, const Row<BF16>& row, const float* tops, int t0, int t1,
                                          const Ask& r, const Weights& W, Prefix kept, uint64_t* sums) {
    const int lane = threadIdx.x & 63;
    const double least = (double)r.least;
    for (int t = t0 + threadIdx.x; t < min(t1, s.nt); t += NT) sums[t] = 0;
    __syncthreads();
    uint64_t x[4] = {0, 0, 0, 0};
    each_tile<NT>(
        row, t0, t1, [&](int t) { return tops[t] >= kept.v && (least == 0.0 || W.of(tops[t]) >= least); },
        [&](int t, const float(&v)[8]) {
            uint64_t y = 0;
            bool is[8], any = false;
#pragma unroll
            for (int j = 0; j < 8; ++j) any |= is[j] = kept.holds(v[j], row.index(t, j, lane));
            if (__any(any)) {
                double w[8];
                W.of<8>(w, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) y += is[j] && !(w[j] < least) ? W.whole(w[j]) : 0;
            }
            x[t & 3] = y;  // t0 is a multiple of 4: a constant place
        },
        [&](int t, uint32_t is) {
            const uint64_t y = wave_totals(x, lane);
            if ((lane & 15) == 0 && (is >> (lane >> 4)) & 1) sums[t + (lane >> 4)] = y;
        });
}

template <bool BF16>
__global__ __launch_bounds__(kTilesNT) void sample_bins_kernel(SampleSpace s) {
    __shared__ uint64_t bins[kBins];
    __shared__ BlockLds<kTilesNT> L;
    const int b = blockIdx.y, t0 = blockIdx.x * s.per_wg;
    const Ask r = find_way<kTilesNT>(s, b, s.tops + (int64_t)b * s.nt, L);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        RowState& st = s.state[b];
        st.way = r.way, st.live = r.live, st.top = r.top, st.under = r.under;
    }
    if (r.way == kDone || r.way == kFew) return;
    const Row<BF16> row(s.a, b);
    const Weights W = weights_of(s, r);
    if (r.way == kSums) {
        tile_sums<kTilesNT>(s, row, s.tops + (int64_t)b * s.nt, t0, t0 + s.per_wg, r, W, Prefix{-INFINITY, -1},
                            s.sums + (int64_t)b * s.nt);
        return;
    }
    const bool mass = r.way == kMass;
    const Scale S = mass ? scale_of_mass(r, W, s.a.V) : scale_of_count(r);
    for (int i = threadIdx.x; i < kBins; i += kTilesNT) bins[i] = 0;
    __syncthreads();
    uint64_t rest = 0;
    if (mass)
        each_tile<kTilesNT>(
            row, t0, t0 + s.per_wg, [](int) { return true; },
            [&](int, const float(&v)[8]) {
                double w[8];
                W.of<8>(w, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint64_t q = W.whole(w[j]);
                    const int n = S.bin(v[j]);
                    rest += n == kBins - 1 ? q : 0;
                    if (n < kBins - 1 && q) add(&bins[n], q);
                }
            });
    else
        each_tile<kTilesNT>(
            row, t0, t0 + s.per_wg, [](int) { return true; },
            [&](int, const float(&v)[8]) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (v[j] > -INFINITY) add_bin(bins, S.bin(v[j]), 1, rest);
            });
    add_rest(bins, rest);
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kTilesNT)
        if (bins[i]) add(&s.bins[(int64_t)b * kBins + i], bins[i]);
}

// Whether the tokens down to the border's bin, `through` by count or weight, are
// at most kList for sure: then all of them are gathered, and the border's
// workgroup has what it needs to draw. Of top_p: none of them weighs less than
// the bin's far edge.
__device__ __forceinline__ bool short_list(bool mass, const Weights& W, const Scale& S, int bin, uint64_t through) {
    if (!mass) return through <= kList;
    if (bin == kBins - 1 || !(S.per > 0.f)) return false;
    const uint64_t edge = W.whole(W.of(S.top - (float)(bin + 2) / S.per));
    return edge > 0 && through / edge <= kList;
}

template <bool BF16>
__global__ __launch_bounds__(kTilesNT) void sample_gather_kernel(SampleSpace s) {
    __shared__ BlockLds<kTilesNT> L;
    __shared__ uint64_t list[kList];
    const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 63, t0 = blockIdx.x * s.per_wg;
    const Ask r = known_way(s, b);
    if (r.way != kCount && r.way != kMass) return;
    const Row<BF16> row(s.a, b);
    const Weights W = weights_of(s, r);
    const bool mass = r.way == kMass;
    const Scale S = mass ? scale_of_mass(r, W, s.a.V) : scale_of_count(r);
    find_bin<kTilesNT>(
        s.bins + (int64_t)b * kBins, 0, [&](uint64_t all) { return mass ? share(r.p, all) : (uint64_t)r.k; }, L);
    const int bin = (int)L.found[0];
    if (bin == kBins) return;
    const bool all = short_list(mass, W, S, bin, L.found[1] + s.bins[(int64_t)b * kBins + bin]);  // uniform
    const float* tops = s.tops + (int64_t)b * s.nt;
    if (tid == 0) L.count = 0;
    __syncthreads();
    each_tile<kTilesNT>(
        row, t0, t0 + s.per_wg, [&](int t) { return S.bin(tops[t]) <= bin; },
        [&](int t, const float(&v)[8]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int n = S.bin(v[j]);
                if (v[j] > -INFINITY && (n == bin || (all && n < bin))) {
                    const uint32_t at = atomicAdd(&L.count, 1u);
                    if (at < kList) list[at] = token(v[j], row.index(t, j, lane));
                }
            }
        });
    __syncthreads();
    const uint32_t n = L.count;
    __syncthreads();
    if (n == 0) return;
    if (tid == 0) L.count = atomicAdd(&s.state[b].count, n);
    __syncthreads();
    for (uint32_t i = tid, at = L.count; i < n && at + i < kList; i += kTilesNT)
        s.list[(int64_t)b * kList + at + i] = list[i];
}

// ------------------------------------------------------------------ borders --
constexpr int kBorderNT = 1024;
struct BorderLds {
    uint64_t bins[kBins];
    uint64_t list[kList];
    uint64_t space[kBorderNT];
    BlockLds<kBorderNT> block;
};

// The n-th (from 1) of the tokens with this logit; there are at least n.
template <bool BF16>
__device__ __forceinline__ Prefix nth_equal(const Row<BF16>& row, const float* tops, float v0, uint64_t n,
                                            BorderLds& L) {
    const int lane = threadIdx.x & 63;
    int sh = 0;  // tiles of a bin, then of one wave's walk
    while (((row.tiles - 1) >> sh) >= kBins) ++sh;
    for (int i = threadIdx.x; i < kBins; i += kBorderNT) L.bins[i] = 0;
    __syncthreads();
    each_tile<kBorderNT>(
        row, 0, row.tiles, [&](int t) { return tops[t] >= v0; },
        [&](int t, const float(&v)[8]) {
            int c = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) c += __popcll(__ballot(v[j] == v0));
            if (lane == 0 && c) add(&L.bins[t >> sh], c);
        });
    __syncthreads();
    find_bin<kBorderNT>(L.bins, 0, [&](uint64_t) { return n; }, L.block);
    const int t0 = (int)L.block.found[0] << sh;
    uint64_t left = n - L.block.found[1];
    if (threadIdx.x < 64)
        for (int t = t0; t < min(t0 + (1 << sh), row.tiles); ++t) {
            u32x4 x[Row<BF16>::P];
            float v[8];
            row.load(x, t, true, lane);
            row.values(v, x, t, lane);
            uint64_t done = 0;
#pragma unroll
            for (int i = 0; i < Row<BF16>::P; ++i) {
                uint32_t c = 0;
#pragma unroll
                for (int e = 0; e < Row<BF16>::E; ++e) c += v[i * Row<BF16>::E + e] == v0;
                const uint64_t in = wave_scan(c);
                uint64_t at = done + in - c;
#pragma unroll
                for (int e = 0; e < Row<BF16>::E; ++e) {
                    const int j = i * Row<BF16>::E + e;
                    if (v[j] == v0 && ++at == left) L.block.found[2] = row.index(t, j, lane);
                }
                done += shfl64(in, 63);
            }
            if (left <= done) break;  // uniform
            left -= done;
        }
    __syncthreads();
    const Prefix p{v0, (int)L.block.found[2]};
    __syncthreads();
    return p;
}

// Of the n <= kList tokens in L.list: the one at which above + the sum of the
// weights from the largest token on reaches `want`. The tokens' range is cut by
// histograms until few are left, which are ranked.
template <class Weight>
__device__ __forceinline__ Prefix rank_list(int n, uint64_t above, uint64_t want, Weight weight, BorderLds& L) {
    constexpr int M = kList / kBorderNT;
    const int tid = threadIdx.x, lane = tid & 63;
    uint64_t mine[M], w[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int i = tid + m * kBorderNT;
        mine[m] = i < n ? L.list[i] : 0;  // no token is 0
        w[m] = i < n ? weight(token_logit(mine[m])) : 0;
    }
    uint64_t low = 1, high = ~0ull;  // the border is in [low, high]
    for (;;) {
        // how many are left, and their range
        uint64_t lo = ~0ull, hi = 0;
        uint32_t c = 0;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const bool in = mine[m] >= low && mine[m] <= high;
            lo = in && mine[m] < lo ? mine[m] : lo;
            hi = in && mine[m] > hi ? mine[m] : hi;
            c += __popcll(__ballot(in));
        }
        lo = wave_all(lo, [](uint64_t a, uint64_t b) { return a < b ? a : b; });
        hi = wave_all(hi, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
        for (int i = tid; i < kBins; i += kBorderNT) L.bins[i] = 0;
        __syncthreads();
        if (tid == 0) {
            L.block.found[0] = ~0ull;
            L.block.found[1] = 0;
            L.block.count = 0;
        }
        __syncthreads();
        if (lane == 0 && c) {
            atomicMin((unsigned long long*)&L.block.found[0], (unsigned long long)lo);
            atomicMax((unsigned long long*)&L.block.found[1], (unsigned long long)hi);
            atomicAdd(&L.block.count, c);
        }
        __syncthreads();
        low = L.block.found[0];
        high = L.block.found[1];
        if (L.block.count <= 64) break;
        const int sh = max(0, 64 - __builtin_clzll(high - low) - 11);  // (high - low) >> sh < 2048
#pragma unroll
        for (int m = 0; m < M; ++m)
            if (mine[m] >= low && mine[m] <= high) add(&L.bins[(high - mine[m]) >> sh], w[m]);
        __syncthreads();
        find_bin<kBorderNT>(L.bins, above, [&](uint64_t) { return want; }, L.block);
        const uint64_t at = L.block.found[0];
        above = L.block.found[1];
        const uint64_t top = high - (at << sh), width = (1ull << sh) - 1;
        low = top - low > width ? top - width : low;
        high = top;
        __syncthreads();
    }
    // at most 64: compacted, then each against the others
    __syncthreads();
    if (tid == 0) L.block.count = 0;
    __syncthreads();
#pragma unroll
    for (int m = 0; m < M; ++m)
        if (mine[m] >= low && mine[m] <= high) {
            const uint32_t at = atomicAdd(&L.block.count, 1u);
            L.list[at] = mine[m];
            L.bins[at] = w[m];
        }
    __syncthreads();
    const int c = (int)L.block.count;
    if (tid < c) {
        const uint64_t me = L.list[tid], mw = L.bins[tid];
        uint64_t before = above;
        for (int j = 0; j < c; ++j)
            if (L.list[j] > me) before += L.bins[j];
        if (before < want && want <= before + mw) L.block.found[2] = me;
    }
    __syncthreads();
    const Prefix p = up_to(L.block.found[2]);
    __syncthreads();
    return p;
}

// A step of a bitonic sort: of two places the lower takes the larger number in a
// falling run of `size`.
__device__ __forceinline__ uint64_t sort_pick(uint64_t x, uint64_t y, int i, int stride, int size) {
    const bool larger = ((i & stride) == 0) == ((i & size) == 0);
    return (x > y) == larger ? x : y;
}
template <int STRIDE>
__device__ __forceinline__ uint64_t sort_steps(uint64_t x, int i, int size) {  // STRIDE, STRIDE / 2, ... 1
    x = sort_pick(x, lane_xor<STRIDE>(x), i, STRIDE, size);
    if constexpr (STRIDE > 1) x = sort_steps<STRIDE / 2>(x, i, size);
    return x;
}
// M numbers a thread, number i = thread + 1024 m, of the first n (a power of 2
// from 64 on), in falling order.
template <int M>
__device__ __forceinline__ void sort_falling(uint64_t (&x)[M], int n, uint64_t* space) {
    const int tid = threadIdx.x;
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int i = tid + m * kBorderNT;
        if (i < n) {  // whole waves
            x[m] = sort_steps<1>(x[m], i, 2);
            x[m] = sort_steps<2>(x[m], i, 4);
            x[m] = sort_steps<4>(x[m], i, 8);
            x[m] = sort_steps<8>(x[m], i, 16);
            x[m] = sort_steps<16>(x[m], i, 32);
            x[m] = sort_steps<32>(x[m], i, 64);
        }
    }
    for (int size = 128; size <= n; size *= 2) {
        if constexpr (M == 2)
            if (size > kBorderNT) {
                const uint64_t y = x[0] > x[1] ? x[0] : x[1];
                x[1] = x[0] > x[1] ? x[1] : x[0];
                x[0] = y;
            }
        for (int stride = min(size, kBorderNT) / 2; stride >= 64; stride /= 2)
#pragma unroll
            for (int m = 0; m < M; ++m) {
                __syncthreads();
                space[tid] = x[m];
                __syncthreads();
                x[m] = sort_pick(x[m], space[tid ^ stride], tid + m * kBorderNT, stride, size);
            }
#pragma unroll
        for (int m = 0; m < M; ++m)
            if (tid + m * kBorderNT < n) x[m] = sort_steps<32>(x[m], tid + m * kBorderNT, size);
    }
    __syncthreads();
}

// From the n <= 1024 M tokens in L.list, which hold every one that can be kept,
// to the draw: in their order, where the filters are prefixes, then by index.
// want: what top_p asks for, where it is the first filter.
template <int M>
__device__ __forceinline__ void finish_list(const SampleSpace& s, int b, const Ask& r, const Weights& W, int n,
                                            uint64_t want, BorderLds& L) {
    const int tid = threadIdx.x;
    const double least = (double)r.least;
    int size = 64;
    while (size < n) size *= 2;
    uint64_t x[M], q[M], all;
    double w[M];
    bool kept[M];
#pragma unroll
    for (int m = 0; m < M; ++m) x[m] = tid + m * kBorderNT < n ? L.list[tid + m * kBorderNT] : 0;
    sort_falling<M>(x, size, L.space);
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int i = tid + m * kBorderNT;
        w[m] = W.of(token_logit(x[m]));
        kept[m] = x[m] != 0 && (r.k == 0 || i < r.k);
        q[m] = kept[m] ? W.whole(w[m]) : 0;
        L.list[i] = x[m];
    }
    if (r.p < 1.f) {
        uint64_t before[M], sum = 0;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            before[m] = sum + block_before<kBorderNT>(q[m], L.block, &all);
            sum += all;
        }
#pragma unroll
        for (int m = 0; m < M; ++m) kept[m] = kept[m] && before[m] < (r.k ? share(r.p, sum) : want);
    }
    // the index, inverted, and the place in the order: 0 where nothing is kept
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int i = tid + m * kBorderNT;
        kept[m] = kept[m] && (!(w[m] < least) || i == 0);
        L.bins[i] = kept[m] ? W.whole(w[m]) : 0;
        x[m] = kept[m] ? x[m] << 32 | (uint32_t)i : 0;
    }
    // what is kept is the first of them, of top_k no more than k
    if (r.k)
        while (size > 64 && size / 2 >= r.k) size /= 2;
    sort_falling<M>(x, size, L.space);
    uint64_t before[M], sum = 0;
#pragma unroll
    for (int m = 0; m < M; ++m) {
        q[m] = x[m] ? L.bins[(uint32_t)x[m]] : 0;
        before[m] = sum + block_before<kBorderNT>(q[m], L.block, &all);
        sum += all;
    }
    const uint64_t pass = draw_at(s, b, sum);
#pragma unroll
    for (int m = 0; m < M; ++m)
        if (before[m] <= pass && pass < before[m] + q[m]) {
            const uint64_t t = L.list[(uint32_t)x[m]];
            s.a.ids[b] = token_index(t);
            s.a.probs[b] = probability(s, W, token_logit(t), sum);
        }
}
__device__ __forceinline__ void finish(const SampleSpace& s, int b, const Ask& r, const Weights& W, int n,
                                       uint64_t want, BorderLds& L) {
    if (n <= kBorderNT)
        finish_list<1>(s, b, r, W, n, want, L);
    else
        finish_list<kList / kBorderNT>(s, b, r, W, n, want, L);
}

// The shortest prefix of `in` with at least k of its tokens (MASS false) or p
// of its weights (MASS true), by this workgroup alone; `in` where it has less.
// No border lies behind bin `last`; tokens behind it are not looked at (of MASS
// it is the last there is). may, only where `in` is every token: where the list
// down to the border is short the draw is made from it, and `drawn` says so.
template <bool BF16, bool MASS>
__device__ __forceinline__ Prefix border(const SampleSpace& s, int b, const Row<BF16>& row, const float* tops,
                                         const Ask& r, const Weights& W, Prefix in, const Scale& S, int last,
                                         BorderLds& L, bool may, bool& drawn) {
    const int tid = threadIdx.x, lane = tid & 63;
    auto weight = [&](float v) -> uint64_t { return MASS ? W.whole(W.of(v)) : 1; };
    for (int i = tid; i < kBins; i += kBorderNT) L.bins[i] = 0;
    __syncthreads();
    uint64_t rest = 0;
    each_tile<kBorderNT>(
        row, 0, row.tiles, [&](int t) { return tops[t] >= in.v && S.bin(tops[t]) <= last; },
        [&](int t, const float(&v)[8]) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (in.holds(v[j], row.index(t, j, lane))) {
                    const int n = S.bin(v[j]);
                    if (n <= last) add_bin(L.bins, n, weight(v[j]), rest);
                }
        });
    add_rest(L.bins, rest);
    __syncthreads();
    const uint64_t want = find_bin<kBorderNT>(
        L.bins, 0, [&](uint64_t all) { return MASS ? share(r.p, all) : (uint64_t)r.k; }, L.block);
    const int bin = (int)L.block.found[0];
    uint64_t above = L.block.found[1];
    __syncthreads();
    if (bin == kBins) return in;
    // the tokens of the border's bin, or down to there
    const bool all = may && short_list(MASS, W, S, bin, above + L.bins[bin]);
    float low = INFINITY, high = -INFINITY;
    if (tid == 0) L.block.count = 0;
    __syncthreads();
    each_tile<kBorderNT>(
        row, 0, row.tiles, [&](int t) { return tops[t] >= in.v && S.bin(tops[t]) <= bin; },
        [&](int t, const float(&v)[8]) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (in.holds(v[j], row.index(t, j, lane)) && (all ? S.bin(v[j]) <= bin : S.bin(v[j]) == bin)) {
                    const uint32_t at = atomicAdd(&L.block.count, 1u);
                    if (at < kList) L.list[at] = token(v[j], row.index(t, j, lane));
                    low = fminf(low, v[j]);
                    high = fmaxf(high, v[j]);
                }
        });
    __syncthreads();
    const int n = (int)L.block.count;
    __syncthreads();
    if (all) {
        finish(s, b, r, W, n, want, L);
        drawn = true;
        return in;
    }
    if (n <= kList) return rank_list(n, above, want, weight, L);
    // more tokens than the list holds: by the digits of their logits' order
    low = wave_min(low);
    high = wave_max(high);
    if (lane == 0) {
        L.block.part_top[tid >> 6] = high;
        L.block.part_under[tid >> 6] = low;
    }
    __syncthreads();
    for (int w = 0; w < kBorderNT / 64; ++w) {
        low = fminf(low, L.block.part_under[w]);
        high = fmaxf(high, L.block.part_top[w]);
    }
    auto key = [](float v) { return (uint32_t)(token(v, 0) >> 32); };
    uint32_t k0 = key(low), k1 = key(high);
    while (k0 != k1) {
        int sh = 0;
        while (((k1 - k0) >> sh) >= kBins) ++sh;
        for (int i = tid; i < kBins; i += kBorderNT) L.bins[i] = 0;
        __syncthreads();
        each_tile<kBorderNT>(
            row, 0, row.tiles, [&](int t) { return key(tops[t]) >= k0; },
            [&](int t, const float(&v)[8]) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t k = key(v[j]);
                    if (k >= k0 && k <= k1 && in.holds(v[j], row.index(t, j, lane)))
                        add(&L.bins[(k1 - k) >> sh], weight(v[j]));
                }
            });
        __syncthreads();
        find_bin<kBorderNT>(L.bins, above, [&](uint64_t) { return want; }, L.block);
        const uint32_t top = k1 - ((uint32_t)L.block.found[0] << sh), width = (1u << sh) - 1;
        above = L.block.found[1];
        k0 = top - k0 > width ? top - width : k0;
        k1 = top;
        __syncthreads();
    }
    const float v0 = token_logit((uint64_t)k1 << 32);
    const uint64_t one = weight(v0);
    return nth_equal(row, tops, v0, (want - above + one - 1) / one, L);
}

// A row without a token that can be drawn.
__device__ __forceinline__ bool no_token(const SampleSpace& s, int b, const Ask& r) {
    if (r.top != -INFINITY) return false;
    if (threadIdx.x == 0) {
        s.a.ids[b] = -1;
        s.a.probs[b] = 0.f;
    }
    return true;
}
// The first token in the order: of the largest logits the one at the lowest
// index.
template <int NT, bool BF16>
__device__ __forceinline__ void first_token(const SampleSpace& s, const Row<BF16>& row, int b, const Ask& r,
                                            const float* tops, BlockLds<NT>& L) {
    const int tid = threadIdx.x, lane = tid & 63;
    if (tid == 0) L.found[0] = ~0ull;
    __syncthreads();
    for (int i = tid; i < s.nt; i += NT)
        if (tops[i] == r.top) atomicMin((unsigned long long*)&L.found[0], (unsigned long long)i);
    __syncthreads();
    if (tid >= 64) return;
    const int t = (int)L.found[0];
    u32x4 x[Row<BF16>::P];
    float v[8];
    row.load(x, t, true, lane);
    row.values(v, x, t, lane);
    int first = 0x7fffffff;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (v[j] == r.top) first = min(first, row.index(t, j, lane));
    first = (int)wave_all((uint32_t)first, [](uint32_t a, uint32_t b) { return min(a, b); });
    if (lane == 0) {
        s.a.ids[b] = first;
        s.a.probs[b] = 1.f;
    }
}

// The draw, from the tiles' sums.
template <int NT, bool BF16>
__device__ __forceinline__ void draw(const SampleSpace& s, const Row<BF16>& row, int b, const Ask& r, const Weights& W,
                                     Prefix kept, const float* tops, const uint64_t* sums, BlockLds<NT>& L) {
    const int tid = threadIdx.x, lane = tid & 63;
    const double least = (double)r.least;
    const int per = (s.nt + NT - 1) / NT, t0 = min(tid * per, s.nt), t1 = min(t0 + per, s.nt);
    uint64_t mine = 0, all;
    for (int i = t0; i < t1; ++i) mine += sums[i];
    uint64_t before = block_before<NT>(mine, L, &all);
    if (all == 0) {  // min_p above every weight
        first_token<NT>(s, row, b, r, tops, L);
        return;
    }
    const uint64_t pass = draw_at(s, b, all);
    if (before <= pass && pass < before + mine) {
        int i = t0;
        for (; before + sums[i] <= pass; ++i) before += sums[i];
        L.found[0] = i;
        L.found[1] = pass - before;
    }
    __syncthreads();
    if (tid >= 64) return;
    const int t = (int)L.found[0];
    const uint64_t left = L.found[1];
    u32x4 x[Row<BF16>::P];
    float v[8];
    row.load(x, t, true, lane);
    row.values(v, x, t, lane);
    uint64_t run = 0;
#pragma unroll
    for (int i = 0; i < Row<BF16>::P; ++i) {
        uint64_t w[Row<BF16>::E], sum = 0;
#pragma unroll
        for (int e = 0; e < Row<BF16>::E; ++e) {
            const int j = i * Row<BF16>::E + e;
            const double wj = W.of(v[j]);
            w[e] = kept.holds(v[j], row.index(t, j, lane)) && !(wj < least) ? W.whole(wj) : 0;
            sum += w[e];
        }
        const uint64_t in = run + wave_scan(sum);
        const uint64_t m = __ballot(in > left);
        if (m) {
            if (lane == __builtin_ctzll(m)) {
                uint64_t at = in - sum;
                bool done = false;
#pragma unroll
                for (int e = 0; e < Row<BF16>::E; ++e) {
                    at += w[e];
                    if (!done && at > left) {
                        const int j = i * Row<BF16>::E + e;
                        s.a.ids[b] = row.index(t, j, lane);
                        s.a.probs[b] = probability(s, W, v[j], all);
                        done = true;
                    }
                }
            }
            return;
        }
        run = shfl64(in, 63);
    }
}

// A top_k up to the number of tiles: whether that was all (drawn), or the border.
// tiles: room for a list of them.
template <bool BF16>
__device__ __forceinline__ bool few(const SampleSpace& s, const Row<BF16>& row, int b, const Ask& r, const Weights& W,
                                    const float* tops, int* tiles, Prefix& kept, BorderLds& L) {
    // at least k tokens lie at or above the k-th largest of the tiles' tops
    const int tid = threadIdx.x, lane = tid & 63;
    const Scale S = scale_of_count(r);
    for (int i = tid; i < kBins; i += kBorderNT) L.bins[i] = 0;
    __syncthreads();
    for (int i = tid; i < s.nt; i += kBorderNT)
        if (tops[i] > -INFINITY) add(&L.bins[S.bin(tops[i])], 1);
    __syncthreads();
    find_bin<kBorderNT>(L.bins, 0, [&](uint64_t) { return (uint64_t)r.k; }, L.block);
    const int last = min((int)L.block.found[0], kBins - 1);
    if (tid == 0) L.block.count = 0;
    __syncthreads();
    for (int i = tid; i < row.tiles; i += kBorderNT)
        if (tops[i] > -INFINITY && S.bin(tops[i]) <= last) tiles[atomicAdd(&L.block.count, 1u)] = i;
    __syncthreads();
    const int live = (int)L.block.count;
    __syncthreads();
    if (tid == 0) L.block.count = 0;
    __syncthreads();
    each_listed<kBorderNT>(
        row, tiles, live, [&](int t, const float(&v)[8]) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (v[j] > -INFINITY && S.bin(v[j]) <= last) {
                    const uint32_t at = atomicAdd(&L.block.count, 1u);
                    if (at < kList) L.list[at] = token(v[j], row.index(t, j, lane));
                }
        });
    __syncthreads();
    const int n = (int)L.block.count;
    bool drawn = n <= kList;
    if (drawn) {
        finish(s, b, r, W, n, 0, L);
        return true;
    }
    kept = border<BF16, false>(s, b, row, tops, r, W, Prefix{-INFINITY, -1}, S, last, L, false, drawn);
    return drawn;
}

template <bool BF16>
__global__ __launch_bounds__(kBorderNT) void sample_border_kernel(SampleSpace s) {
    extern __shared__ float lds_tops[];  // [nt], then a list of tiles
    __shared__ BorderLds L;
    const int tid = threadIdx.x, b = blockIdx.x;
    const Ask r = known_way(s, b);
    if (r.way == kSums || r.way == kDone) return;
    const Row<BF16> row(s.a, b);
    const Weights W = weights_of(s, r);
    const float* tops = lds_tops;
    for (int i = tid; i < s.nt; i += kBorderNT) lds_tops[i] = s.tops[(int64_t)b * s.nt + i];
    const Prefix every{-INFINITY, -1};
    Prefix kept = every;
    bool drawn = false;
    if (r.way == kFew) {
        drawn = few(s, row, b, r, W, tops, reinterpret_cast<int*>(lds_tops + s.nt), kept, L);
    } else {
        const bool mass = r.way == kMass;
        const uint64_t want = find_bin<kBorderNT>(
            s.bins + (int64_t)b * kBins, 0, [&](uint64_t all) { return mass ? share(r.p, all) : (uint64_t)r.k; },
            L.block);
        const int bin = (int)L.block.found[0], n = (int)s.state[b].count;
        const uint64_t above = L.block.found[1];
        const Scale S = mass ? scale_of_mass(r, W, s.a.V) : scale_of_count(r);
        __syncthreads();
        if (bin < kBins && n <= kList) {
            for (int i = tid; i < n; i += kBorderNT) L.list[i] = s.list[(int64_t)b * kList + i];
            __syncthreads();
            drawn = short_list(mass, W, S, bin, above + s.bins[(int64_t)b * kBins + bin]);
            if (drawn)
                finish(s, b, r, W, n, want, L);
            else
                kept = rank_list(n, above, want, [&](float v) -> uint64_t { return mass ? W.whole(W.of(v)) : 1; }, L);
        } else if (bin < kBins) {
            kept = mass ? border<BF16, true>(s, b, row, tops, r, W, every, S, kBins - 1, L, false, drawn)
                        : border<BF16, false>(s, b, row, tops, r, W, every, S, kBins - 1, L, false, drawn);
        }
    }
    if (!drawn && r.k && r.p < 1.f)
        kept = border<BF16, true>(s, b, row, tops, r, W, kept, scale_of_mass(r, W, s.a.V), kBins - 1, L, false, drawn);
    if (tid == 0) {
        s.state[b].drawn = drawn;
        s.state[b].kept = kept;
    }
}

// Everything of a row by one workgroup, in one launch.
template <bool BF16>
__global__ __launch_bounds__(kBorderNT) void sample_row_kernel(SampleSpace s) {
    extern __shared__ uint64_t lds_sums[];  // [nt], then the tiles' largest logits, then a list of tiles
    __shared__ BorderLds L;
    const int tid = threadIdx.x, lane = tid & 63, b = blockIdx.x;
    float* tops = reinterpret_cast<float*>(lds_sums + s.nt);
    const Row<BF16> row(s.a, b);
    each_tile<kBorderNT>(
        row, 0, row.tiles, [](int) { return true; }, [&](int t, const float(&v)[8]) { tile_top(tops, t, v, lane); });
    for (int t = row.tiles + tid; t < s.nt; t += kBorderNT) tops[t] = -INFINITY;
    __syncthreads();
    const Ask r = find_way(s, b, tops, L.block);
    __syncthreads();
    if (no_token(s, b, r)) return;
    if (r.way == kDone) {
        first_token(s, row, b, r, tops, L.block);
        return;
    }
    const Weights W = weights_of(s, r);
    const Prefix every{-INFINITY, -1};
    Prefix kept = every;
    bool drawn = false;
    if (r.way == kFew)
        drawn = few(s, row, b, r, W, tops, reinterpret_cast<int*>(tops + s.nt), kept, L);
    else if (r.way == kCount)
        kept = border<BF16, false>(s, b, row, tops, r, W, every, scale_of_count(r), kBins - 1, L, true, drawn);
    if (!drawn && r.p < 1.f)
        kept = border<BF16, true>(s, b, row, tops, r, W, kept, scale_of_mass(r, W, s.a.V), kBins - 1, L,
                                  r.way == kMass, drawn);
    if (drawn) return;
    tile_sums<kBorderNT>(s, row, tops, 0, row.tiles, r, W, kept, lds_sums);
    for (int t = row.tiles + tid; t < s.nt; t += kBorderNT) lds_sums[t] = 0;
    __syncthreads();
    draw(s, row, b, r, W, kept, tops, lds_sums, L.block);
}

template <bool BF16>
__global__ __launch_bounds__(kTilesNT) void sample_sums_kernel(SampleSpace s) {
    const int b = blockIdx.y, t0 = blockIdx.x * s.per_wg;
    const Ask r = known_way(s, b);
    if (s.state[b].drawn || r.way == kDone || r.way == kSums) return;
    const Row<BF16> row(s.a, b);
    tile_sums<kTilesNT>(s, row, s.tops + (int64_t)b * s.nt, t0, t0 + s.per_wg, r, weights_of(s, r), s.state[b].kept,
                        s.sums + (int64_t)b * s.nt);
}

template <bool BF16>
__global__ __launch_bounds__(kTilesNT) void sample_draw_kernel(SampleSpace s) {
    __shared__ BlockLds<kTilesNT> L;
    const int b = blockIdx.x;
    const Ask r = known_way(s, b);
    if (s.state[b].drawn || no_token(s, b, r)) return;
    const Row<BF16> row(s.a, b);
    const float* tops = s.tops + (int64_t)b * s.nt;
    if (r.way == kDone) {
        first_token<kTilesNT>(s, row, b, r, tops, L);
        return;
    }
    const Prefix kept = r.way == kSums ? Prefix{-INFINITY, -1} : s.state[b].kept;
    draw<kTilesNT>(s, row, b, r, weights_of(s, r), kept, tops, s.sums + (int64_t)b * s.nt, L);
}

// -------------------------------------------------------------------- host --
static size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

// Whether a row is one workgroup's from end to end: where it is short, or longer
// and rows fill the chip. us of a workgroup a row against over the chip, bf16, of
// rows without a filter, with top_k 50 and top_p 0.9, with top_p 0.9 alone, of the
// likeliest token, and of a batch with filters of every kind:
//     1 row   of 16000    14 15   18 26   21 27    5  7   20 27
//    16 rows  of 32768    18 15   14 21   41 38    6  8   43 48
//     8       of 40000    19 15   14 21   46 37    6  8   37 39
//    64       of 40960    20 18   15 21   47 45    6  9   50 50
//    96       of 45056    22 20   15 22   52 49    6  9   55 52
//    48       of 50021    22 18   15 22   55 45    6  9   58 50
//    96       of 65536    28 22   15 22   71 56    7  9   72 54
//   192       of 65536    29 31   16 27   71 76    7 12   72 65
//   256       of 65536    30 37   16 31   72 83    7 14   72 70
// Past that the row that takes longest holds up the rest: 256 of 131072 fp32, every
// kind, 139 against 103.
static bool one_a_row(int B, int V) { return V <= (B >= 192 ? 65536 : B >= 32 ? 40960 : 32768); }

size_t sample_workspace(int B, int V) {
    if (one_a_row(B, V)) return 0;
    const size_t tiles = (size_t)B * sample_tiles(V);
    return align256((size_t)B * kBins * 8) + align256(tiles * 8) + align256((size_t)B * kList * 8) +
           align256(tiles * 4) + align256((size_t)B * sizeof(RowState));
}

template <bool BF16>
static hipError_t run(const SampleSpace& s, hipStream_t st, StageTimer* tm) {
    const dim3 tiles((s.nt + s.per_wg - 1) / s.per_wg, s.a.B), rows(s.a.B);
    if (one_a_row(s.a.B, s.a.V))
        return launch_shm(tm, "sample_row", sample_row_kernel<BF16>, rows, dim3(kBorderNT), s.nt * 16, st, s);
    const bool filters = s.a.top_k || s.a.top_p;
    hipError_t e = launch(tm, "sample_tops", sample_tops_kernel<BF16>, tiles, dim3(kTilesNT), st, s);
    if (e == hipSuccess)
        e = launch(tm, "sample_bins", sample_bins_kernel<BF16>, tiles, dim3(kTilesNT), st, s);
    if (e == hipSuccess && filters) {
        e = launch(tm, "sample_gather", sample_gather_kernel<BF16>, tiles, dim3(kTilesNT), st, s);
        if (e == hipSuccess)
            e = launch_shm(tm, "sample_border", sample_border_kernel<BF16>, rows, dim3(kBorderNT), s.nt * 8, st, s);
        if (e == hipSuccess) e = launch(tm, "sample_sums", sample_sums_kernel<BF16>, tiles, dim3(kTilesNT), st, s);
    }
    if (e == hipSuccess) e = launch(tm, "sample_draw", sample_draw_kernel<BF16>, rows, dim3(kTilesNT), st, s);
    return e;
}

hipError_t sample(const SampleArgs& a, bool bf16, hipStream_t st, StageTimer* tm) {
    SampleSpace s{};
    s.a = a;
    // V weights of at most 2^shift add up to less than 2^63
    int bits = 0;
    while ((int64_t)1 << bits < a.V) ++bits;
    s.lift = (double)((int64_t)1 << (52 - std::min(46, 62 - bits)));
    s.nt = sample_tiles(a.V);
    // 4 a wave, whose loads are in flight at once. More would bring fewer
    // histograms to memory (64 tiles, 256 rows of 128k: 30 against 50 us where
    // every row makes one), but rows of a batch mostly go different ways, and the
    // few that pass over all tiles are then spread thinner (39 against 28 us)
    s.per_wg = 16;
    const size_t tiles = (size_t)a.B * s.nt;
    char* ws = static_cast<char*>(a.workspace);
    s.bins = reinterpret_cast<uint64_t*>(ws);
    ws += align256((size_t)a.B * kBins * 8);
    s.sums = reinterpret_cast<uint64_t*>(ws);
    ws += align256(tiles * 8);
    s.list = reinterpret_cast<uint64_t*>(ws);
    ws += align256((size_t)a.B * kList * 8);
    s.tops = reinterpret_cast<float*>(ws);
    ws += align256(tiles * 4);
    s.state = reinterpret_cast<RowState*>(ws);
    return bf16 ? run<true>(s, st, tm) : run<false>(s, st, tm);
}

}  // namespace lora
