// A mixture-of-experts layer for a few tokens:
//   logits = x R^T;  ids, w = the k largest of each token and their softmax;
//   y[t] = sum_j w[t][j] down_e( silu(gate_e x_t) * up_e x_t ),  e = ids[t][j]
// with the experts' weights in bf16 or MXFP4. With few tokens the layer is
// bound by the weights of the experts that are reached: each is read once,
// in 16-byte pieces, for all of its tokens, which ride as the 16 columns of
// the matrix-core products (weights are the left operand).
//
// Route: a wave sums the logit of an expert and a token in 64 bits, so that
// the choice among close logits does not hang on the rounding of a sum; a
// workgroup per token then ranks its logits. 32 tokens and experts of width
// 4096: 4 us each, launches.
// Experts: gate_up (a workgroup takes one reached expert and 32 inner columns:
// 32 gate and 32 up rows), down (one reached expert and 64 output columns),
// combine (the weighted sum of a token's k terms, in the order of j). 32
// tokens, 4 of 32 MXFP4 experts, 4096 x 1792 (all reached, 374 MB): gate_up
// 51 us (4.9 TB/s), down 34 us (3.7 TB/s), combine 4 us.
#include "fuse.h"
#include "kernels.h"
#include "mx4.h"

namespace lora {

// ------------------------------------------------------------------ route --
// A lane's parts of the 64-bit dot products of one bf16 row with NE others
// (rows of `stride` elements), in the order of k; CH pieces of every row in
// flight at once. A product of two bf16 is exact in 64 bits; in fp32 it could
// leave the range (and is no faster but for large calls: 64 tokens x 64 experts
// of width 4096, 4.8 against 5.1 us).
template <int NE, int CH>
__device__ __forceinline__ void dot_rows(const uint16_t* __restrict__ xp, const uint16_t* __restrict__ rp,
                                         int64_t stride, int H, int lane, double (&s)[NE]) {
#pragma unroll
    for (int e = 0; e < NE; ++e) s[e] = 0.0;
    for (int k0 = lane * 8; k0 < H; k0 += 512 * CH) {
        u32x4 a[CH], b[NE][CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const bool ok = k0 + 512 * c < H;
            a[c] = *or_zero(ok, xp + k0 + 512 * c);
#pragma unroll
            for (int e = 0; e < NE; ++e) b[e][c] = *or_zero(ok, rp + e * stride + k0 + 512 * c);
        }
        issue_fence();
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int e = 0; e < NE; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[e] = __builtin_fma((double)__uint_as_float(a[c][i] << 16),
                                         (double)__uint_as_float(b[e][c][i] << 16), s[e]);
                    s[e] = __builtin_fma((double)__uint_as_float(a[c][i] & 0xffff0000u),
                                         (double)__uint_as_float(b[e][c][i] & 0xffff0000u), s[e]);
                }
    }
}
template <int O, int NE>
__device__ __forceinline__ void sum_steps(double (&s)[NE]) {
#pragma unroll
    for (int e = 0; e < NE; ++e) s[e] += lane_xor<O>(s[e]);
    if constexpr (O > 1) sum_steps<O / 2>(s);
}
template <int NE>
__device__ __forceinline__ void wave_sum(double (&s)[NE]) {
    sum_steps<32>(s);
}
// The same sums of 16 values, s[i] in the lanes 4 i to 4 i + 3: every step down
// to lane ^ 4 halves how many values a lane goes on with.
template <int O, int N>
__device__ __forceinline__ double wave_sum16(double (&s)[N]) {
    if constexpr (N > 1) {
        double h[N / 2];
        const bool up = threadIdx.x & O;
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            h[i] = (up ? s[i + N / 2] : s[i]) + lane_xor<O>(up ? s[i] : s[i + N / 2]);
        return wave_sum16<O / 2>(h);
    } else {
        sum_steps<O>(s);
        return s[0];
    }
}

// The order of logits as signed integers: NaN below every number, -0 as 0.
__device__ __forceinline__ int64_t rank_key(double v) {
    const int64_t b = __builtin_bit_cast(int64_t, v + 0.0);
    return v != v ? INT64_MIN : b ^ ((b >> 63) & INT64_MAX);
}

// The k largest of the E logits in LDS, by rank: RT threads of the 1024 count
// for one logit how many come before it (larger, or equal at a lower index);
// ranks below k are the choices. No round waits on another, whatever k. A NaN
// ranks last, so the ids stay valid and distinct; the weights are NaN where it
// is in their sum.
__device__ __forceinline__ void topk_token(const double* logits, int E, int k, int renorm, int32_t* ids,
                                           float* weights, double* sel) {
    const int tid = threadIdx.x;
    const int rt = E <= 64 ? 16 : E <= 128 ? 8 : E <= 256 ? 4 : 2;  // threads per logit, neighbours in a wave
    const int e = tid / rt, part = tid % rt;
    int before = 0;
    if (e < E) {
        const int64_t mine = rank_key(logits[e]);
        for (int j = part; j < E; j += rt) {
            const int64_t other = rank_key(logits[j]);
            before += other > mine || (other == mine && j < e);
        }
    }
    for (int o = 1; o < rt; o <<= 1) before += __shfl_xor(before, o);
    if (e < E && part == 0 && before < k) {
        ids[before] = e;
        sel[before] = logits[e];
    }
    __syncthreads();
    if (tid >= 64) return;
    // weights: exp(l_j - max) over the sum of the chosen (renorm) or of all
    const double top = sel[0];
    const float p = tid < k ? expf((float)(sel[tid] - top)) : 0.f;
    float den = p;
    if (!renorm) {
        den = 0.f;
        for (int i = tid; i < E; i += 64) den += expf((float)(logits[i] - top));
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) den += __shfl_xor(den, o);
    if (tid < k) weights[tid] = p / den;
}

// The logits of a token into LDS: the workgroup's 16 waves take four experts
// at a time.
__device__ __forceinline__ void token_logits(const uint16_t* __restrict__ xp, const uint16_t* __restrict__ R, int H,
                                             int E, double* logits) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int e0 = wave * 4; e0 < E; e0 += 64) {
        double s[4];
        if (e0 + 4 <= E) {  // uniform
            dot_rows<4, 4>(xp, R + (int64_t)e0 * H, H, H, lane, s);
            wave_sum(s);
        } else {
            for (int i = 0; i < 4; ++i) {
                double one[1] = {0.0};
                if (e0 + i < E) dot_rows<1, 4>(xp, R + (int64_t)(e0 + i) * H, H, H, lane, one);
                wave_sum(one);
                s[i] = one[0];
            }
        }
        if (lane < 4 && e0 + lane < E)
            logits[e0 + lane] = lane == 0 ? s[0] : lane == 1 ? s[1] : lane == 2 ? s[2] : s[3];
    }
    __syncthreads();
}

__global__ __launch_bounds__(1024) void moe_route_kernel(const uint16_t* __restrict__ X,
                                                         const uint16_t* __restrict__ R, int H, int E, int k,
                                                         int renorm, int32_t* __restrict__ ids,
                                                         float* __restrict__ weights) {
    __shared__ double logits[kMoeMaxExperts];
    __shared__ double sel[kMoeMaxK];
    const int t = blockIdx.x;
    token_logits(X + (int64_t)t * H, R, H, E, logits);
    topk_token(logits, E, k, renorm, ids + t * k, weights + t * k, sel);
}

// The same over two launches, logits and then one workgroup per token: a
// router too large for one CU to read quickly (512 KB: 11 us in one launch, 8
// in two). A wave takes TE experts and TT tokens, so that rows in registers meet
// several others: 64 tokens and 256 experts of width 4096 take 6.8 us as 4 x 4,
// 13.6 as 1 x 1: one wave a SIMD, whose 2470 vector instructions (1024 of them the
// products, most others unpack and convert their operands) issue for 60 % of
// its life and which waits for loads for 24 %. Each logit is summed as dot_rows does it, whatever the tile.
template <int TE, int TT>
__global__ __launch_bounds__(256) void moe_logits_kernel(const uint16_t* __restrict__ X,
                                                         const uint16_t* __restrict__ R, int T, int H, int E,
                                                         double* __restrict__ logits) {
    constexpr int CH = TE * TT == 1 ? 4 : 2;  // pieces of a row in flight
    const int lane = threadIdx.x & 63, e0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * TE, t0 = blockIdx.y * TT;
    if (e0 >= E) return;
    double s[TE][TT];
#pragma unroll
    for (int e = 0; e < TE; ++e)
#pragma unroll
        for (int t = 0; t < TT; ++t) s[e][t] = 0.0;
    for (int k0 = lane * 8; k0 < H; k0 += 512 * CH) {
        u32x4 a[TE][CH], b[TT][CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = k0 + 512 * c;
#pragma unroll
            for (int e = 0; e < TE; ++e) a[e][c] = *or_zero(k < H, R + (int64_t)min(e0 + e, E - 1) * H + k);
#pragma unroll
            for (int t = 0; t < TT; ++t) b[t][c] = *or_zero(k < H, X + (int64_t)min(t0 + t, T - 1) * H + k);
        }
        issue_fence();
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    double x[TE], y[TT];
#pragma unroll
                    for (int e = 0; e < TE; ++e)
                        x[e] = (double)__uint_as_float(h ? a[e][c][i] & 0xffff0000u : a[e][c][i] << 16);
#pragma unroll
                    for (int t = 0; t < TT; ++t)
                        y[t] = (double)__uint_as_float(h ? b[t][c][i] & 0xffff0000u : b[t][c][i] << 16);
#pragma unroll
                    for (int e = 0; e < TE; ++e)
#pragma unroll
                        for (int t = 0; t < TT; ++t) s[e][t] = __builtin_fma(y[t], x[e], s[e][t]);
                }
    }
    if constexpr (TE * TT == 16) {
        double v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = s[i % TE][i / TE];
        v[0] = wave_sum16<32>(v);
        const int i = lane >> 2, e = e0 + i % TE, t = t0 + i / TE;
        if ((lane & 3) == 0 && e < E && t < T) logits[(int64_t)t * E + e] = v[0];
    } else {
        static_assert(TE * TT == 1, "16 logits a wave, or one");
        wave_sum(s[0]);
        if (lane == 0) logits[(int64_t)t0 * E + e0] = s[0][0];
    }
}

__global__ __launch_bounds__(1024) void moe_topk_kernel(const double* __restrict__ logits, int E, int k, int renorm,
                                                        int32_t* __restrict__ ids, float* __restrict__ weights) {
    __shared__ double lds[kMoeMaxExperts];
    __shared__ double sel[kMoeMaxK];
    const int t = blockIdx.x;
    for (int i = threadIdx.x; i < E; i += 1024) lds[i] = logits[(int64_t)t * E + i];
    __syncthreads();
    topk_token(lds, E, k, renorm, ids + t * k, weights + t * k, sel);
}

// ----------------------------------------------------------- route by scores --
// s_e = sigmoid(l_e), or the softmax of all logits; c_e = s_e + bias_e. With
// groups of n = E / groups neighbours, a group's value is the sum of its
// group_best largest c, and the experts of the top_groups groups of the
// largest values are left. Of these the k largest c are chosen; their weights
// are their s, divided by its sum where renorm, times scale. Everything is
// held in 64 bits, and every choice is by rank, as in topk_token: equal values
// to the lower index, NaN below every number.
// Bound by launches and barriers: 1 token, 128 experts of width 4096 in 8 groups,
// logits 3.3 us and this 5.4; 64 tokens, 256 experts 9.4 and 8.0.
// Above INT64_MIN + 1, so that experts that are not left rank behind every NaN
// (and a key less 1 is one).
__device__ __forceinline__ int64_t score_key(double c) { return max(rank_key(c), INT64_MIN + 2); }
constexpr int64_t kNotLeft = INT64_MIN;
// How many of keys from, from + step, ... below `end` come before number e: larger,
// or equal at a lower index. (One comparison a key: up to e with a number less.)
__device__ __forceinline__ int ranked_before(const int64_t* key, int from, int end, int step, int e) {
    const int64_t mine = key[e];
    int before = 0, j = from;
#pragma unroll 4
    for (; j < min(e, end); j += step) before += key[j] > mine - 1;
#pragma unroll 4
    for (; j < end; j += step) before += key[j] > mine;
    return before;
}
// Chosen scores (by a bias, or by groups) whose sum is below this are near the end
// of 64 bits, or past it, at 0. Both kinds of score are there in proportion to
// e^l, a sigmoid to 2^-960 of itself, so that they are taken against the largest.
constexpr double kSmallScores = 0x1p-960;
struct ScoredLds {
    double logits[kMoeMaxExperts], scores[kMoeMaxExperts];
    int64_t key[kMoeMaxExperts];    // of c; of experts that are not left kNotLeft
    double best[kMoeMaxExperts];    // [groups][group_best] largest c
    int left[kMoeMaxExperts];       // is this group left?
    double sel[kMoeMaxK], sel_logit[kMoeMaxK];
};
__device__ __forceinline__ void scored_token(ScoredLds& L, int E, int k, const RouteScored& r, int32_t* ids,
                                             float* weights) {
    const int tid = threadIdx.x, lane = tid & 63, n = E / r.groups;
    // every wave that holds a score takes the softmax's maximum and sum for itself
    double top = -INFINITY, den = 0.0;
    if (!r.sigmoid && tid - lane < E) {
        for (int i = lane; i < E; i += 64) top = fmax(top, L.logits[i]);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) top = fmax(top, __shfl_xor(top, o));
        for (int i = lane; i < E; i += 64) den += exp(L.logits[i] - top);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) den += __shfl_xor(den, o);
    }
    double s = 0.0, c = 0.0;
    if (tid < E) {
        const double l = L.logits[tid];
        s = r.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - top) / den;
        c = r.bias ? s + (double)r.bias[tid] : s;
        L.key[tid] = score_key(c);
        L.scores[tid] = s;
    }
    __syncthreads();
    const int best = min(r.group_best, n);
    if (r.groups > 1) {
        if (tid < E) {
            const int g0 = tid / n * n, before = ranked_before(L.key, g0, g0 + n, 1, tid);
            if (before < best) L.best[tid / n * best + before] = c;
        }
        __syncthreads();
        if (tid < r.groups) {
            auto value = [&](int g) { return score_key(best == 2 ? L.best[2 * g] + L.best[2 * g + 1] : L.best[g]); };
            const int64_t mine = value(tid);
            int before = 0;
            for (int g = 0; g < r.groups; ++g) {
                const int64_t other = value(g);
                before += other > mine || (other == mine && g < tid);
            }
            L.left[tid] = before < r.top_groups;
        }
        __syncthreads();
        if (tid < E && !L.left[tid / n]) L.key[tid] = kNotLeft;
    }
    __syncthreads();
    const int rt = E <= 64 ? 16 : E <= 128 ? 8 : E <= 256 ? 4 : 2;  // threads per expert, neighbours in a wave
    const int e = tid / rt, part = tid % rt;
    const bool on = e < E && L.key[e] != kNotLeft;
    int before = on ? ranked_before(L.key, part, E, rt, e) : 0;
    for (int o = 1; o < rt; o <<= 1) before += __shfl_xor(before, o);
    if (on && part == 0 && before < k) {
        ids[before] = e;
        L.sel[before] = L.scores[e];
        L.sel_logit[before] = L.logits[e];
    }
    __syncthreads();
    if (tid < k) {
        double mine = L.sel[tid], sum = 1.0;
        if (r.renorm) {
            sum = 0.0;
            for (int j = 0; j < k; ++j) sum += L.sel[j];
            if (sum < kSmallScores) {  // uniform
                double most = -INFINITY;
                for (int j = 0; j < k; ++j) most = fmax(most, L.sel_logit[j]);
                mine = exp(L.sel_logit[tid] - most);
                sum = 0.0;
                for (int j = 0; j < k; ++j) sum += exp(L.sel_logit[j] - most);
            }
        }
        weights[tid] = (float)(mine / sum * (double)r.scale);
    }
}

__global__ __launch_bounds__(1024) void moe_scored_kernel(const uint16_t* __restrict__ X,
                                                          const uint16_t* __restrict__ R, int H, int E, int k,
                                                          RouteScored r, int32_t* __restrict__ ids,
                                                          float* __restrict__ weights) {
    __shared__ ScoredLds L;
    const int t = blockIdx.x;
    token_logits(X + (int64_t)t * H, R, H, E, L.logits);
    scored_token(L, E, k, r, ids + t * k, weights + t * k);
}

__global__ __launch_bounds__(1024) void moe_scored_topk_kernel(const double* __restrict__ logits, int E, int k,
                                                               RouteScored r, int32_t* __restrict__ ids,
                                                               float* __restrict__ weights) {
    __shared__ ScoredLds L;
    const int t = blockIdx.x;
    for (int i = threadIdx.x; i < E; i += 1024) L.logits[i] = logits[(int64_t)t * E + i];
    __syncthreads();
    scored_token(L, E, k, r, ids + t * k, weights + t * k);
}

// ---------------------------------------------------------------- experts --
// The (token, choice) pairs grouped by expert: order lists the pairs of
// active expert a at [first[a], first[a + 1]); pairs whose id is outside
// [0, E) are left out. Over more than 64 pairs one workgroup makes it once
// for both kernels (in each of their workgroups its barriers cost about as
// much as the workgroup's loads); fewer take moe_find.
struct MoePlan {
    int n;                        // experts reached
    int expert[kMoeMaxPairs];     // ascending
    int first[kMoeMaxPairs + 1];
    int order[kMoeMaxPairs];      // sorted position -> pair
};

__global__ __launch_bounds__(512) void moe_plan_kernel(const int32_t* __restrict__ ids, int P, int E,
                                                       MoePlan* __restrict__ pl) {
    __shared__ int cnt[kMoeMaxExperts];
    __shared__ int wsum[2][8];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    static_assert(kMoeMaxExperts == 512 && kMoeMaxPairs == 512, "one expert and one pair a thread");
    const int id = tid < P ? ids[tid] : -1;
    cnt[tid] = 0;
    __syncthreads();
    const bool ok = id >= 0 && id < E;
    // the place of a pair inside its expert's run only says which column of
    // the products it rides in: the results do not depend on it
    const int at = ok ? atomicAdd(&cnt[id], 1) : 0;
    __syncthreads();
    const int c = cnt[tid];
    int s = c, a = c > 0;  // inclusive sums of pairs and of reached experts
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int ps = __shfl_up(s, o), pa = __shfl_up(a, o);
        if (lane >= o) {
            s += ps;
            a += pa;
        }
    }
    if (lane == 63) {
        wsum[0][wave] = s;
        wsum[1][wave] = a;
    }
    __syncthreads();
    for (int w = 0; w < wave; ++w) {
        s += wsum[0][w];
        a += wsum[1][w];
    }
    if (c > 0) {
        pl->expert[a - 1] = tid;
        pl->first[a - 1] = s - c;
    }
    if (tid == 511) {
        pl->n = a;
        pl->first[a] = s;
    }
    __syncthreads();
    cnt[tid] = s - c;  // first sorted position of expert tid
    __syncthreads();
    if (ok) pl->order[cnt[id] + at] = tid;
}

// Active expert z of at most 64 pairs, in the order of first mention, found by
// every wave for itself with no barrier: its pairs as a lane mask (pair =
// lane), each wave's list of them in its own part of LDS.
constexpr int kMoeWavePairs = 64;
struct MoeRun {
    int e, n;          // expert (or -1: fewer than z + 1 are reached), its pairs
    const int* order;  // their indices
};
__device__ __forceinline__ MoeRun moe_find(const int32_t* __restrict__ ids, int P, int E, int z, int* list, int lane) {
    const int id = lane < P ? ids[lane] : -1;
    const bool ok = id >= 0 && id < E;
    uint64_t left = __ballot(ok);
    MoeRun r{-1, 0, list};
    for (int c = 0; left; ++c) {
        const int ex = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        const uint64_t mine = __ballot(ok && id == ex);
        if (c == z) {
            r.e = ex;
            r.n = __popcll(mine);
            if ((mine >> lane) & 1) list[__popcll(mine & ((1ull << lane) - 1))] = lane;
            break;
        }
        left &= ~mine;
    }
    // the list is read by other lanes than the ones that wrote it (and through
    // a generic pointer): the writes have landed before any of them
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
    __builtin_amdgcn_wave_barrier();
    return r;
}

// The run of pairs a workgroup of the experts' kernels works on. lists: LDS,
// kMoeWavePairs per wave.
__device__ __forceinline__ MoeRun moe_run(const MoeArgs& a, const MoePlan* __restrict__ pl, int z, int* lists,
                                          int lane, int wave) {
    if (a.T * a.k <= kMoeWavePairs) return moe_find(a.ids, a.T * a.k, a.E, z, lists + wave * kMoeWavePairs, lane);
    if (z >= pl->n) return MoeRun{-1, 0, nullptr};
    const int lo = pl->first[z];
    return MoeRun{pl->expert[z], pl->first[z + 1] - lo, pl->order + lo};
}

// A tile's products go in steps: 128 k (4-bit, 2 a tile of 256 k) or 32 k
// (bf16, 4 a tile of 128 k), for each of which a lane holds kPieces pieces of
// the 16-bit operand.
template <bool MX>
constexpr int kTileK = MX ? 256 : 128;
template <bool MX>
constexpr int kSteps = MX ? 2 : 4;
template <bool MX>
constexpr int kPieces = MX ? 4 : 1;

// RB 16-row blocks of one expert's matrix from row r0 on, read through buffer
// resources: per-lane row offsets, the k of a tile in the uniform offset, which
// is not checked against the resource's end. So a row that ends inside a tile
// (TAIL, chosen on the host) has 4-bit codes addressed by the per-lane offset
// alone: past a row's end they are the next row's, and zeros past the last one;
// any code under the zero scale bytes there is finite, and meets zeros of x.
// 16-bit values past a row's end are not read: the next row's may be infinite.
// (Codes by the per-lane offset on every call: gate_up 59 against 51 us at 32
// tokens of 4 of 32 experts, 4096 x 1792.)
template <bool MX, int RB>
struct WRows {
    brsrc data, scales;
    uint32_t off[RB], soff;
    int bytes;  // of a row
};
template <bool MX, int RB>
__device__ __forceinline__ WRows<MX, RB> rows_of(const MoeWeights& W, int e, int N, int K, int r0, int lane) {
    const int fr = lane & 15, fc = lane >> 4;
    const int64_t rb = MX ? mx4_row_bytes(K) : (int64_t)K * 2, kts = mx4_k_tiles(K);
    const int64_t sb = mx4_scale_bytes(N, K);
    WRows<MX, RB> r;
    r.data = make_rsrc(static_cast<const uint8_t*>(W.data) + (int64_t)e * N * rb, (uint32_t)(N * rb));
    r.scales = make_rsrc(MX ? W.scales + (int64_t)e * sb : nullptr, MX ? (uint32_t)sb : 0u);
    r.bytes = (int)rb;
    r.soff = (uint32_t)((r0 >> 6) * kts * kMxTileBytes) + lane * 8;
#pragma unroll
    for (int j = 0; j < RB; ++j) r.off[j] = (uint32_t)(min(r0 + 16 * j + fr, N - 1) * rb) + fc * 16;
    return r;
}

// A tile of those rows, as a wave holds it: a 16-byte piece per row, step and lane.
template <bool MX, int RB>
struct WTile {
    u32x4 w[RB][kSteps<MX>];
    u32x2 sc;  // 4-bit: scale words of the tile's 64-row group
};
template <bool TAIL, bool MX, int RB>
__device__ __forceinline__ void load_wtile(WTile<MX, RB>& t, const WRows<MX, RB>& r, int kt, int lane) {
    constexpr int TB = kTileK<MX> * (MX ? 1 : 4) / 2;  // bytes of a row in a tile
    if constexpr (MX)
        t.sc = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r.scales, r.soff, kt * kMxTileBytes, 0));
    auto pieces = [&](auto end) {
#pragma unroll
        for (int s = 0; s < kSteps<MX>; ++s) {
            const int at = kt * TB + s * 64;
#pragma unroll
            for (int j = 0; j < RB; ++j) {
                uint32_t off = r.off[j];
                if constexpr (decltype(end)::value)
                    off = MX ? off + at : at + (lane >> 4) * 16 < r.bytes ? off + at : kOutOfRange;
                // the minimum never takes effect; without it register reuse puts a
                // wait between a tile's loads (gate_up 54.6 against 51.5 us, as above)
                t.w[j][s] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                          r.data, off, decltype(end)::value ? 0 : min(at, r.bytes), 0));
            }
        }
    };
    // 16-bit values: the last, partial tile apart (uniform); the checks on every
    // tile take 1 us of gate_up's 14 at 7 tokens of 2 of 8 experts, 2056 x 1000
    if (TAIL && (MX || (kt + 1) * TB > r.bytes)) pieces(std::true_type{});
    else pieces(std::false_type{});
}

// acc[c][j] += (16-row block j of the tile) (x[c][0] + x[c][1] + ..)^T over
// step i for NC column tiles of NX operands each, every decoded weight used
// for all of them. j0: the tile's first 16-row block in its group of four.
template <bool MX, int RB, int NC, int NX>
__device__ __forceinline__ void mac_wtile(f32x4 (&acc)[NC][RB], const WTile<MX, RB>& t, int j0, int i,
                                          const u32x4 (&x)[NC][NX][kPieces<MX>]) {
    if constexpr (MX) {
        float sc[RB];
#pragma unroll
        for (int j = 0; j < RB; ++j) sc[j] = mx4_scale(t.sc[i] >> (8 * (j0 + j)) & 255);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
#pragma unroll
            for (int j = 0; j < RB; ++j) {
                const u32x4 wf = mx4_bf16x8(t.w[j][i][m], sc[j]);
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int n = 0; n < NX; ++n) acc[c][j] = mfma16x16x32(wf, x[c][n][m], acc[c][j]);
            }
            __builtin_amdgcn_sched_barrier(0);  // one piece's decoded weights at a time
        }
    } else {
#pragma unroll
        for (int j = 0; j < RB; ++j)
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int n = 0; n < NX; ++n) acc[c][j] = mfma16x16x32(t.w[j][i], x[c][n][0], acc[c][j]);
    }
}

// One lane's row of 16-bit values at tile kt and step i as mac_wtile takes it.
// off: byte offset of the row's first value in x (kOutOfRange: zeros); K:
// values in the row; PERM: stored in the 4-bit side's order (moe_at).
template <bool MX, bool PERM>
__device__ __forceinline__ void load_x(brsrc x, uint32_t off, int K, int kt, int i, int lane,
                                       u32x4 (&v)[kPieces<MX>]) {
    const int fc = lane >> 4, k0 = kt * kTileK<MX> + i * (MX ? 128 : 32);
#pragma unroll
    for (int m = 0; m < kPieces<MX>; ++m) {
        const int k = PERM && MX ? 32 * fc + 8 * m : 32 * m + 8 * fc;
        // the uniform offset stays inside the rows: stored rows (PERM) are
        // whole 128-value groups and come in pairs, others end at K
        const int at = PERM ? k0 * 2 + m * 64 : min(k0 + 32 * m, K) * 2;
        v[m] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                             x, k0 + k < K ? off + fc * 16 : kOutOfRange, at, 0));
    }
    if constexpr (MX && !PERM) mx4_transpose(v);
}

// The inner values of a pair: rows of whole 128-value groups, hi then lo;
// written up to a whole block, zeros behind I. Beside 4-bit weights a group
// is stored [8 k piece][block] instead of [block][8 k piece], so that the
// down kernel's loads are consecutive without a transpose.
__host__ __device__ inline int moe_inner(int I) { return (I + 31) & ~31; }
__host__ __device__ inline int moe_act_row(int I) { return (I + 127) & ~127; }
template <bool MX>
__device__ __forceinline__ int moe_at(int i) {
    return MX ? (i & ~127) | (i >> 3 & 3) << 5 | (i >> 5 & 3) << 3 | (i & 7) : i;
}

// Workgroup (inner columns 32 bx .. + 31, active expert by): gate and up rows
// over all of H, the k tiles dealt round the waves and their sums added in
// wave order; then silu(g) * u, kept as bf16 hi + lo (two products in the
// down kernel, which waits on memory: the inner values keep 16 bits of
// mantissa instead of 8) in act[pair][2][moe_act_row(I)]. A pass takes 16 or,
// where more are left, 32 of the expert's pairs.
template <bool MX, bool TAIL, int NW>
__global__ __launch_bounds__(64 * NW, 4) void moe_gate_up_kernel(MoeArgs a, const MoePlan* __restrict__ pl,
                                                                 uint16_t* __restrict__ act) {
    static_assert(NW == 8, "a thread per element of a row block pair");
    __shared__ int lists[NW * kMoeWavePairs];
    __shared__ f32x4 red[NW][4][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const MoeRun run = moe_run(a, pl, blockIdx.y, lists, lane, wave);
    if (run.e < 0) return;  // uniform for the workgroup
    const int e = run.e, hi = run.n;
    const int r0 = blockIdx.x * 32, kts = (a.H + kTileK<MX> - 1) / kTileK<MX>, Ir = moe_act_row(a.I);
    const auto rg = rows_of<MX, 2>(a.gate, e, a.I, a.H, r0, lane), ru = rows_of<MX, 2>(a.up, e, a.I, a.H, r0, lane);
    const brsrc rx = make_rsrc(a.X, (uint32_t)a.T * (uint32_t)a.H * 2u);
    auto pass = [&](int t0, auto nc) {
        constexpr int NC = decltype(nc)::value;
        uint32_t xo[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int p = t0 + 16 * c + (lane & 15);
            xo[c] = p < hi ? (uint32_t)(run.order[p] / a.k) * (uint32_t)a.H * 2u : kOutOfRange;
        }
        f32x4 g[NC][2], u[NC][2];
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 2; ++j) g[c][j] = u[c][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int kt = wave; kt < kts; kt += NW) {
            WTile<MX, 2> wg, wu;
            load_wtile<TAIL>(wg, rg, kt, lane);
            load_wtile<TAIL>(wu, ru, kt, lane);
#pragma unroll
            for (int i = 0; i < kSteps<MX>; ++i) {
                u32x4 x[NC][1][kPieces<MX>];
#pragma unroll
                for (int c = 0; c < NC; ++c) load_x<MX, false>(rx, xo[c], a.H, kt, i, lane, x[c][0]);
                mac_wtile(g, wg, r0 >> 4 & 3, i, x);
                mac_wtile(u, wu, r0 >> 4 & 3, i, x);
            }
        }
#pragma unroll
        for (int cc = 0; cc < NC; ++cc) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                red[wave][j][lane] = g[cc][j];
                red[wave][2 + j][lane] = u[cc][j];
            }
            __syncthreads();
            // thread (j, l, c): element c of lane l's result in row block j
            const int j = tid >> 8, l = tid >> 2 & 63, c = tid & 3;
            float gs = 0.f, us = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                gs += red[w][j][l][c];
                us += red[w][2 + j][l][c];
            }
            const int q = t0 + 16 * cc + (l & 15), i = r0 + 16 * j + 4 * (l >> 4) + c;
            if (q < hi && i < moe_inner(a.I)) {
                const float v = i < a.I ? gs / (1.f + expf(-gs)) * us : 0.f;
                uint16_t* ap = act + (int64_t)run.order[q] * 2 * Ir + moe_at<MX>(i);
                const uint16_t h = bf16_hi(v);
                ap[0] = h;
                ap[Ir] = f32_to_bf16(v - bf16_to_f32(h));
            }
        }
    };
    int t0 = 0;
    for (; hi - t0 > 16; t0 += 32) pass(t0, std::integral_constant<int, 2>{});
    if (t0 < hi) pass(t0, std::integral_constant<int, 1>{});
}

// Workgroup (output columns 64 bx .. + 63, active expert by): the down
// product of the expert's pairs, k tiles dealt round the waves, sums in wave
// order, into o[pair][H] in fp32; every pair has one expert, so each element
// is written once.
template <bool MX, bool TAIL, int NW>
__global__ __launch_bounds__(64 * NW, NW == 8 ? 2 : 3) void moe_down_kernel(MoeArgs a, const MoePlan* __restrict__ pl,
                                                              const uint16_t* __restrict__ act,
                                                              float* __restrict__ o) {
    __shared__ int lists[NW * kMoeWavePairs];
    __shared__ f32x4 red[NW][4][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const MoeRun run = moe_run(a, pl, blockIdx.y, lists, lane, wave);
    if (run.e < 0) return;  // uniform for the workgroup
    const int e = run.e, hi = run.n;
    const int r0 = blockIdx.x * 64, kts = (a.I + kTileK<MX> - 1) / kTileK<MX>;
    const int Ip = moe_inner(a.I), Ir = moe_act_row(a.I);
    const auto rd = rows_of<MX, 4>(a.down, e, a.H, a.I, r0, lane);
    const brsrc rx = make_rsrc(act, (uint32_t)(a.T * a.k) * 4u * (uint32_t)Ir);
    auto pass = [&](int t0, auto nc) {
        constexpr int NC = decltype(nc)::value;
        uint32_t ao[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int p = t0 + 16 * c + (lane & 15);
            ao[c] = p < hi ? (uint32_t)run.order[p] * 4u * (uint32_t)Ir : kOutOfRange;
        }
        f32x4 acc[NC][4];
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[c][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int kt = wave; kt < kts; kt += NW) {
            WTile<MX, 4> w;
            load_wtile<TAIL>(w, rd, kt, lane);
            if constexpr (MX && NC == 1) {
                // the inner values of both steps asked for with the codes, one
                // round of memory: 34 against 38 us at 32 tokens of 4 of 32
                // experts, 1792 -> 4096 (two column tiles of them would spill)
                u32x4 x[2][1][2][kPieces<MX>];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    load_x<MX, true>(rx, ao[0], Ip, kt, i, lane, x[i][0][0]);
                    load_x<MX, true>(rx, ao[0] + 2u * (uint32_t)Ir, Ip, kt, i, lane, x[i][0][1]);
                }
                issue_fence();
                mac_wtile(acc, w, 0, 0, x[0]);
                mac_wtile(acc, w, 0, 1, x[1]);
                continue;
            }
#pragma unroll
            for (int i = 0; i < kSteps<MX>; ++i) {
                u32x4 x[NC][2][kPieces<MX>];
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    load_x<MX, true>(rx, ao[c], Ip, kt, i, lane, x[c][0]);
                    load_x<MX, true>(rx, ao[c] + 2u * (uint32_t)Ir, Ip, kt, i, lane, x[c][1]);
                }
                mac_wtile(acc, w, 0, i, x);
            }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 4; ++j) red[wave][j][lane] = acc[c][j];
            __syncthreads();
            // thread (j, l) adds the waves' sums of lane l in row block j
            for (int task = tid; task < 256; task += 64 * NW) {
                const int j = task >> 6, l = task & 63;
                f32x4 s = red[0][j][l];
#pragma unroll
                for (int w = 1; w < NW; ++w) s += red[w][j][l];
                const int q = t0 + 16 * c + (l & 15), n = r0 + 16 * j + 4 * (l >> 4);
                if (q < hi && n < a.H)  // H is a multiple of 8
                    *reinterpret_cast<f32x4*>(o + (int64_t)run.order[q] * a.H + n) = s;
            }
        }
    };
    int t0 = 0;
    for (; hi - t0 > 16; t0 += 32) pass(t0, std::integral_constant<int, 2>{});
    if (t0 < hi) pass(t0, std::integral_constant<int, 1>{});
}

// y[t] = sum_j w[t][j] o[t k + j], in the order of j; 4 columns a thread
__global__ __launch_bounds__(256) void moe_combine_kernel(MoeArgs a, const float* __restrict__ o) {
    const int t = blockIdx.y, n = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (n >= a.H) return;
    f32x4 y{0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < a.k; j0 += 4) {
        f32x4 v[4];
        float w[4];
        bool ok[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // all loads first; choices past k or without an expert are not added
            const int64_t p = (int64_t)t * a.k + min(j0 + j, a.k - 1);
            const int id = a.ids[p];
            ok[j] = j0 + j < a.k && id >= 0 && id < a.E;
            w[j] = a.weights[p];
            v[j] = *reinterpret_cast<const f32x4*>(o + p * a.H + n);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (ok[j]) y += w[j] * v[j];
    }
    const u32x2 r{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
    *reinterpret_cast<u32x2*>(a.Y + (int64_t)t * a.H + n) = r;
}

// Both forms sum a logit in the same order, so they choose alike.
constexpr int64_t kMoeRouteOne = 1 << 16;  // router values one workgroup reads: 128 KB

size_t moe_route_workspace(int T, int H, int E) {
    return (int64_t)E * H <= kMoeRouteOne ? 0 : (size_t)T * E * sizeof(double);
}

static hipError_t moe_logits(const uint16_t* X, const uint16_t* router, int T, int H, int E, double* logits,
                             hipStream_t st, StageTimer* tm) {
    // tiles of 4 x 4 where they still are two waves a CU, of 1 x 1 otherwise
    if ((int64_t)T * E >= 16 * 512)
        return launch(tm, "moe_logits", moe_logits_kernel<4, 4>, dim3((E + 15) / 16, (T + 3) / 4), dim3(256), st, X,
                      router, T, H, E, logits);
    return launch(tm, "moe_logits", moe_logits_kernel<1, 1>, dim3((E + 3) / 4, T), dim3(256), st, X, router, T, H, E,
                  logits);
}

hipError_t moe_route(const uint16_t* X, const uint16_t* router, int T, int H, int E, int k, int renorm, int32_t* ids,
                     float* weights, void* workspace, hipStream_t st, StageTimer* tm) {
    if ((int64_t)E * H <= kMoeRouteOne)
        return launch(tm, "moe_route", moe_route_kernel, dim3(T), dim3(1024), st, X, router, H, E, k, renorm, ids,
                      weights);
    double* logits = static_cast<double*>(workspace);
    hipError_t e = moe_logits(X, router, T, H, E, logits, st, tm);
    if (e != hipSuccess) return e;
    return launch(tm, "moe_topk", moe_topk_kernel, dim3(T), dim3(1024), st, (const double*)logits, E, k, renorm, ids,
                  weights);
}

hipError_t moe_route_scored(const uint16_t* X, const uint16_t* router, int T, int H, int E, int k,
                            const RouteScored& r, int32_t* ids, float* weights, void* workspace, hipStream_t st,
                            StageTimer* tm) {
    if ((int64_t)E * H <= kMoeRouteOne)
        return launch(tm, "moe_scored", moe_scored_kernel, dim3(T), dim3(1024), st, X, router, H, E, k, r, ids,
                      weights);
    double* logits = static_cast<double*>(workspace);
    hipError_t e = moe_logits(X, router, T, H, E, logits, st, tm);
    if (e != hipSuccess) return e;
    return launch(tm, "moe_scored_topk", moe_scored_topk_kernel, dim3(T), dim3(1024), st, (const double*)logits, E, k,
                  r, ids, weights);
}

// the inner values of every pair, its down products, then the plan
static size_t align256(size_t n) { return (n + 255) & ~size_t(255); }
static size_t moe_act_bytes(int T, int I, int k) {
    return align256((size_t)T * k * 2 * moe_act_row(I) * sizeof(uint16_t));
}
size_t moe_experts_workspace(int T, int H, int I, int k) {
    return moe_act_bytes(T, I, k) + align256((size_t)T * k * H * sizeof(float)) + align256(sizeof(MoePlan));
}

template <bool MX>
static hipError_t experts(const MoeArgs& a, hipStream_t st, StageTimer* tm) {
    // waves of a workgroup: gate_up 8 (128 registers, 2 workgroups a CU), down 4
    // (168 registers, 3 a CU) or, where that leaves a CU one workgroup at most,
    // 8: at 32 tokens of 4 of 32 experts, 4096 x 1792, gate_up takes 54 us
    // against 58 with 4, down 34 against 45 with 8; at one token 7 us with 8
    // against 8
    constexpr int NW = 8;
    const int P = a.T * a.k, reached = P < a.E ? P : a.E;  // experts at most
    char* ws = static_cast<char*>(a.workspace);
    uint16_t* act = reinterpret_cast<uint16_t*>(ws);
    float* o = reinterpret_cast<float*>(ws + moe_act_bytes(a.T, a.I, a.k));
    MoePlan* pl = reinterpret_cast<MoePlan*>(reinterpret_cast<char*>(o) + align256((size_t)P * a.H * sizeof(float)));
    hipError_t e = hipSuccess;
    if (P > kMoeWavePairs) e = launch(tm, "moe_plan", moe_plan_kernel, dim3(1), dim3(512), st, a.ids, P, a.E, pl);
    const bool tail_h = a.H % kTileK<MX> != 0, tail_i = a.I % kTileK<MX> != 0;
    if (e == hipSuccess)
        e = launch(tm, "moe_gate_up", tail_h ? moe_gate_up_kernel<MX, true, NW> : moe_gate_up_kernel<MX, false, NW>,
                   dim3(moe_inner(a.I) / 32, reached), dim3(64 * NW), st, a, (const MoePlan*)pl, act);
    const dim3 down((a.H + 63) / 64, reached);
    const bool few = down.x * down.y <= 256;
    auto ker = few ? (tail_i ? moe_down_kernel<MX, true, 8> : moe_down_kernel<MX, false, 8>)
                   : (tail_i ? moe_down_kernel<MX, true, 4> : moe_down_kernel<MX, false, 4>);
    if (e == hipSuccess)
        e = launch(tm, "moe_down", ker, down, dim3(few ? 512 : 256), st, a, (const MoePlan*)pl, (const uint16_t*)act,
                   o);
    if (e == hipSuccess)
        e = launch(tm, "moe_combine", moe_combine_kernel, dim3((a.H / 4 + 255) / 256, a.T), dim3(256), st, a,
                   (const float*)o);
    return e;
}

hipError_t moe_experts(const MoeArgs& a, bool mx4, hipStream_t st, StageTimer* tm) {
    return mx4 ? experts<true>(a, st, tm) : experts<false>(a, st, tm);
}

}  // namespace lora
