// A mixture-of-experts layer for a few tokens:
//   logits = x R^T;  ids, w = the k largest of each token and their softmax;
//   y[t] = sum_j w[t][j] down_e( silu(gate_e x_t) * up_e x_t ),  e = ids[t][j]
// with the experts' weights in bf16 or MXFP4. With few tokens the layer is
// bound by the weights of the experts that are reached: each is read once,
// in 16-byte pieces, for all of its tokens, which ride as the 16 columns of
// the matrix-core products (weights are the left operand).
//
// Route: one wave per (expert, token) sums the logit in 64 bits, so that the
// choice among close logits does not hang on the rounding of a sum; one wave
// per token then takes the k largest.
// Experts: two kernels. gate_up: a workgroup takes one reached expert and 32
// inner columns (32 gate and 32 up rows); down: a workgroup takes 16 output
// columns and goes through every reached expert, so that a token's k terms
// meet in one workgroup and are added in the order of j.
#include "kernels.h"
#include "mx4.h"

namespace lora {

// ------------------------------------------------------------------ route --
// A lane's part of the 64-bit dot product of two bf16 rows.
__device__ __forceinline__ double dot_rows(const uint16_t* __restrict__ xp, const uint16_t* __restrict__ rp, int H,
                                           int lane) {
    double s[2] = {0.0, 0.0};
#pragma unroll 4
    for (int k = lane * 8; k < H; k += 512) {
        const u32x4 a = *as_global<u32x4>(xp + k), b = *as_global<u32x4>(rp + k);
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // a product of two bf16 is exact in fp32
            s[0] += (double)(__uint_as_float(a[i] << 16) * __uint_as_float(b[i] << 16));
            s[1] += (double)(__uint_as_float(a[i] & 0xffff0000u) * __uint_as_float(b[i] & 0xffff0000u));
        }
    }
    return s[0] + s[1];
}

// One wave, lane l holding logits l, l + 64, ...: k rounds of a maximum over
// the wave, equal logits to the lower index. A NaN counts as the lowest of
// all, so the ids stay valid and distinct; its weights are NaN.
constexpr int kMoePerLane = kMoeMaxExperts / 64;
__device__ __forceinline__ void topk_token(const double* logits, int E, int k, int renorm, int32_t* ids,
                                           float* weights, int lane) {
    double v[kMoePerLane];
    uint32_t taken = 0;
#pragma unroll
    for (int i = 0; i < kMoePerLane; ++i) v[i] = i * 64 + lane < E ? logits[i * 64 + lane] : 0.0;
    double top = 0.0, mine = 0.0;  // the largest logit; the one chosen in round `lane`
    int id = 0;
    for (int j = 0; j < k; ++j) {
        double best = 0.0;
        int at = -1;
#pragma unroll
        for (int i = 0; i < kMoePerLane; ++i) {
            if (i * 64 + lane >= E || (taken >> i & 1)) continue;
            if (at < 0 || v[i] > best || (best != best && v[i] == v[i])) {
                best = v[i];
                at = i * 64 + lane;
            }
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const double ov = __shfl_xor(best, o);
            const int oa = __shfl_xor(at, o);
            const bool bn = best != best, on = ov != ov;
            bool take;
            if (oa < 0 || at < 0) take = at < 0;
            else if (bn != on) take = bn;
            else if (bn || ov == best) take = oa < at;
            else take = ov > best;
            if (take) {
                best = ov;
                at = oa;
            }
        }
        if ((at & 63) == lane) taken |= 1u << (at >> 6);
        if (j == 0) top = best;
        if (j == lane) {
            mine = best;
            id = at;
        }
    }
    // weights: exp(l_j - max) over the sum of the chosen (renorm) or of all
    const float p = lane < k ? expf((float)(mine - top)) : 0.f;
    float den = p;
    if (!renorm) {
        den = 0.f;
#pragma unroll
        for (int i = 0; i < kMoePerLane; ++i)
            if (i * 64 + lane < E) den += expf((float)(v[i] - top));
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) den += __shfl_xor(den, o);
    if (lane < k) {
        ids[lane] = id;
        weights[lane] = p / den;
    }
}

// One workgroup per token: its 16 waves take the experts in turn, the first
// wave then the k largest of the logits in LDS.
__global__ __launch_bounds__(1024) void moe_route_kernel(const uint16_t* __restrict__ X,
                                                         const uint16_t* __restrict__ R, int H, int E, int k,
                                                         int renorm, int32_t* __restrict__ ids,
                                                         float* __restrict__ weights) {
    __shared__ double logits[kMoeMaxExperts];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = blockIdx.x;
    for (int e = wave; e < E; e += 16) {
        double s = dot_rows(X + (int64_t)t * H, R + (int64_t)e * H, H, lane);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
        if (lane == 0) logits[e] = s;
    }
    __syncthreads();
    if (wave == 0) topk_token(logits, E, k, renorm, ids + t * k, weights + t * k, lane);
}

// The same over two launches, one wave per (expert, token) and then one per
// token: a router too large for one CU to read quickly, and few tokens.
__global__ __launch_bounds__(256) void moe_logits_kernel(const uint16_t* __restrict__ X,
                                                         const uint16_t* __restrict__ R, int H, int E,
                                                         double* __restrict__ logits) {
    const int lane = threadIdx.x & 63, e = blockIdx.x * 4 + (threadIdx.x >> 6), t = blockIdx.y;
    if (e >= E) return;
    double s = dot_rows(X + (int64_t)t * H, R + (int64_t)e * H, H, lane);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    if (lane == 0) logits[(int64_t)t * E + e] = s;
}

__global__ __launch_bounds__(64) void moe_topk_kernel(const double* __restrict__ logits, int E, int k, int renorm,
                                                      int32_t* __restrict__ ids, float* __restrict__ weights) {
    const int t = blockIdx.x;
    topk_token(logits + (int64_t)t * E, E, k, renorm, ids + t * k, weights + t * k, threadIdx.x);
}

// ---------------------------------------------------------------- experts --
// The (token, choice) pairs grouped by expert: order lists the pairs of
// active expert a at [first[a], first[a + 1]); pairs whose id is outside
// [0, E) are left out. Every workgroup builds it in LDS from the ids.
constexpr int kMoePlanThreads = 512;
struct MoePlan {
    int n;                         // experts reached
    int expert[kMoeMaxPairs];      // ascending
    int first[kMoeMaxPairs + 1];
    int16_t order[kMoeMaxPairs];   // sorted position -> pair
    int16_t pos[kMoeMaxPairs];     // pair -> sorted position, or -1
    int cnt[kMoeMaxExperts];
    int wsum[2][kMoePlanThreads / 64];
};

__device__ __forceinline__ void moe_plan(const int32_t* __restrict__ ids, int P, int E, MoePlan& pl) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    static_assert(kMoeMaxExperts == kMoePlanThreads && kMoeMaxPairs == kMoePlanThreads,
                  "one expert and one pair a thread");
    const bool on = tid < kMoePlanThreads;
    const int id = tid < P ? ids[tid] : -1;
    if (on) pl.cnt[tid] = 0;
    __syncthreads();
    const bool ok = id >= 0 && id < E;
    // the place of a pair inside its expert's run only says which column of
    // the products it rides in: the results do not depend on it
    const int at = ok ? atomicAdd(&pl.cnt[id], 1) : 0;
    __syncthreads();
    const int c = on ? pl.cnt[tid] : 0;
    int s = c, a = c > 0;  // inclusive sums of pairs and of reached experts
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int ps = __shfl_up(s, o), pa = __shfl_up(a, o);
        if (lane >= o) {
            s += ps;
            a += pa;
        }
    }
    if (on && lane == 63) {
        pl.wsum[0][wave] = s;
        pl.wsum[1][wave] = a;
    }
    __syncthreads();
    if (on) {
        for (int w = 0; w < wave; ++w) {
            s += pl.wsum[0][w];
            a += pl.wsum[1][w];
        }
        if (c > 0) {
            pl.expert[a - 1] = tid;
            pl.first[a - 1] = s - c;
        }
        if (tid == kMoePlanThreads - 1) {
            pl.n = a;
            pl.first[a] = s;
        }
        pl.cnt[tid] = s - c;  // first sorted position of expert tid
    }
    __syncthreads();
    if (tid < P) pl.pos[tid] = ok ? (int16_t)(pl.cnt[id] + at) : (int16_t)-1;
    if (ok) pl.order[pl.cnt[id] + at] = (int16_t)tid;
    __syncthreads();
}

// 256 k of RB 16-row blocks of one expert's matrix, as a wave holds them: 2
// (4-bit) or 8 (bf16) 16-byte pieces per row and lane.
template <bool MX, int RB>
struct WTile {
    u32x4 w[RB][MX ? 2 : 8];
    u32x2 sc;  // 4-bit: scale words of the tile's 64-row group
};

// rows r0 .. r0 + 16 RB (clamped to N rows) of expert e at k tile kt
template <bool MX, int RB>
__device__ __forceinline__ void load_wtile(WTile<MX, RB>& t, const MoeWeights& W, int e, int N, int K, int r0, int kt,
                                           int lane) {
    const int fr = lane & 15, fc = lane >> 4;
    if constexpr (MX) {
        const int64_t rb = mx4_row_bytes(K), kts = mx4_k_tiles(K);
        const uint8_t* base = static_cast<const uint8_t*>(W.data) + (int64_t)e * N * rb;
        t.sc = *reinterpret_cast<const u32x2*>(W.scales + (int64_t)e * mx4_scale_bytes(N, K) +
                                               ((int64_t)(r0 >> 6) * kts + kt) * kMxTileBytes + lane * 8);
#pragma unroll
        for (int j = 0; j < RB; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int blk = kt * 8 + h * 4 + fc;
                t.w[j][h] = *or_zero(blk * 32 < K, base + (int64_t)min(r0 + 16 * j + fr, N - 1) * rb + blk * 16);
            }
    } else {
        const uint16_t* base = static_cast<const uint16_t*>(W.data) + (int64_t)e * N * K;
#pragma unroll
        for (int j = 0; j < RB; ++j)
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const int k = kt * 256 + 32 * s + 8 * fc;
                t.w[j][s] = *or_zero(k < K, base + (int64_t)min(r0 + 16 * j + fr, N - 1) * K + k);
            }
    }
}

// A tile's products go in steps: 128 k (4-bit, 2 a tile) or 32 k (bf16, 8), for
// each of which a lane holds kPieces pieces of the 16-bit operand.
template <bool MX>
constexpr int kSteps = MX ? 2 : 8;
template <bool MX>
constexpr int kPieces = MX ? 4 : 1;

// acc[j] += (16-row block j of the tile) (x)^T over step i. j0: the tile's
// first 16-row block in its group of four.
template <bool MX, int RB>
__device__ __forceinline__ void mac_wtile(f32x4 (&acc)[RB], const WTile<MX, RB>& t, int j0, int i,
                                          const u32x4 (&x)[kPieces<MX>]) {
    if constexpr (MX) {
        float sc[RB];
#pragma unroll
        for (int j = 0; j < RB; ++j) sc[j] = mx4_scale(t.sc[i] >> (8 * (j0 + j)) & 255);
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int j = 0; j < RB; ++j) acc[j] = mfma16x16x32(mx4_bf16x8(t.w[j][i][m], sc[j]), x[m], acc[j]);
    } else {
#pragma unroll
        for (int j = 0; j < RB; ++j) acc[j] = mfma16x16x32(t.w[j][i], x[0], acc[j]);
    }
}

// One lane's row of 16-bit values (null: zeros) at tile kt as mac_wtile takes
// it. K: values in the row; PERM: stored in the 4-bit side's order (moe_at).
template <bool MX, bool PERM>
__device__ __forceinline__ void load_x(const uint16_t* row, int K, int kt, int i, int lane, u32x4 (&v)[kPieces<MX>]) {
    const int fc = lane >> 4;
    if constexpr (MX) {
        const int k0 = kt * 256 + i * 128;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int k = PERM ? k0 + 32 * fc + 8 * m : k0 + 32 * m + 8 * fc;
            v[m] = *or_zero(row && k < K, row + k0 + 32 * m + 8 * fc);
        }
        if constexpr (!PERM) mx4_transpose(v);
    } else {
        const int k = kt * 256 + 32 * i + 8 * fc;
        v[0] = *or_zero(row && k < K, row + k);
    }
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
// mantissa instead of 8) in act[pair][2][moe_act_row(I)].
template <bool MX, int NW>
__global__ __launch_bounds__(64 * NW) void moe_gate_up_kernel(MoeArgs a, uint16_t* __restrict__ act) {
    __shared__ MoePlan pl;
    __shared__ f32x4 red[NW][4][64];
    const int P = a.T * a.k;
    moe_plan(a.ids, P, a.E, pl);
    if ((int)blockIdx.y >= pl.n) return;
    const int e = pl.expert[blockIdx.y], lo = pl.first[blockIdx.y], hi = pl.first[blockIdx.y + 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int r0 = blockIdx.x * 32, kts = (a.H + 255) / 256, Ir = moe_act_row(a.I);
    for (int t0 = lo; t0 < hi; t0 += 16) {
        const int p = t0 + (lane & 15);
        const uint16_t* xr = p < hi ? a.X + (int64_t)(pl.order[p] / a.k) * a.H : nullptr;
        f32x4 g[2], u[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) g[j] = u[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int kt = wave; kt < kts; kt += NW) {
            WTile<MX, 2> wg, wu;
            load_wtile(wg, a.gate, e, a.I, a.H, r0, kt, lane);
            load_wtile(wu, a.up, e, a.I, a.H, r0, kt, lane);
#pragma unroll
            for (int i = 0; i < kSteps<MX>; ++i) {
                u32x4 x[kPieces<MX>];
                load_x<MX, false>(xr, a.H, kt, i, lane, x);
                mac_wtile(g, wg, r0 >> 4 & 3, i, x);
                mac_wtile(u, wu, r0 >> 4 & 3, i, x);
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            red[wave][j][lane] = g[j];
            red[wave][2 + j][lane] = u[j];
        }
        __syncthreads();
        // thread (j, l, c): element c of lane l's result in row block j
        const int j = tid >> 8 & 1, l = tid >> 2 & 63, c = tid & 3;
        if (tid >= 512) continue;  // uniform for a wave; the next barrier is met by all
        float gs = 0.f, us = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            gs += red[w][j][l][c];
            us += red[w][2 + j][l][c];
        }
        const int q = t0 + (l & 15), i = r0 + 16 * j + 4 * (l >> 4) + c;
        if (q < hi && i < moe_inner(a.I)) {
            const float v = i < a.I ? gs / (1.f + expf(-gs)) * us : 0.f;
            uint16_t* ap = act + (int64_t)pl.order[q] * 2 * Ir + moe_at<MX>(i);
            const uint16_t h = f32_to_bf16(v);
            ap[0] = h;
            // an infinite or NaN value has no remainder
            const float rest = v - bf16_to_f32(h);
            ap[Ir] = rest == rest ? f32_to_bf16(rest) : uint16_t(0);
        }
    }
}

// Workgroup: output columns 16 bx .. + 15 of every pair. Work items (active
// expert, up to 32 of its pairs, k tiles of class kc mod KC) go round the
// waves; an item's results land in o[kc][pair position][column], each written
// once, and are added in the order of kc and then of j. A wave's tiles form
// one sequence over all its items, the next tile's weights in flight while
// the current one is multiplied.
constexpr int kMoeOutFloats = kMoeMaxPairs * 16;  // 32 KB
template <bool MX, int NW>
__global__ __launch_bounds__(64 * NW) void moe_down_kernel(MoeArgs a, const uint16_t* __restrict__ act, int KC) {
    __shared__ MoePlan pl;
    __shared__ float o[kMoeOutFloats];
    const int P = a.T * a.k;
    moe_plan(a.ids, P, a.E, pl);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r0 = blockIdx.x * 16, kts = (a.I + 255) / 256, Ip = moe_inner(a.I), Ir = moe_act_row(a.I);
    const int n_items = pl.n * KC;
    int it = wave, kt = 0, t0 = 0;  // the tile in hand: item, k tile, first pair of the pass
    auto locate = [&](int item) {
        kt = item % KC;
        t0 = pl.first[min(item, n_items - 1) / KC];
    };
    WTile<MX, 1> w;
    auto fetch = [&](WTile<MX, 1>& t, int item, int k_tile) {
        load_wtile(t, a.down, pl.expert[item / KC], a.H, a.I, r0, k_tile, lane);
    };
    if (it < n_items) {
        locate(it);
        fetch(w, it, kt);
    }
    f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
    while (it < n_items) {
        const int ai = it / KC, kc = it - ai * KC, hi = pl.first[ai + 1], ck = kt, ct = t0;
        // the tile after this one: along K, then the item's next pairs, then the next item
        bool last = false;  // this tile ends its pass
        kt += KC;
        if (kt >= kts) {
            last = true;
            t0 += 32;
            if (t0 < hi) {
                kt = kc;
            } else {
                it += NW;
                locate(it);
            }
        }
        WTile<MX, 1> next;
        if (it < n_items) fetch(next, it, kt);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (ct + 16 * i >= hi) break;  // uniform
            const int p = ct + 16 * i + (lane & 15);
            const uint16_t* ar = p < hi ? act + (int64_t)pl.order[p] * 2 * Ir : nullptr;
            f32x4 c[1] = {acc[i]};
#pragma unroll
            for (int q = 0; q < kSteps<MX>; ++q) {
                u32x4 hi16[kPieces<MX>], lo16[kPieces<MX>];
                load_x<MX, true>(ar, Ip, ck, q, lane, hi16);
                load_x<MX, true>(ar ? ar + Ir : nullptr, Ip, ck, q, lane, lo16);
                mac_wtile(c, w, r0 >> 4 & 3, q, hi16);
                mac_wtile(c, w, r0 >> 4 & 3, q, lo16);
            }
            acc[i] = c[0];
            if (last) {
                if (p < hi) *reinterpret_cast<f32x4*>(&o[(kc * P + p) * 16 + 4 * (lane >> 4)]) = acc[i];
                acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
        }
        w = next;
    }
    __syncthreads();
    for (int i = tid; i < a.T * 16; i += 64 * NW) {
        const int t = i >> 4, n = i & 15;
        if (r0 + n >= a.H) continue;
        float y = 0.f;
        for (int j = 0; j < a.k; ++j) {
            const int p = pl.pos[t * a.k + j];
            if (p < 0) continue;
            float v = 0.f;
            for (int kc = 0; kc < KC; ++kc) v += o[(kc * P + p) * 16 + n];
            y += a.weights[t * a.k + j] * v;
        }
        a.Y[(int64_t)t * a.H + r0 + n] = f32_to_bf16(y);
    }
}

// Both forms sum a logit in the same order, so they choose alike.
constexpr int64_t kMoeRouteOne = 1 << 16;  // router values one workgroup reads: 128 KB

size_t moe_route_workspace(int T, int E) { return (size_t)T * E * sizeof(double); }

hipError_t moe_route(const uint16_t* X, const uint16_t* router, int T, int H, int E, int k, int renorm, int32_t* ids,
                     float* weights, void* workspace, hipStream_t st, StageTimer* tm) {
    if ((int64_t)E * H <= kMoeRouteOne)
        return launch(tm, "moe_route", moe_route_kernel, dim3(T), dim3(1024), st, X, router, H, E, k, renorm, ids,
                      weights);
    double* logits = static_cast<double*>(workspace);
    hipError_t e = launch(tm, "moe_logits", moe_logits_kernel, dim3((E + 3) / 4, T), dim3(256), st, X, router, H, E,
                          logits);
    if (e != hipSuccess) return e;
    return launch(tm, "moe_topk", moe_topk_kernel, dim3(T), dim3(64), st, (const double*)logits, E, k, renorm, ids,
                  weights);
}

size_t moe_experts_workspace(int T, int I, int k) { return (size_t)T * k * 2 * moe_act_row(I) * sizeof(uint16_t); }

template <bool MX>
static hipError_t experts(const MoeArgs& a, hipStream_t st, StageTimer* tm) {
    constexpr int NG = 8, ND = 16;  // waves of a workgroup
    uint16_t* act = static_cast<uint16_t*>(a.workspace);
    const int P = a.T * a.k, kts = (a.I + 255) / 256;
    hipError_t e = launch(tm, "moe_gate_up", moe_gate_up_kernel<MX, NG>,
                          dim3(moe_inner(a.I) / 32, P < a.E ? P : a.E), dim3(64 * NG), st, a, act);
    if (e != hipSuccess) return e;
    // k classes per expert: as many as the planes of results hold and the
    // tiles of K fill, 8 at most
    int KC = kMoeOutFloats / (16 * P);
    KC = KC < 8 ? KC : 8;
    KC = KC < kts ? KC : kts;
    return launch(tm, "moe_down", moe_down_kernel<MX, ND>, dim3((a.H + 15) / 16), dim3(64 * ND), st, a,
                  (const uint16_t*)act, KC);
}

hipError_t moe_experts(const MoeArgs& a, bool mx4, hipStream_t st, StageTimer* tm) {
    return mx4 ? experts<true>(a, st, tm) : experts<false>(a, st, tm);
}

}  // namespace lora
