// Attention of one new token a request over a paged key-value cache:
//   out[b][h] = sum_j p_j v_j,  p = softmax_j(scale q . k_j)
// over the request's positions j, read through its row of the page table. All
// heads of a kv head ride as columns of the matrix-core products, so every
// key and value is read once; 8-bit values turn into bf16 (exactly) on the way
// to them.
//
// A wave takes tiles of kTile positions, with a running maximum m, sum l and
// output o of its own (base 2):
//   S = K q   (rows: positions, columns: heads; a lane holds 8 neighbouring
//              positions of one head per 32)
//   o = o f + V^T P   (rows: dimensions, columns: heads), P as two bf16 halves:
//              16 bits of mantissa against the 8 of the output; l has P whole
// The lane that holds a head's scores holds its column of P and of o too, so
// the running maximum is shared by two lane swaps a tile and nothing else
// moves. Keys and values go straight to LDS (kTile rows each, one buffer a
// wave: the next tile's keys are asked for once the products with this one's
// are made, its values likewise); values are read from there transposed. No
// wave waits on another until the end of a piece.
//
// Long work is split by what there is, not by request: the positions of all
// requests and kv heads, in units of 4 tiles, are one line, of which every
// workgroup takes an equal part. It finds its part from the lengths itself. A
// part that ends inside a request leaves m, l and o in the workspace, and a
// second kernel joins the pieces of each request. Short rows (a kv head of a
// request each) go to a workgroup from end to end, in one launch.
//
// Positions whose page is outside the cache are left out, so no table makes a
// kernel read past it; nothing past a request's length is read either.
//
// Bound by HBM: 64 requests of 4096 to 16384 positions, 32 heads over 8 of 128,
// bf16 (2.7 GB) 471 us, 5.7 TB/s (a 1 GiB copy moves 5.1); without the second
// halves of P it is no faster. Rows of 128 bytes of a head (8-bit, [page][row]
// [head]) come at 5.0 TB/s, of 64 bytes, two heads of them together, at 5.1. 1
// request of 131072 positions, 8-bit (268 MB): 49 us and 4 to 7 for the join; some
// 8 us of every call are its beginning and end.
#include <algorithm>

#include "attn_plan.h"
#include "fuse.h"
#include "kernels.h"

namespace lora {

constexpr float kLowest = -3.402823466e38f;  // below every finite score, and finite

// How the work is laid out, decided on the host.
struct AttnPlan {
    AttnArgs a;
    int wgs;          // workgroups the line of units is split over; 0: one workgroup a row, no line
    int rows;         // rows a request: kv heads x head blocks
    int blocks;       // head blocks a kv head
    int block_heads;  // heads a block
    int hd;           // dimensions of a head: a.c.dim, or half of it where kv heads go in pairs
    int pair;         // heads of the first kv head of a pair; 0: no pairs
    uint32_t magic;   // position / page_rows = umulhi(position, magic) >> shift (page_rows > 1)
    int shift;
    int whole;        // whole tiles by AttnTile::group
    float* part;      // [wgs + B rows][block_heads][dim] o of a piece
    float2* ml;       // [wgs + B rows][block_heads] m, l of a piece
    int2* meta;       // [B rows] first piece, pieces
};

// DP: dimensions padded to 64, 128 or 256 (zeros behind dim). RT: 16-head
// blocks of a kv head's heads. W: waves a workgroup: 4, or 8 where a workgroup
// takes a row from end to end and two waves a SIMD have the registers. PAIR: two
// kv heads as one, each of half the dimensions, which is one 64-byte chunk of the
// reads of keys.
template <int DP_, bool F8_, int RT_, int W_, bool PAIR_ = false>
struct AttnCfg {
    static constexpr int DP = DP_, RT = RT_, W = W_;
    static constexpr bool F8 = F8_, PAIR = PAIR_;
    static constexpr int ROWB = DP * (F8 ? 1 : 2);  // bytes of a row in LDS
    static constexpr int CH = ROWB / 16;            // its 16-byte chunks
    static constexpr int RW = CH < 16 ? 16 / CH : 1;  // rows of a 256-byte window (all banks)
    static constexpr int LRW = RW == 1 ? 0 : RW == 2 ? 1 : 2;
    static constexpr int TK = ROWB <= 128 ? 64 : 32;  // positions of a tile
    static constexpr int NB = TK / 32;
    static constexpr int STAGE = TK * ROWB;
    static constexpr int NI = STAGE / 1024;  // load instructions a stage
    static constexpr int RI = 64 / CH;       // rows a load instruction
    static constexpr int U = W * TK;
    // waves a SIMD to compile for: 2 leaves 256 registers, where the products take
    // vector registers alone and o is not copied to and fro
    static constexpr int MinWaves = DP * RT <= 128 ? 2 : 1;
};

// Chunk c of row r lies at chunk c ^ swizzle(r) of its row, so that the reads
// of 16 lanes meet all banks: keys are read as 16 rows {0-3, 8-11, 16-19,
// 24-27} (+4) at one chunk, values transposed as 8 rows {0-3, 8-11} at two
// neighbouring chunks (16-bit) or 16 rows at one (8-bit).
template <class C>
__device__ __forceinline__ constexpr int swz_k(int r) {
    return ((r & 3) | ((r >> 3) & 3) << 2) >> C::LRW;
}
template <class C>
__device__ __forceinline__ constexpr int swz_v(int r) {
    return C::F8 ? (r & 15) >> C::LRW : (((r & 3) | ((r >> 3) & 1) << 2) >> C::LRW) << 1;
}

// LDS reads with their wait in one block, so that nothing is in flight when
// the compiler goes on. N: rows of addresses; each address and the one `step`
// bytes on.
template <int STEP>
__device__ __forceinline__ void lds_rows(u32x4 (&lo)[1], u32x4 (&hi)[1], const uint32_t (&a)[1]) {
    asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %2 offset:%3\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(lo[0]), "=&v"(hi[0])
                 : "v"(a[0]), "i"(STEP)
                 : "memory");
}
template <int STEP>
__device__ __forceinline__ void lds_rows(u32x4 (&lo)[2], u32x4 (&hi)[2], const uint32_t (&a)[2]) {
    asm volatile(
        "ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:%6\n\t"
        "ds_read_b128 %2, %5\n\tds_read_b128 %3, %5 offset:%6\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(lo[0]), "=&v"(hi[0]), "=&v"(lo[1]), "=&v"(hi[1])
        : "v"(a[0]), "v"(a[1]), "i"(STEP)
        : "memory");
}
template <int STEP>
__device__ __forceinline__ void lds_rows(u32x4 (&lo)[4], u32x4 (&hi)[4], const uint32_t (&a)[4]) {
    asm volatile(
        "ds_read_b128 %0, %8\n\tds_read_b128 %1, %8 offset:%12\n\t"
        "ds_read_b128 %2, %9\n\tds_read_b128 %3, %9 offset:%12\n\t"
        "ds_read_b128 %4, %10\n\tds_read_b128 %5, %10 offset:%12\n\t"
        "ds_read_b128 %6, %11\n\tds_read_b128 %7, %11 offset:%12\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(lo[0]), "=&v"(hi[0]), "=&v"(lo[1]), "=&v"(hi[1]), "=&v"(lo[2]), "=&v"(hi[2]), "=&v"(lo[3]),
          "=&v"(hi[3])
        : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "i"(STEP)
        : "memory");
}
// Transposed: of 16 lanes' 8-byte pieces, 4 rows x 16 columns of 16-bit values
// (two such reads, STEP bytes apart) or 8 rows x 16 columns of 8-bit ones,
// lane i gets column i.
template <int STEP>
__device__ __forceinline__ void lds_columns16(u32x2 (&lo)[4], u32x2 (&hi)[4], const uint32_t (&a)[4]) {
    asm volatile(
        "ds_read_b64_tr_b16 %0, %8\n\tds_read_b64_tr_b16 %1, %8 offset:%12\n\t"
        "ds_read_b64_tr_b16 %2, %9\n\tds_read_b64_tr_b16 %3, %9 offset:%12\n\t"
        "ds_read_b64_tr_b16 %4, %10\n\tds_read_b64_tr_b16 %5, %10 offset:%12\n\t"
        "ds_read_b64_tr_b16 %6, %11\n\tds_read_b64_tr_b16 %7, %11 offset:%12\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(lo[0]), "=&v"(hi[0]), "=&v"(lo[1]), "=&v"(hi[1]), "=&v"(lo[2]), "=&v"(hi[2]), "=&v"(lo[3]),
          "=&v"(hi[3])
        : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "i"(STEP)
        : "memory");
}
__device__ __forceinline__ void lds_columns8(u32x2 (&r)[4], const uint32_t (&a)[4]) {
    asm volatile(
        "ds_read_b64_tr_b8 %0, %4\n\tds_read_b64_tr_b8 %1, %5\n\t"
        "ds_read_b64_tr_b8 %2, %6\n\tds_read_b64_tr_b8 %3, %7\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3])
        : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3])
        : "memory");
}

// 8 E4M3 values as bf16 (exact).
__device__ __forceinline__ u32x4 widen8(uint32_t a, uint32_t b) {
    u32x4 r;
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, false));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.f, true));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, false));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.f, true));
    return r;
}

// The kv head that head h of a row reads.
__device__ __forceinline__ int kv_head(const AttnPlan& p, int hk, int h) {
    return p.pair ? 2 * hk + (h >= p.pair) : hk;
}

// Over the four lanes that hold a head (lane, lane ^ 16, ^ 32, ^ 48).
__device__ __forceinline__ float head_max(float v) {
    const uint32_t a = __float_as_uint(v);
    const auto p = __builtin_amdgcn_permlane32_swap(a, a, false, false);
    const float w = fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
    const uint32_t b = __float_as_uint(w);
    const auto q = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
__device__ __forceinline__ float head_sum(float v) {
    const uint32_t a = __float_as_uint(v);
    const auto p = __builtin_amdgcn_permlane32_swap(a, a, false, false);
    const float w = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    const uint32_t b = __float_as_uint(w);
    const auto q = __builtin_amdgcn_permlane16_swap(b, b, false, false);
    return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// The positions [lo, hi) a request attends to; tiles start at lo rounded down
// to 16, so that 16 rows of a load never straddle a page of 16.
__device__ __forceinline__ void attn_range(const AttnArgs& a, int b, int* lo, int* hi) {
    const int n = min(max(a.lengths[b], 0), a.width * a.c.page_rows);
    *lo = a.window > 0 ? max(n - a.window, 0) : 0;
    *hi = n;
}
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
template <class C>
__device__ __forceinline__ int attn_units(const AttnArgs& a, int b) {
    int lo, hi;
    attn_range(a, b, &lo, &hi);
    return (hi - (lo & ~15) + C::U - 1) / C::U;
}

// Units a workgroup, from the units there are: an equal part each, at least
// kMinUnits.
constexpr int kMinUnits = 1;
__device__ __forceinline__ int64_t units_per_wg(int64_t units, int wgs) {
    return max((int64_t)kMinUnits, (units + wgs - 1) / wgs);
}

template <class C>
struct AttnLds {
    alignas(1024) u32x4 kv[C::W][2 * C::STAGE / 16];
    float m[C::W][16], l[C::W][16];
    int64_t scan[C::W];
    int64_t found[2];
    int request;
};

// 64 entries of a request's page table, one a lane: a wait for them is one for
// everything the wave has asked for, so they are fetched for many tiles at once
// (page_rows 16: 8 tiles, 64: 32).
struct AttnPages {
    const int32_t* table;
    int first, last;  // entries held, the request's last one
    int page;
};
__device__ __forceinline__ int page_of(const AttnPlan& p, int pos) {
    return p.a.c.page_rows > 1 ? (int)(__umulhi((uint32_t)pos, p.magic) >> p.shift) : pos;
}

// Where a tile's rows are. Whole tiles over pages of a multiple of 16 rows, with
// dim filling its chunks, are four numbers or two; of others every lane has its
// row's, and the mask says which are attended to.
template <class C>
struct AttnTile {
    static constexpr int G = C::TK / 16;
    bool whole;
    int64_t group[G];  // bytes to each 16 rows
    int64_t off;       // bytes to this lane's row (lane = row of the tile)
    uint64_t mask;     // rows that are attended to
};
template <class C>
__device__ __forceinline__ AttnTile<C> tile_rows(const AttnPlan& p, AttnPages& pages, int pos, int lo, int hi,
                                                 int64_t head) {
    constexpr int ES = C::F8 ? 1 : 2;
    const KvCache& c = p.a.c;
    const int lane = threadIdx.x & 63, e0 = page_of(p, pos), e1 = page_of(p, min(pos + C::TK, hi) - 1);
    if (e1 - pages.first >= 64) {  // uniform
        pages.first = e0;
        pages.page = pages.table[min(e0 + lane, pages.last)];
        asm volatile("" : "+v"(pages.page));  // waited for here
    }
    AttnTile<C> t;
    t.whole = p.whole && pos >= lo && pos + C::TK <= hi;
    if (t.whole) {
#pragma unroll
        for (int g = 0; g < AttnTile<C>::G; ++g) {
            const int at = pos + 16 * g, e = page_of(p, at);
            const int page = __builtin_amdgcn_readlane(pages.page, e - pages.first);
            t.whole &= page >= 0 && page < c.n_pages;
            t.group[g] = (page * c.page_stride + (int64_t)(at - e * c.page_rows) * c.row_stride + head) * ES;
        }
        t.mask = C::TK == 64 ? ~0ull : 0xffffffffull;
    }
    if (!t.whole) {
        const int at = min(pos + lane, hi - 1), e = page_of(p, at);
        const int page = __shfl(pages.page, min(e - pages.first, 63));
        t.off = (page * c.page_stride + (int64_t)(at - e * c.page_rows) * c.row_stride + head) * ES;
        t.mask = __ballot(lane < C::TK && pos + lane >= lo && pos + lane < hi && page >= 0 && page < c.n_pages);
    }
    return t;
}

// A tile's rows of keys or values into LDS; rows that are left out, and chunks
// behind dim, as zeros. The swizzle is in the source address, since the LDS
// address goes lane by lane.
template <class C, bool V>
__device__ __forceinline__ void load_stage(const AttnPlan& p, const void* base, const AttnTile<C>& t, u32x4* dst,
                                           uint32_t lane) {
    constexpr int ES = C::F8 ? 1 : 2;
    // what follows from the lane is computed again for every stage: kept from
    // one to the next it takes the registers of the products
    asm volatile("" : "+v"(lane));
    const uint32_t r0 = lane / C::CH, c0 = lane % C::CH;
    if (t.whole) {  // uniform
#pragma unroll
        for (int j = 0; j < C::NI; ++j) {
            const uint32_t r = j * C::RI + r0;
            const char* at = static_cast<const char*>(base) + t.group[j * C::RI / 16] +
                             (int64_t)(j * C::RI % 16) * p.a.c.row_stride * ES;
            const uint32_t off = r0 * ((uint32_t)p.a.c.row_stride * ES) + (c0 ^ (V ? swz_v<C>(r) : swz_k<C>(r))) * 16;
            dma16(as_global<u32x4>(at + off), dst + j * 64);
        }
        return;
    }
    const uint32_t dim_chunks = p.a.c.dim * ES / 16;
#pragma unroll
    for (int j = 0; j < C::NI; ++j) {
        const uint32_t r = j * C::RI + r0;
        const uint32_t chunk = c0 ^ (V ? swz_v<C>(r) : swz_k<C>(r));
        const uint32_t lo32 = __shfl((int)(uint32_t)t.off, r), hi32 = __shfl((int)(uint32_t)(t.off >> 32), r);
        const int64_t at = (int64_t)((uint64_t)hi32 << 32 | lo32);
        const bool ok = ((t.mask >> r) & 1) && chunk < dim_chunks;
        dma16(or_zero(ok, static_cast<const char*>(base) + at + chunk * 16), dst + j * 64);
    }
}

// One piece: units [t0, t1) of row `row` of request b.
template <class C>
__device__ __forceinline__ void attn_piece(const AttnPlan& p, AttnLds<C>& L, int b, int row, int t0, int t1, bool whole,
                                           int64_t slot) {
    constexpr int DP = C::DP, RT = C::RT, NB = C::NB, NK = DP / 32, ND = DP / 16;
    const AttnArgs& a = p.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, fg = lane >> 4, D = p.hd;
    const int hk = row / p.blocks, hb = row % p.blocks, group = a.heads / a.c.kv_heads;
    const int h0 = hk * group + hb * p.block_heads, nq = min(p.block_heads, group - hb * p.block_heads);
    int lo, hi;
    attn_range(a, b, &lo, &hi);
    lo = uniform(lo), hi = uniform(hi);
    const int start = lo & ~15;
    // this wave's tiles: position start + (W unit + wave) TK
    const int first = start + (C::W * t0 + wave) * C::TK;
    const int end = min(hi, start + t1 * C::U);
    const int nt = first < end ? (end - first + C::U - 1) / C::U : 0;
    const int64_t head = hk * a.c.head_stride;
    AttnPages pages{a.table + b * a.table_stride, -64, nt > 0 ? page_of(p, hi - 1) : 0, 0};

    u32x4* kbuf = L.kv[wave];
    u32x4* vbuf = kbuf + C::STAGE / 16;
    // q as the right operand: column fr = head, 8 k a lane; ahead of the tiles, so
    // that the wait for it is not one for them
    u32x4 q[RT][NK];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int c = 0; c < NK; ++c) {
            const int h = rt * 16 + fr;
            // 8-bit keys: a lane's 16-byte read holds the k of two products
            const int d = C::F8 ? (c >> 1) * 64 + fg * 16 + (c & 1) * 8 : c * 32 + fg * 8;
            const int at = C::PAIR ? d % (DP / 2) : d;
            q[rt][c] = *or_zero(h < nq && at < D, a.q + b * a.q_stride + (int64_t)(h0 + h) * D + at);
        }
    AttnTile<C> tile{};
    if (nt > 0) {
        tile = tile_rows<C>(p, pages, first, lo, hi, head);
        load_stage<C, false>(p, a.c.k, tile, kbuf, lane);
        issue_fence();
        load_stage<C, true>(p, a.c.v, tile, vbuf, lane);
        issue_fence();
    }

#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int c = 0; c < NK; ++c) asm volatile("" : "+v"(q[rt][c]));  // it has landed
    float sc[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
        sc[rt] = a.scale_log2 * (C::F8 ? a.c.k_scale[C::PAIR ? kv_head(p, hk, min(rt * 16 + fr, nq - 1)) : hk] : 1.f);

    f32x4 o[RT][ND];
    float m[RT], l[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        m[rt] = kLowest;
        l[rt] = 0.f;
#pragma unroll
        for (int d = 0; d < ND; ++d) o[rt][d] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    const int kr = 8 * (fr >> 2) + (fr & 3);  // key row of the first block; the second's is 4 on
    const uint32_t k0 = lds_offset(kbuf) + kr * C::ROWB + ((fg ^ swz_k<C>(kr)) << 4);
    // value rows 8 fg + (fr / 4) (and 4 on), columns 4 (fr % 4); 8-bit: 8 fg + fr / 2, 8 (fr % 2)
    const int vr = C::F8 ? 8 * fg + (fr >> 1) : 8 * fg + (fr >> 2);
    const uint32_t v0 = lds_offset(vbuf) + vr * C::ROWB +
                        (C::F8 ? (swz_v<C>(vr) << 4) + (fr & 1) * 8
                               : ((((fr & 3) >> 1) ^ swz_v<C>(vr)) << 4) + (fr & 1) * 8);

    f32x4 s[RT][NB][2];
    u32x4 ph[RT][NB], pl[RT][NB];
    auto scores = [&]() {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int n = 0; n < NB; ++n) s[rt][n][0] = s[rt][n][1] = f32x4{0.f, 0.f, 0.f, 0.f};
        constexpr int NR = C::F8 ? (DP / 64) : (NK < 4 ? NK : 4);  // 16-byte reads of a row at once
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int c0 = 0; c0 < C::CH / 4; c0 += NR) {
                uint32_t addr[NR];
                u32x4 k[2][NR];
#pragma unroll
                for (int c = 0; c < NR; ++c) addr[c] = (k0 ^ ((c0 + c) << 6)) + n * 32 * C::ROWB;
                lds_rows<4 * C::ROWB>(k[0], k[1], addr);
                if constexpr (C::PAIR) {
                    // each kv head's products by themselves (with zeros in q a NaN of
                    // one would reach the other's), of which a column takes its own
                    static_assert(RT == 1 && NR == 2 && C::CH == 2 * 4, "a chunk a kv head");
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        f32x4 r[2];
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            r[c] = f32x4{0.f, 0.f, 0.f, 0.f};
                            if constexpr (C::F8) {
                                r[c] = mfma16x16x32(widen8(k[h][c][0], k[h][c][1]), q[0][2 * c], r[c]);
                                r[c] = mfma16x16x32(widen8(k[h][c][2], k[h][c][3]), q[0][2 * c + 1], r[c]);
                            } else {
                                r[c] = mfma16x16x32(k[h][c], q[0][c], r[c]);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[0][n][h][i] = fr < p.pair ? r[0][i] : r[1][i];
                    }
                    continue;
                }
#pragma unroll
                for (int c = 0; c < NR; ++c)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if constexpr (C::F8) {
                            const u32x4 x = widen8(k[h][c][0], k[h][c][1]), y = widen8(k[h][c][2], k[h][c][3]);
#pragma unroll
                            for (int rt = 0; rt < RT; ++rt) {
                                s[rt][n][h] = mfma16x16x32(x, q[rt][2 * (c0 + c)], s[rt][n][h]);
                                s[rt][n][h] = mfma16x16x32(y, q[rt][2 * (c0 + c) + 1], s[rt][n][h]);
                            }
                        } else {
#pragma unroll
                            for (int rt = 0; rt < RT; ++rt)
                                s[rt][n][h] = mfma16x16x32(k[h][c], q[rt][c0 + c], s[rt][n][h]);
                        }
                    }
            }
    };
    auto weights = [&](uint64_t mask) {
        // scores (base 2), the running maximum, P as two bf16 halves
        const bool all = C::TK == 64 ? mask == ~0ull : mask == 0xffffffffull;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            float e[NB][8], top = kLowest;
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int j = 0; j < 8; ++j) e[n][j] = s[rt][n][j >> 2][j & 3] * sc[rt];
            if (!all)
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const uint32_t bits = (uint32_t)(mask >> (32 * n)) >> (8 * fg);
#pragma unroll
                    for (int j = 0; j < 8; ++j) e[n][j] = (bits >> j) & 1 ? e[n][j] : -INFINITY;
                }
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int j = 0; j < 8; ++j) top = fmaxf(top, e[n][j]);
            top = fmaxf(m[rt], head_max(top));
            if (__any(top > m[rt])) {
                const float f = __builtin_amdgcn_exp2f(m[rt] - top);
                l[rt] *= f;
#pragma unroll
                for (int d = 0; d < ND; ++d) o[rt][d] *= f;
                m[rt] = top;
            }
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float x = __builtin_amdgcn_exp2f(e[n][j] - m[rt]), y = __builtin_amdgcn_exp2f(e[n][j + 1] - m[rt]);
                    l[rt] += x + y;
                    const uint32_t h = pack_bf16x2(x, y);
                    ph[rt][n][j >> 1] = h;
                    pl[rt][n][j >> 1] =
                        pack_bf16x2(x - __uint_as_float(h << 16), y - __uint_as_float(h & 0xffff0000u));
                }
        }
    };
    auto values = [&]() {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int d0 = 0; d0 < ND; d0 += 4) {
                uint32_t addr[4];
                u32x4 v[4];
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    addr[d] = (v0 ^ ((d0 + d) << (C::F8 ? 4 : 5))) + n * 32 * C::ROWB;
                if constexpr (C::F8) {
                    u32x2 x[4];
                    lds_columns8(x, addr);
#pragma unroll
                    for (int d = 0; d < 4; ++d) v[d] = widen8(x[d][0], x[d][1]);
                } else {
                    u32x2 x[4], y[4];
                    lds_columns16<4 * C::ROWB>(x, y, addr);
#pragma unroll
                    for (int d = 0; d < 4; ++d) v[d] = u32x4{x[d][0], x[d][1], y[d][0], y[d][1]};
                }
#pragma unroll
                for (int d = 0; d < 4; ++d)
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        o[rt][d0 + d] = mfma16x16x32(v[d], ph[rt][n], o[rt][d0 + d]);
                        o[rt][d0 + d] = mfma16x16x32(v[d], pl[rt][n], o[rt][d0 + d]);
                    }
            }
    };
    // Loads land in their order, keys of tile i + 1 behind the values of i, so
    // that a wait names how many of the later ones may still be out.
    for (int i = 0; i + 1 < nt; ++i) {
        vm_landed<C::NI>();  // the keys: the values were asked for after them
        scores();
        const AttnTile<C> next = tile_rows<C>(p, pages, first + (i + 1) * C::U, lo, hi, head);
        load_stage<C, false>(p, a.c.k, next, kbuf, lane);
        issue_fence();
        weights(tile.mask);
        vm_landed<C::NI>();  // the values: the next keys were asked for after them
        values();
        load_stage<C, true>(p, a.c.v, next, vbuf, lane);
        issue_fence();
        tile = next;
    }
    if (nt > 0) {
        vm_landed<C::NI>();
        scores();
        weights(tile.mask);
        vm_landed<0>();
        values();
    }

    // the waves' m, l and o joined through LDS, 16 heads at a time
    const int64_t out_row = (int64_t)b * a.heads + h0;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        if (rt * 16 >= nq) break;  // uniform
        f32x4* mine = reinterpret_cast<f32x4*>(kbuf);
        const float sum = head_sum(l[rt]);
        if (fg == 0) {
            L.m[wave][fr] = m[rt];
            L.l[wave][fr] = sum;
        }
#pragma unroll
        for (int d = 0; d < ND; ++d) mine[fr * (DP / 4) + ((4 * d + fg) ^ fr)] = o[rt][d];
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * (D / 4); i += 64 * C::W) {
            const int h = i / (D / 4), d4 = i % (D / 4);
            if (rt * 16 + h >= nq) break;
            const int hq = rt * 16 + h, from = C::PAIR && hq >= p.pair ? d4 + D / 4 : d4;
            float top = L.m[0][h], den = 0.f;
            f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 1; w < C::W; ++w) top = fmaxf(top, L.m[w][h]);
#pragma unroll
            for (int w = 0; w < C::W; ++w) {
                const float f = __builtin_amdgcn_exp2f(L.m[w][h] - top);
                den += f * L.l[w][h];
                x += f * reinterpret_cast<const f32x4*>(L.kv[w])[h * (DP / 4) + (from ^ h)];
            }
            if (whole) {
                const float vs = C::F8 ? a.c.v_scale[C::PAIR ? kv_head(p, hk, hq) : hk] : 1.f;
                const float r = den == 0.f ? 0.f : vs / den;
                const u32x2 y = {pack_bf16x2(x[0] * r, x[1] * r), pack_bf16x2(x[2] * r, x[3] * r)};
                *reinterpret_cast<u32x2*>(a.out + (out_row + hq) * D + 4 * d4) = y;
                if (a.lse && d4 == 0)
                    a.lse[out_row + hq] = den == 0.f ? -INFINITY : (top + log2f(den)) * 0.6931471805599453f;
            } else {
                *reinterpret_cast<f32x4*>(p.part + (slot * p.block_heads + hq) * D + 4 * d4) = x;
                if (d4 == 0) p.ml[slot * p.block_heads + hq] = make_float2(top, den);
            }
        }
        __syncthreads();
    }
}

template <class C>
__global__ __launch_bounds__(64 * C::W, C::MinWaves) void attn_decode_kernel(AttnPlan p) {
    __shared__ AttnLds<C> L;
    const AttnArgs& a = p.a;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (C::W == 8 || p.wgs == 0) {
        const int b = blockIdx.x / p.rows, row = blockIdx.x % p.rows;
        attn_piece<C>(p, L, b, row, 0, attn_units<C>(a, b), true, 0);
        return;
    }
    // the line: where every request's units begin
    const int per_thread = (a.B + 64 * C::W - 1) / (64 * C::W);
    const int b0 = min(tid * per_thread, a.B), b1 = min(b0 + per_thread, a.B);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += attn_units<C>(a, b);
    mine *= p.rows;
    int64_t in = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t v = __shfl_up(in, o);
        if (lane >= o) in += v;
    }
    if (lane == 63) L.scan[wave] = in;
    __syncthreads();
    int64_t total = 0, before = in - mine;
    for (int w = 0; w < C::W; ++w) {
        if (w < wave) before += L.scan[w];
        total += L.scan[w];
    }
    const int64_t per = units_per_wg(total, p.wgs);
    const int64_t u0 = blockIdx.x * per, u1 = min(u0 + per, total);
    if (u0 >= total) return;  // uniform
    if (u0 >= before && u0 < before + mine) {
        int b = b0;
        for (;; ++b) {
            const int64_t n = (int64_t)attn_units<C>(a, b) * p.rows;
            if (u0 < before + n) break;
            before += n;
        }
        L.request = b;
        L.found[0] = before;
    }
    __syncthreads();
    int b = uniform(L.request);
    int64_t at = L.found[0];  // where request b begins
    for (int64_t u = u0; u < u1 && b < a.B;) {
        const int n = uniform(attn_units<C>(a, b));
        const int64_t all = (int64_t)n * p.rows;
        if (u >= at + all) {
            at += all;
            ++b;
            continue;
        }
        // a request's units are far under 2^31, its part of a workgroup's too
        const int row = uniform((int)((u - at) / n)), t0 = uniform((int)(u - at - (int64_t)row * n));
        const int t1 = uniform((int)min((int64_t)n, t0 + (u1 - u)));
        const int64_t r = (int64_t)b * p.rows + row, slot = blockIdx.x + r;
        if (t0 == 0 && tid == 0) {
            const int64_t s = at + (int64_t)row * n;
            p.meta[r] = make_int2((int)slot, (int)((s + n - 1) / per - s / per + 1));
        }
        attn_piece<C>(p, L, b, row, t0, t1, t0 == 0 && t1 == n, slot);
        u += t1 - t0;
    }
}

// Rows of more than one piece joined, rows without a position written as
// zeros. A workgroup takes all heads of a row, or, where there are fewer than
// 256 rows, as many as make 256 workgroups (8 rows of 4 heads and 64 pieces: 6.4
// us with all, 4.3 with one; the attention of 128 rows of 64 heads, 600 positions
// each, 92 us with one, 28 with 32): its threads 4 dimensions of a head each, and
// where there are few of those, several share a head's pieces.
constexpr int kJoinThreads = 512;
template <bool F8>
__global__ __launch_bounds__(kJoinThreads) void attn_join_kernel(AttnPlan p) {
    __shared__ f32x4 so[kJoinThreads];
    __shared__ float2 sml[kJoinThreads];
    const AttnArgs& a = p.a;
    const int64_t r = blockIdx.x;
    const int b = (int)(r / p.rows), row = (int)(r - (int64_t)b * p.rows), D = p.hd;
    const int hk = row / p.blocks, hb = row % p.blocks, group = a.heads / a.c.kv_heads;
    const int nq = min(p.block_heads, group - hb * p.block_heads);
    const int64_t out_row = (int64_t)b * a.heads + hk * group + hb * p.block_heads;
    int lo, hi;
    attn_range(a, b, &lo, &hi);
    const int2 meta = hi > lo ? p.meta[r] : make_int2(0, 0);
    if (hi > lo && meta.y == 1) return;  // written by the first kernel
    const int per = (p.block_heads + gridDim.y - 1) / gridDim.y, h0 = blockIdx.y * per, heads = min(per, nq - h0);
    if (heads <= 0) return;
    const int items = heads * (D / 4);
    int share = 1;
    while (2 * share * items <= kJoinThreads) share *= 2;
    const int at = threadIdx.x / share, sub = threadIdx.x % share;
    for (int i0 = 0; i0 < items; i0 += kJoinThreads / share) {
        const int i = i0 + at, h = h0 + i / (D / 4), d4 = i % (D / 4);
        float m = kLowest, l = 0.f;
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
        if (i < items) {
#pragma unroll 4
            for (int n = sub; n < meta.y; n += share) {
                const int64_t s = (int64_t)(meta.x + n) * p.block_heads + h;
                const float2 ml = p.ml[s];
                const f32x4 y = *reinterpret_cast<const f32x4*>(p.part + s * D + 4 * d4);
                const float top = fmaxf(m, ml.x);
                const float f = __builtin_amdgcn_exp2f(m - top), g = __builtin_amdgcn_exp2f(ml.x - top);
                l = l * f + ml.y * g;
                x = x * f + y * g;
                m = top;
            }
        }
        so[threadIdx.x] = x;
        sml[threadIdx.x] = make_float2(m, l);
        __syncthreads();
        if (sub == 0 && i < items) {
            for (int n = 1; n < share; ++n) {
                const float2 ml = sml[threadIdx.x + n];
                const float top = fmaxf(m, ml.x);
                const float f = __builtin_amdgcn_exp2f(m - top), g = __builtin_amdgcn_exp2f(ml.x - top);
                l = l * f + ml.y * g;
                x = x * f + so[threadIdx.x + n] * g;
                m = top;
            }
            const float vs = F8 ? a.c.v_scale[kv_head(p, hk, hb * p.block_heads + h)] : 1.f;
            const float k = l == 0.f ? 0.f : vs / l;
            const u32x2 y = {pack_bf16x2(x[0] * k, x[1] * k), pack_bf16x2(x[2] * k, x[3] * k)};
            *reinterpret_cast<u32x2*>(a.out + (out_row + h) * D + 4 * d4) = y;
            if (a.lse && d4 == 0) a.lse[out_row + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------- host --
namespace {

template <int DP, bool F8, int RT>
auto attn_kernel(int waves) {
    if constexpr (DP * RT <= 128)
        if (waves == 8) return attn_decode_kernel<AttnCfg<DP, F8, RT, 8>>;
    return attn_decode_kernel<AttnCfg<DP, F8, RT, 4>>;
}
template <bool F8>
auto attn_kernel(const AttnShape& s, bool pair) {
    if (pair) {
        constexpr int DP = F8 ? 128 : 64;
        return s.waves == 8 ? attn_decode_kernel<AttnCfg<DP, F8, 1, 8, true>>
                            : attn_decode_kernel<AttnCfg<DP, F8, 1, 4, true>>;
    }
    if (s.dp == 256) return attn_kernel<256, F8, 1>(s.waves);
    if (s.dp == 128) return s.rt == 1 ? attn_kernel<128, F8, 1>(s.waves) : attn_kernel<128, F8, 2>(s.waves);
    return s.rt == 1   ? attn_kernel<64, F8, 1>(s.waves)
           : s.rt == 2 ? attn_kernel<64, F8, 2>(s.waves)
                       : attn_kernel<64, F8, 4>(s.waves);
}

}  // namespace

size_t attn_decode_workspace(int B, int heads, int kv_heads, int dim, int width, int page_rows) {
    return attn_workspace_bytes(B, heads, kv_heads, dim, width, page_rows);
}

hipError_t attn_decode(const AttnArgs& a, bool f8, hipStream_t st, StageTimer* tm) {
    const KvCache& c = a.c;
    const AttnLayout l = attn_layout(a.B, a.heads, c.kv_heads, c.dim, a.width, c.page_rows, a.window, f8,
                                     c.head_stride == c.dim);
    if (l.bytes > a.workspace_bytes) return hipErrorInvalidValue;
    const AttnShape& s = l.s;
    AttnPlan p{};
    p.a = a;
    p.hd = c.dim;
    if (l.pair) {
        p.pair = a.heads / c.kv_heads;
        p.a.c.kv_heads /= 2;
        p.a.c.dim *= 2;
        p.a.c.head_stride *= 2;
    }
    p.wgs = s.wgs;
    p.blocks = s.blocks;
    p.block_heads = s.block_heads;
    p.rows = p.a.c.kv_heads * s.blocks;
    // t / P for t < 2^31: with 2^(sh) < P <= 2^(sh + 1) and magic =
    // floor(2^(32 + sh) / P) + 1, t magic / 2^(32 + sh) is over t / P by less than 1 / P
    int sh = 0;
    while ((2ll << sh) < c.page_rows) ++sh;
    p.shift = sh;
    p.magic = c.page_rows > 1 ? (uint32_t)((1ull << (32 + sh)) / c.page_rows + 1) : 0;
    p.whole = c.page_rows % 16 == 0 && p.a.c.dim == s.dp && c.row_stride < (1 << 24);  // 16 rows' bytes in 31 bits
    char* ws = static_cast<char*>(a.workspace);
    p.part = reinterpret_cast<float*>(ws);
    p.ml = reinterpret_cast<float2*>(ws + l.ml_at);
    p.meta = reinterpret_cast<int2*>(ws + l.meta_at);
    auto kernel = f8 ? attn_kernel<true>(s, p.pair) : attn_kernel<false>(s, p.pair);
    const uint32_t rows = (uint32_t)l.rows, grid = s.wgs ? s.wgs : rows;
    hipError_t e = launch(tm, "attn_decode", kernel, dim3(grid), dim3(64 * s.waves), st, p);
    if (e != hipSuccess || s.wgs == 0) return e;
    const uint32_t splits = std::max(1u, std::min((uint32_t)s.block_heads, 256 / rows));
    return launch(tm, "attn_join", f8 ? attn_join_kernel<true> : attn_join_kernel<false>,
                  dim3(rows, splits), dim3(kJoinThreads), st, p);
}

}  // namespace lora
