// How decode attention (attn.hip) lays out its work, from sizes alone and on the
// host: the variant, how many workgroups it is split over, and the workspace.
// The workspace that a caller is told to bring is the most over what a call of
// those sizes can take, from the same function as the call's own.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

namespace lora {

// wgs: workgroups that the line of units is split over; 0: a workgroup a row and
// no line, join or workspace. It never falls as `longest` rises.
struct AttnShape {
    int dp, rt, blocks, block_heads, waves, wgs;
};
inline AttnShape attn_shape(int B, int heads, int kv_heads, int dim, int longest, bool f8) {
    AttnShape s;
    s.dp = dim <= 64 ? 64 : dim <= 128 ? 128 : 256;
    // heads a workgroup: as many as its registers hold
    const int group = heads / kv_heads, most = s.dp == 256 ? 16 : s.dp == 128 ? 32 : 64;
    s.blocks = (group + most - 1) / most;
    s.block_heads = (group + s.blocks - 1) / s.blocks;
    s.rt = s.block_heads <= 16 ? 1 : s.block_heads <= 32 ? 2 : 4;
    const int64_t rows = (int64_t)B * kv_heads * s.blocks;
    // 8 waves a workgroup where that is all there is to fill a CU, and two waves a
    // SIMD have the registers: bf16, 32 heads over 8 of 128, 1024 positions of 1
    // request (8 rows) 9.5 against 12.0 us with 4, 600 of 16 (128 rows) 10.6 against
    // 11.5, 128 of 64 (512 rows) 9.7 against 6.7
    const bool wide = rows <= 256 && s.dp * s.rt <= 128;
    // Short rows go to a workgroup each from end to end, which saves finding the
    // parts and the join (some 8 us): the same heads, 1000 positions of 1 request
    // 10.4 against 14.1 us, 2048 15.2 against 12.5; of 64 requests of 1 to 2048
    // 52 against 56 us, to 3300 93 against 92; 16 heads over 4 of 256, 600
    // positions of 1 request 16.0 against 14.3
    if (longest <= (rows >= 128 ? 2048 : wide ? 1536 : 512)) {
        s.wgs = 0;
        s.waves = wide ? 8 : 4;
    } else {  // two workgroups a CU, where their LDS allows it
        s.wgs = s.dp * (f8 ? 1 : 2) > 256 ? 256 : 512;
        s.waves = 4;
    }
    return s;
}

// Two neighbouring kv heads as one of twice the dimensions, where rows of one are
// half a 128-byte line, whose rest another workgroup would read at its own time
// (8-bit, 32 heads over 8 of 64, 16384 positions of 64 requests 208 against 337
// us), and where they are many, if whole rows: 600 positions of 32 requests (256
// rows) 8.4 against 10.7, of 16 8.2 against 6.5.
inline bool attn_pairs(int heads, int kv_heads, int dim, bool f8) {
    return dim * (f8 ? 1 : 2) == 64 && kv_heads % 2 == 0 && 2 * (heads / kv_heads) <= 16;
}

struct AttnLayout {
    AttnShape s;
    bool pair;     // kv heads in pairs
    size_t rows;   // requests x kv heads (or pairs) x head blocks
    size_t slots;  // pieces that the workspace holds
    size_t ml_at, meta_at, bytes;  // m and l of the pieces behind their o, the rows' pieces, the end
};
// adjacent: the heads of a cache's row follow one another without a gap.
inline AttnLayout attn_layout(int B, int heads, int kv_heads, int dim, int width, int page_rows, int window, bool f8,
                              bool adjacent) {
    // positions a request can attend to, and the ones its first tile may begin
    // ahead of them, which are positions of the table too
    const int most = width * page_rows;
    const int longest = window > 0 && window < most ? std::min(window + 15, most) : most;
    AttnLayout l{};
    l.s = attn_shape(B, heads, kv_heads, dim, longest, f8);
    l.rows = (size_t)B * kv_heads * l.s.blocks;
    l.pair = adjacent && attn_pairs(heads, kv_heads, dim, f8) && (l.s.wgs || l.rows >= 256);
    if (l.pair) {
        l.s = attn_shape(B, heads, kv_heads / 2, 2 * dim, longest, f8);
        l.rows = (size_t)B * (kv_heads / 2);
    }
    l.slots = l.s.wgs + l.rows;
    if (l.s.wgs == 0) return l;
    auto align256 = [](size_t n) { return (n + 255) & ~size_t(255); };
    l.ml_at = align256(l.slots * l.s.block_heads * dim * 4);
    l.meta_at = l.ml_at + align256(l.slots * l.s.block_heads * 8);
    l.bytes = l.meta_at + align256(l.rows * 8);
    return l;
}

// For any window, form and strides: without a window nothing is shorter.
inline size_t attn_workspace_bytes(int B, int heads, int kv_heads, int dim, int width, int page_rows) {
    size_t most = 0;
    for (bool f8 : {false, true})
        for (bool adjacent : {false, true})
            most = std::max(most, attn_layout(B, heads, kv_heads, dim, width, page_rows, 0, f8, adjacent).bytes);
    return most;
}

}  // namespace lora
