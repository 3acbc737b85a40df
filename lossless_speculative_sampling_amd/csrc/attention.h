// Attention of rows that share a long prefix: launch arguments, the choice of a query tile and the
// workspace, shared by the C ABI and the kernels.
#pragma once

#include "common.h"

namespace sv {
namespace attn {

constexpr int kMaxD = 256;
constexpr int kThreads = 256;  // four waves

struct Args {
    const void* q;
    int64_t q_row, q_head;
    int R, q_heads, heads, D, per;  // per = q_heads / heads
    spec_kv_cache cache;
    int page_shift;  // log2 of the page size, -1 where it is no power of two
    int G;
    const int32_t* row_start;
    const int32_t* table;
    int max_pages;
    const int32_t* prefix_len;
    const int32_t* lists;
    int max_suffix;
    const int32_t* suffix_len;
    float scale;
    void* out;
    int64_t out_row, out_head;
    float* lse;
    // plan and workspace
    int want, slots;     // prefix pieces per cache head aimed at, and room for
    int suffix_blocks;   // workgroups of the suffix lists
    float* piece_o;      // [slots * heads][tile][D]
    float2* piece_ml;    // [slots * heads][tile]  (reference exponent, sum)
    float* suffix_o;     // [R][q_heads][D]
    float2* suffix_ml;   // [R][q_heads]
    int2* groups;        // [G]  (first piece, pieces along the prefix)
};

// Queries (row, head of the cache head) a workgroup takes: MB blocks of 16 per wave, WQ waves side by
// side over queries and 4 / WQ over keys.
struct Tile {
    int mb, wq;
    int queries() const { return 16 * mb * wq; }
};

// The tile that holds an average group's queries of one cache head (fewer passes over a prefix
// cost more than idle columns of a matrix instruction), as far as the registers go.
inline Tile tile_of(int R, int G, int per, int D) {
    const int64_t m = ((int64_t)R * per + G - 1) / G;
    if (D > 128) return Tile{1, 4};
    return m <= 32 ? Tile{1, 2} : m <= 64 ? Tile{2, 2} : Tile{2, 4};
}

struct Plan {
    Tile tile;
    int want, slots;
    int64_t suffix_blocks;
    size_t piece_o, piece_ml, suffix_o, suffix_ml, groups, bytes;  // offsets into the workspace
};

// Pieces: as many workgroups as are resident at once, two on every compute unit (three for the
// largest tile).  More of them, measured up to 2048, cost more in their beginnings and ends than they
// give in balance.
inline int pieces_of(const Tile& t) { return t.mb * t.wq == 8 ? 768 : 512; }

inline Plan plan_of(int R, int G, int q_heads, int heads, int D, int64_t max_prefix, int max_suffix) {
    const int per = q_heads / heads;
    Plan p{};
    p.tile = tile_of(R, G, per, D);
    // tiles of one cache head: at most one begun per group beyond the whole ones
    const int64_t tiles = (int64_t)R * per / p.tile.queries() + G;
    p.want = (pieces_of(p.tile) + heads - 1) / heads;
    p.slots = max_prefix ? (int)(p.want + tiles) : 0;
    const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t pieces = (size_t)p.slots * heads, q = p.tile.queries();
    const size_t rows = max_suffix ? (size_t)R * q_heads : 0;
    p.suffix_blocks = max_suffix ? ((int64_t)R * heads * ((per + 15) / 16) + 3) / 4 : 0;
    size_t at = 0;
    const auto take = [&](size_t n) { const size_t was = at; at += up(n); return was; };
    p.piece_o = take(pieces * q * D * sizeof(float));
    p.piece_ml = take(pieces * q * sizeof(float2));
    p.suffix_o = take(rows * D * sizeof(float));
    p.suffix_ml = take(rows * sizeof(float2));
    p.groups = take((size_t)G * sizeof(int2));
    p.bytes = at;
    return p;
}

void launch(const Args& a, const Tile& tile, int dtype, hipStream_t stream);

}  // namespace attn
}  // namespace sv
