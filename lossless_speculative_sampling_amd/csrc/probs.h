// Verification from given probabilities and random numbers: launch arguments and the cut of a
// vocabulary row into cells, shared by the C ABI and the kernels.
#pragma once

#include "common.h"

namespace sv {
namespace probs {

constexpr int kThreads = 256;
constexpr int kTile = kThreads * 8;  // elements one workgroup takes in one step (8 per thread)
constexpr int kMaxCells = 1024;      // cell masses per request the second kernel scans at once
constexpr int kCellsAtOnce = 4;      // most cells a workgroup of the first takes
constexpr size_t kCacheBytes = 256u << 20;  // the last cache before HBM
constexpr int kOneLaunchV = 4 * kTile;

// What the first kernel hands to the second for a request.
struct Rec {
    int32_t k;        // accepted tokens, -1 for a bad request
    int32_t len;      // drafted tokens
    uint32_t status;
    int32_t pad;
};

struct Args {
    const void* draft;
    int64_t draft_req, draft_row;
    const void* target;
    int64_t target_req, target_row;
    int B, K, V;
    const int32_t* tokens;
    const int32_t* lens;
    const void* u;
    const void* v;
    int u64;          // random numbers are doubles
    uint32_t flags;
    int32_t* out_k;
    int32_t* out_tstar;
    int32_t* out_emitted;
    float* out_mass;
    uint32_t* out_status;
    int cell, cells;  // elements per cell (a multiple of kTile), cells per row
    int per;          // cells per workgroup of the first kernel
    double* sums;     // [B][cells] cell masses
    Rec* recs;        // [B]
};

// A row is cut into cells whose masses the draw finds its place by: one tile each, up to kMaxCells
// of them (longer rows: longer cells).
inline int cell_of(int V) {
    const int64_t tiles = ((int64_t)V + kTile - 1) / kTile, t = (tiles + kMaxCells - 1) / kMaxCells;
    return (int)(t * kTile);
}
// Workgroups take one cell while that gives at most eight or so per compute unit, several beyond
// (fewer scans for the same streaming).
inline int per_of(int B, int cells) { return (int64_t)B * cells <= 2048 ? 1 : kCellsAtOnce; }

void launch(const Args& a, int dtype, hipStream_t stream);

}  // namespace probs
}  // namespace sv
