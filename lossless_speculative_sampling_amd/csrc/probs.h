// Verification from given probabilities and random numbers: launch arguments and the cut of a
// vocabulary row into chunks, shared by the C ABI and the kernels.
#pragma once

#include "common.h"

namespace sv {
namespace probs {

constexpr int kThreads = 256;
constexpr int kTile = kThreads * 8;  // elements one workgroup takes in one step (8 per thread)
constexpr int kMaxChunks = 1024;     // chunk masses per request the second kernel scans at once
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
    int chunk, chunks;  // elements per chunk (a multiple of kTile), chunks per row
    double* sums;       // [B][chunks] chunk masses
    Rec* recs;          // [B]
};

// Chunk length: the whole row up to kOneLaunchV tokens (one launch then does all); one tile while that gives at most eight workgroups per compute unit or so, four
// tiles beyond (fewer chunk masses and decisions for the same streaming), and for rows of more
// than kMaxChunks of those whatever keeps kMaxChunks.
inline int chunk_of(int B, int V) {
    const int64_t tiles = ((int64_t)V + kTile - 1) / kTile;
    if (V <= kOneLaunchV) return (int)(tiles * kTile);
    int64_t t = (int64_t)B * tiles <= 2048 ? 1 : 4;
    if (tiles > t * kMaxChunks) t = (tiles + kMaxChunks - 1) / kMaxChunks;
    return (int)(t * kTile > 0x7fffffff - kTile ? 0x7fffffff / kTile * kTile : t * kTile);
}

void launch(const Args& a, int dtype, hipStream_t stream);

}  // namespace probs
}  // namespace sv
