// Draft-tree rows, and rotary positions with the append to the paged cache: launch arguments
// shared by the C ABI and the kernels.
#pragma once

#include "common.h"

namespace sv {
namespace kv {

constexpr int kThreads = 256;
constexpr int kLdsNodes = 4096;  // trees up to this size are walked in LDS

struct RowsArgs {
    const int32_t* tokens;
    const int32_t* parents;
    const int32_t* slots;
    const int32_t* ctx;
    int B, N, depth;
    int32_t* out_pos;
    int32_t* out_append;
    int32_t* out_lists;
    int32_t* out_len;
};

struct Strided {
    int64_t token, head;  // in elements
};

struct AppendArgs {
    const void* q;
    void* q_out;
    const void* k;
    const void* v;
    Strided qs, qo, ks, vs;
    int T, q_heads, heads, D;
    const int32_t* positions;
    const int32_t* slots;
    const double* freqs;
    int rot;
    float rope_scale;
    int interleaved;
    spec_kv_cache cache;
    uint32_t* out_status;
};

void launch_rows(const RowsArgs& a, hipStream_t stream);
void launch_append(const AppendArgs& a, int dtype, bool vec, hipStream_t stream);

}  // namespace kv
}  // namespace sv
