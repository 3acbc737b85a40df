// Attention of rows that share a long prefix: launch arguments shared by the C ABI and the kernels.
#pragma once

#include "common.h"

namespace sv {
namespace attn {

constexpr int kMaxD = 256;

struct Args {
    const void* q;
    int64_t q_row, q_head;
    int R, q_heads, heads, D, per;  // per = q_heads / heads
    spec_kv_cache cache;
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
};

void launch(const Args& a, int dtype, hipStream_t stream);

}  // namespace attn
}  // namespace sv
