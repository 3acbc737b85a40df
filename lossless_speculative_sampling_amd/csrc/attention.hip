// Attention of rows that share a long prefix of the paged cache.
//
// One wave per (row, query head): the wave walks the row's tokens with a running maximum and sum,
// its lanes spread over the head's elements.  Right for every case, and slow: every row reads the
// prefix again.
#include "attention.h"

namespace sv {
namespace attn {

template <typename C>
__device__ __forceinline__ float cached(const void* p, int64_t i) {
    return (float)static_cast<const C*>(p)[i];
}
template <>
__device__ __forceinline__ float cached<uint8_t>(const void* p, int64_t i) {
    return __builtin_amdgcn_cvt_f32_fp8((int)static_cast<const uint8_t*>(p)[i], 0);
}

// The group of row r: the largest g with row_start[g] <= r, or -1 outside every group.
__device__ __forceinline__ int group_of(const Args& a, int r) {
    int lo = -1, hi = a.G;  // row_start[lo] <= r < row_start[hi], with fences at either end
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.row_start[mid] <= r) lo = mid;
        else hi = mid;
    }
    return lo >= 0 && r < a.row_start[lo + 1] ? lo : -1;
}

template <typename T, typename C>
__global__ __launch_bounds__(kWave) void attention_kernel(Args a) {
    constexpr int kPer = kMaxD / kWave;
    const int r = blockIdx.x, h = blockIdx.y, lane = threadIdx.x;
    const int g = group_of(a, r);
    if (g < 0) return;
    const int kvh = h / a.per;
    const int page = a.cache.page_size;
    float q[kPer], o[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int d = lane + e * kWave;
        q[e] = d < a.D ? (float)static_cast<const T*>(a.q)[r * a.q_row + h * a.q_head + d] : 0.0f;
        o[e] = 0.0f;
    }
    const float ks = a.cache.k_scale ? a.cache.k_scale[kvh] : 1.0f, vs = a.cache.v_scale ? a.cache.v_scale[kvh] : 1.0f;
    const int64_t slots = (int64_t)a.cache.num_pages * page;
    const int64_t most = (int64_t)a.max_pages * page;
    int64_t L = a.max_pages ? a.prefix_len[g] : 0;
    L = L < 0 ? 0 : (L > most ? most : L);
    int S = a.max_suffix ? a.suffix_len[r] : 0;
    S = S < 0 ? 0 : (S > a.max_suffix ? a.max_suffix : S);
    float m = -__builtin_inff(), l = 0.0f;
    for (int64_t t = 0; t < L + S; ++t) {
        int64_t slot;
        if (t < L) {
            const int64_t id = a.table[(int64_t)g * a.max_pages + t / page];
            slot = id >= 0 && id < a.cache.num_pages ? id * page + t % page : -1;
        } else {
            slot = a.lists[(int64_t)r * a.max_suffix + (t - L)];
        }
        if (slot < 0 || slot >= slots) continue;
        const int64_t at = slot / page * a.cache.page_stride + slot % page * a.cache.token_stride + (int64_t)kvh * a.cache.head_stride;
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int d = lane + e * kWave;
            if (d < a.D) s += q[e] * cached<C>(a.cache.k, at + d);
        }
        s = wave_sum(s) * ks * a.scale;
        if (s == -__builtin_inff()) continue;
        const float top = s > m ? s : (s == s ? m : s);
        const float keep = m == -__builtin_inff() ? 0.0f : expf(m - top), w = expf(s - top);
        l = l * keep + w;
        m = top;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int d = lane + e * kWave;
            o[e] = o[e] * keep + (d < a.D ? w * cached<C>(a.cache.v, at + d) : 0.0f);
        }
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        const int d = lane + e * kWave;
        if (d < a.D) static_cast<T*>(a.out)[r * a.out_row + h * a.out_head + d] = (T)(l == 0.0f ? 0.0f : o[e] * vs / l);
    }
    if (a.lse && lane == 0) a.lse[(int64_t)r * a.q_heads + h] = l == 0.0f ? -__builtin_inff() : m + logf(l);
}

template <typename T, typename C>
static void launch_typed(const Args& a, hipStream_t stream) {
    hipLaunchKernelGGL((attention_kernel<T, C>), dim3((unsigned)a.R, (unsigned)a.q_heads), dim3(kWave), 0, stream, a);
}

void launch(const Args& a, int dtype, hipStream_t stream) {
    const bool eight = a.cache.dtype == SPEC_E4M3;
    if (dtype == SPEC_BF16) {
        if (eight) launch_typed<__bf16, uint8_t>(a, stream);
        else launch_typed<__bf16, __bf16>(a, stream);
    } else {
        if (eight) launch_typed<_Float16, uint8_t>(a, stream);
        else launch_typed<_Float16, _Float16>(a, stream);
    }
}

}  // namespace attn
}  // namespace sv
