// Draft-tree rows, and rotary positions with the append to the paged cache.
#include "kvcache.h"

namespace sv {
namespace kv {

// ------------------------------------------------------------------------------------------
// Draft-tree rows.  Every node walks to its root: once to find its depth and whether all of its
// path is part of the tree, once to write the path's slots from the far end.  One workgroup per
// request holds the tree in LDS (a hop then costs an LDS read instead of a trip to L2); bounded by
// the longest walk's latency for few requests (16 trees of 37 nodes: 3.2 us, most of it the launch), by
// the lists' write, row by row, for many (512 trees of 255 nodes, lists of 12: 9.7 us).
// ------------------------------------------------------------------------------------------

constexpr int kOutside = -2;  // parent of a node that is not part of the tree itself

__device__ __forceinline__ int parent_of(int token, int parent, int n) {
    return token < 0 || parent < -1 || parent >= n ? kOutside : parent;
}

template <bool LDS>
__global__ __launch_bounds__(kThreads) void tree_rows_kernel(RowsArgs a) {
    __shared__ int32_t lp[LDS ? kLdsNodes : 1], ls[LDS ? kLdsNodes : 1];
    const int b = blockIdx.x;
    const size_t base = (size_t)b * a.N;
    if (LDS) {
        for (int n = threadIdx.x; n < a.N; n += kThreads) {
            lp[n] = parent_of(a.tokens[base + n], a.parents[base + n], n);
            ls[n] = a.slots[base + n];
        }
        __syncthreads();
    }
    auto up = [&](int n) { return LDS ? lp[n] : parent_of(a.tokens[base + n], a.parents[base + n], n); };
    auto slot = [&](int n) { return LDS ? ls[n] : a.slots[base + n]; };
    const int ctx = a.ctx[b];
    for (int n = threadIdx.x; n < a.N; n += kThreads) {
        int depth = 0, x = n;  // a parent is below its child's index, so the walk ends
        while (x >= 0 && depth <= a.depth) {
            x = up(x);
            ++depth;
        }
        // x is -1 past a root; still a node where the path is longer than the lists
        const bool in = x == -1 && depth <= a.depth;
        int32_t* list = a.out_lists + (base + n) * a.depth;
        if (!in) depth = 0;
        a.out_pos[base + n] = in ? ctx + depth - 1 : -1;
        a.out_append[base + n] = in ? slot(n) : -1;
        a.out_len[base + n] = depth;
        x = n;
        for (int d = a.depth - 1; d >= 0; --d) {
            int32_t s = -1;
            if (d < depth) {
                s = slot(x);
                x = up(x);
            }
            list[d] = s;
        }
    }
}

void launch_rows(const RowsArgs& a, hipStream_t stream) {
    if (a.N <= kLdsNodes)
        hipLaunchKernelGGL(tree_rows_kernel<true>, dim3((unsigned)a.B), dim3(kThreads), 0, stream, a);
    else
        hipLaunchKernelGGL(tree_rows_kernel<false>, dim3((unsigned)a.B), dim3(kThreads), 0, stream, a);
}

// ------------------------------------------------------------------------------------------
// Rotary positions and the append.  A copy in which pairs of elements turn, so bounded by HBM for
// many tokens (16383 tokens with 32 query and 8 cache heads of 128 in bf16: 62 us, 6.5 TB/s; a copy of
// 4 GiB runs at 4.8) and by the launch for few (16 tokens: 3.9 us).  One workgroup per token: its threads take the angles
// first (each pair index once, for all heads): position * freq less its whole turns in fp64, because
// an fp32 angle of a position around 10^6 is off by 0.06; sin and cos of the remainder then need
// fp32 only.
// ------------------------------------------------------------------------------------------

constexpr double kTwoPi = 6.283185307179586232, kTwoPiLow = 2.4492935982947064e-16;
constexpr double kInvTwoPi = 0.15915494309189533577;
constexpr float kE4m3Most = 448.0f;

// fp32 to an 8-bit float: to nearest, ties to even, values past the range to its end, NaN kept.
__device__ __forceinline__ uint8_t to_e4m3(float x) {
    x = x > kE4m3Most ? kE4m3Most : (x < -kE4m3Most ? -kE4m3Most : x);
    return (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(x, 0.0f, 0, false) & 0xFF);
}

template <typename T>
struct Eight {
    T x[8];
};

// Eight elements from and to where whole vectors of them start.  What is read is read once and leaves
// the caches to what is written, which the attention reads next (16383 tokens: 86 us with ordinary
// loads, 62 so; non-temporal stores as well 65).
template <typename T>
__device__ __forceinline__ Eight<T> take(const T* p) {
    typedef uint32_t words __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(Eight<T>, __builtin_nontemporal_load(reinterpret_cast<const words*>(p)));
}
template <typename T>
__device__ __forceinline__ void put(T* p, const Eight<T>& x) {
    typedef uint32_t words __attribute__((ext_vector_type(sizeof(T) * 2)));
    *reinterpret_cast<words*>(p) = __builtin_bit_cast(words, x);
}

// The cache's element for a value: q's type as it is, 8 bits through the head's scale.
template <typename T, typename C>
struct Store;
template <typename T>
struct Store<T, T> {
    static __device__ __forceinline__ T value(float x, float) { return (T)x; }
};
template <typename T>
struct Store<T, uint8_t> {
    static __device__ __forceinline__ uint8_t value(float x, float scale) { return to_e4m3(x / scale); }
};

template <typename T>
__device__ __forceinline__ void turn(float x, float y, float c, float s, float& ox, float& oy) {
    ox = x * c - y * s;
    oy = y * c + x * s;
}

// One head of D elements: `item` < items_of() names either a vector of eight pairs (half layout:
// two vectors rot / 2 apart; interleaved: two neighbouring half-vectors are four pairs) or, past
// the rotated part, eight elements that pass through.
template <typename T, typename O>
__device__ __forceinline__ void vector_item(const T* in, O* out, int item, int rot, int interleaved, const float2* cs,
                                            float scale) {
    Eight<T> x;
    Eight<O> y;
    const int half = rot >> 1;
    const int turning = interleaved ? rot >> 3 : half >> 3;
    if (item < turning && !interleaved) {
        const int i = item * 8;
        Eight<T> x2;
        Eight<O> y2;
        x = take(in + i);
        x2 = take(in + half + i);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float a, b;
            turn<T>((float)x.x[e], (float)x2.x[e], cs[i + e].x, cs[i + e].y, a, b);
            y.x[e] = Store<T, O>::value(a, scale);
            y2.x[e] = Store<T, O>::value(b, scale);
        }
        put(out + i, y);
        put(out + half + i, y2);
        return;
    }
    const int i = interleaved ? item * 8 : rot + (item - turning) * 8;
    x = take(in + i);
    if (item < turning) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            float a, b;
            const float2 t = cs[(i + e) >> 1];
            turn<T>((float)x.x[e], (float)x.x[e + 1], t.x, t.y, a, b);
            y.x[e] = Store<T, O>::value(a, scale);
            y.x[e + 1] = Store<T, O>::value(b, scale);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) y.x[e] = Store<T, O>::value((float)x.x[e], scale);
    }
    put(out + i, y);
}

// The same element by element: `item` is a pair of the rotated part, or one element past it.
template <typename T, typename O>
__device__ __forceinline__ void scalar_item(const T* in, O* out, int item, int rot, int interleaved, const float2* cs,
                                            float scale) {
    const int half = rot >> 1;
    if (item < half) {
        const int i = interleaved ? 2 * item : item, j = interleaved ? i + 1 : i + half;
        float a, b;
        turn<T>((float)in[i], (float)in[j], cs[item].x, cs[item].y, a, b);
        out[i] = Store<T, O>::value(a, scale);
        out[j] = Store<T, O>::value(b, scale);
    } else {
        const int i = rot + item - half;
        out[i] = Store<T, O>::value((float)in[i], scale);
    }
}

template <typename T, typename C, bool VEC>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(AppendArgs a) {
    extern __shared__ float2 cs[];  // cos, sin of each pair, times the scale
    const int64_t t = blockIdx.x;
    const int half = a.rot >> 1;
    if (a.rot) {
        const double pos = (double)a.positions[t];
        for (int i = threadIdx.x; i < half; i += kThreads) {
            // angle - 2 pi n with 2 pi in two parts (the remainder is off by the product's rounding only)
            const double angle = pos * a.freqs[i];
            const double n = __builtin_rint(angle * kInvTwoPi);
            const double rest = fma(-n, kTwoPiLow, fma(-n, kTwoPi, angle));
            const float part = (float)(rest * kInvTwoPi);
            float s, c;
            sincospif(2.0f * part, &s, &c);
            cs[i] = make_float2(c * a.rope_scale, s * a.rope_scale);
        }
        __syncthreads();
    }
    const int32_t slot = a.slots ? a.slots[t] : -1;
    const int64_t all = (int64_t)a.cache.num_pages * a.cache.page_size;
    const bool stores = a.k && slot >= 0 && slot < all;
    if (a.out_status && threadIdx.x == 0)
        a.out_status[t] = slot >= -1 && (slot < 0 || slot < all) ? 0u : (uint32_t)SPEC_ST_BAD_SLOT;
    const int turned = VEC ? (a.interleaved ? a.rot >> 3 : half >> 3) : half;  // items of a rotated head
    const int per = turned + (VEC ? (a.D - a.rot) >> 3 : a.D - a.rot);
    const int flat = VEC ? a.D >> 3 : a.D;
    const int nq = a.q ? a.q_heads * per : 0;
    const int nk = stores ? a.heads * per : 0, nv = stores ? a.heads * flat : 0;
    int64_t at = 0;
    if (stores) at = (int64_t)(slot / a.cache.page_size) * a.cache.page_stride + (int64_t)(slot % a.cache.page_size) * a.cache.token_stride;
    for (int x = threadIdx.x; x < nq + nk + nv; x += kThreads) {
        if (x < nq) {
            const int h = x / per, i = x % per;
            const T* in = static_cast<const T*>(a.q) + t * a.qs.token + h * a.qs.head;
            T* out = static_cast<T*>(a.q_out) + t * a.qo.token + h * a.qo.head;
            if (VEC) vector_item<T, T>(in, out, i, a.rot, a.interleaved, cs, 1.0f);
            else scalar_item<T, T>(in, out, i, a.rot, a.interleaved, cs, 1.0f);
        } else if (x < nq + nk) {
            const int h = (x - nq) / per, i = (x - nq) % per;
            const T* in = static_cast<const T*>(a.k) + t * a.ks.token + h * a.ks.head;
            C* out = static_cast<C*>(a.cache.k) + at + h * a.cache.head_stride;
            const float scale = a.cache.k_scale ? a.cache.k_scale[h] : 1.0f;
            if (VEC) vector_item<T, C>(in, out, i, a.rot, a.interleaved, cs, scale);
            else scalar_item<T, C>(in, out, i, a.rot, a.interleaved, cs, scale);
        } else {
            const int h = (x - nq - nk) / flat, i = (x - nq - nk) % flat;
            const T* in = static_cast<const T*>(a.v) + t * a.vs.token + h * a.vs.head;
            C* out = static_cast<C*>(a.cache.v) + at + h * a.cache.head_stride;
            const float scale = a.cache.v_scale ? a.cache.v_scale[h] : 1.0f;
            if (VEC) vector_item<T, C>(in, out, i, 0, a.interleaved, cs, scale);
            else scalar_item<T, C>(in, out, i, 0, a.interleaved, cs, scale);
        }
    }
}

template <typename T, typename C>
static void launch_typed(const AppendArgs& a, bool vec, hipStream_t stream) {
    const size_t lds = (size_t)(a.rot / 2) * sizeof(float2);
    if (vec)
        hipLaunchKernelGGL((kv_append_kernel<T, C, true>), dim3((unsigned)a.T), dim3(kThreads), lds, stream, a);
    else
        hipLaunchKernelGGL((kv_append_kernel<T, C, false>), dim3((unsigned)a.T), dim3(kThreads), lds, stream, a);
}

void launch_append(const AppendArgs& a, int dtype, bool vec, hipStream_t stream) {
    const bool eight = a.k && a.cache.dtype == SPEC_E4M3;
    if (dtype == SPEC_BF16) {
        if (eight) launch_typed<__bf16, uint8_t>(a, vec, stream);
        else launch_typed<__bf16, __bf16>(a, vec, stream);
    } else {
        if (eight) launch_typed<_Float16, uint8_t>(a, vec, stream);
        else launch_typed<_Float16, _Float16>(a, vec, stream);
    }
}

}  // namespace kv
}  // namespace sv
