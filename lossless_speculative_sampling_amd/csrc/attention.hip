// Attention of rows that share a long prefix of the paged cache.
//
// out = sum_t softmax_t(scale q . k_t) v_t over a prefix that all rows of a group see and a list
// of slots of each row's own.  Two launches:
//
// 1. pieces.  The queries of a group that use one cache head (row by row, the heads of a row
//    together) form tiles; a piece is a tile against a stretch of the prefix.  Every key and value
//    of the stretch goes through LDS once for the whole tile.  The stretch's length is the same
//    for all groups and chosen on the device from their lengths, so that the pieces of a ragged
//    batch are alike and about as many as the card holds at once.  Further workgroups of the same
//    launch take the suffix lists, one wave per row and cache head.
// 2. join.  A row's pieces and its suffix are joined by their maxima and sums.
//
// Within a piece the scores are taken transposed, S^T = K Q^T: a lane then holds scores of one
// query (its column), so the running maximum and sum need no exchange between lanes, and the
// weights lie as the second product O^T = V^T P^T wants its right operand, so they go from one
// matrix instruction to the next within the lane's registers.  (The order of the 32 keys inside
// that product is free as long as both operands agree; it is the order the first product leaves.)
// V^T comes out of LDS by the transposing read.
//
// The reference exponent of a query is moved only when a score exceeds it by more than 2^8:
// weights stay below 2^8, where nothing is lost in fp32 sums nor, relatively, in the 16 bits of
// the second product's operand, and nearly every step needs neither the exchange between lanes
// nor the scaling of the output.
// Bound by reading the cache once where a group has up to 64 or so queries per cache head (six rows
// over 131071 tokens in e4m3: the pieces 54 us, 5.0 TB/s; 16 groups of 16 queries per cache head over
// 6144 tokens in bf16: 73 us in all, 5.5 TB/s; a plain read reaches 5.6); by the products and the exponentials
// beyond (128 queries: 104 to 108 us for the same; 320 per cache head over 8192 tokens: 150 us, 570 TFLOP/s).
// Matrix and vector instructions of two or three waves per SIMD share the time there: of 64 keys
// against 32 queries a wave spends 1024 cycles in the matrix cores and about 1250 in the vector unit.
#include "attention.h"

namespace sv {
namespace attn {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.69314718055994531f;
constexpr float kNone = -3.0e38f;  // reference exponent before any score
constexpr float kSlack = 8.0f;     // scores up to 2^8 over the reference leave it where it is

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// ------------------------------------------------------------------------------------------
// Matrix instructions and element types
// ------------------------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ f32x4 mma(s16x8 a, s16x8 b, f32x4 c);
template <>
__device__ __forceinline__ f32x4 mma<__bf16>(s16x8 a, s16x8 b, f32x4 c) {
    typedef __bf16 v __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v, a), __builtin_bit_cast(v, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x4 mma<_Float16>(s16x8 a, s16x8 b, f32x4 c) {
    typedef _Float16 v __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v, a), __builtin_bit_cast(v, b), c, 0, 0, 0);
}

template <typename T>
__device__ __forceinline__ s16x8 narrow8(const float (&x)[8]) {
    typedef T v __attribute__((ext_vector_type(8)));
    v r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = (T)x[e];
    return __builtin_bit_cast(s16x8, r);
}

// Eight cache elements as loaded, and as the matrix instructions take them.  An 8-bit float is
// exact in either 16-bit type; its scale enters the scores' factor and the output.
template <typename T, typename C>
struct Raw;
template <typename T>
struct Raw<T, T> {
    typedef u32x4 type;
    static __device__ __forceinline__ s16x8 widen(u32x4 x) { return __builtin_bit_cast(s16x8, x); }
};
template <typename T>
struct Raw<T, uint8_t> {
    typedef u32x2 type;
    static __device__ __forceinline__ s16x8 widen(u32x2 x) {
        uint32_t y[4];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            if constexpr (__is_same(T, __bf16)) {
                y[2 * w] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[w], 1.0f, false));
                y[2 * w + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[w], 1.0f, true));
            } else {
                y[2 * w] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x[w], 1.0f, false));
                y[2 * w + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x[w], 1.0f, true));
            }
        }
        return __builtin_bit_cast(s16x8, u32x4{y[0], y[1], y[2], y[3]});
    }
};

// max over the four lanes that hold one query's scores (lanes l, l ^ 16, l ^ 32, l ^ 48)
__device__ __forceinline__ float max_over_quarters(float x) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_over_quarters(float x) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// ------------------------------------------------------------------------------------------
// LDS tiles: rows of DP elements, 16-byte chunks exchanged within a row so that what one read takes
// at once (of keys one chunk of 16 rows, of values a pair of chunks of 8 rows) covers all banks.
// Two rows of 64 elements share a span of the banks, so there the row's second bit on counts.
// ------------------------------------------------------------------------------------------
template <int DP>
__device__ __forceinline__ int k_at(int key, int chunk) {
    return key * DP * 2 + ((chunk ^ (DP == 64 ? (key >> 1) & 7 : key & 15)) << 4);
}
template <int DP>
__device__ __forceinline__ int v_at(int key, int chunk) {
    return key * DP * 2 + ((chunk ^ (DP == 64 ? key & 6 : (key & 7) << 1)) << 4);
}

// The exchanges touch bits 4 to 7 of an address, chunks come in by exclusive or, so one address serves
// all reads of a row.  Kept opaque, or the compiler holds each of them in a register of its own
// through the loop, and those are worth more than an instruction.
__device__ __forceinline__ int again(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

__device__ __forceinline__ s16x4 transposed4(const char* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
}

// The running softmax of a wave's query blocks: lane l holds query l % 16 of each block, of the
// output the elements 16 b + 4 (l / 16) .. + 3 of every block b, of the sum its own keys' part (of the
// weights before their rounding: the log of the sum is an output too).
template <int MB, int DP>
struct State {
    f32x4 o[MB][DP / 16];
    float m[MB], l[MB];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            m[i] = kNone;
            l[i] = 0.0f;
#pragma unroll
            for (int b = 0; b < DP / 16; ++b) o[i][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
    }
};

// Scores of 32 keys (s[i][0]: keys 0..15, s[i][1]: 16..31; lane l has keys 4 (l / 16) .. + 3 of each)
// into weights, and the product with their values from `vl`.  `valid`: which keys exist.
template <typename T, int MB, int DP>
__device__ __forceinline__ void weigh(State<MB, DP>& st, f32x4 (&s)[MB][2], uint32_t valid, float c, const char* vl) {
    const int lane = threadIdx.x & (kWave - 1), g = lane >> 4, i = lane & 15;
    if (valid != 0xffffffffu) {
        const uint32_t mine = valid >> (g * 4);
#pragma unroll
        for (int n = 0; n < MB; ++n)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[n][kb][e] = (mine >> (kb * 16 + e)) & 1 ? s[n][kb][e] : -__builtin_inff();
    }
    float top[MB];
    bool up = false;
#pragma unroll
    for (int n = 0; n < MB; ++n) {
        // (the kind of maximum that passes NaN on: a query that meets one is NaN whatever its reference)
        float x = s[n][0][0];
#pragma unroll
        for (int e = 1; e < 8; ++e) x = __builtin_elementwise_maximum(x, s[n][e >> 2][e & 3]);
        top[n] = x * c;
        up = up || top[n] > st.m[n] + kSlack;
    }
    if (__any(up)) {
#pragma unroll
        for (int n = 0; n < MB; ++n) {
            const float m = fmaxf(st.m[n], max_over_quarters(top[n]));
            const float f = exp2_fast(st.m[n] - m);
            st.m[n] = m;
            st.l[n] *= f;
#pragma unroll
            for (int b = 0; b < DP / 16; ++b) st.o[n][b] *= f;
        }
    }
    s16x8 p[MB];
#pragma unroll
    for (int n = 0; n < MB; ++n) {
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = exp2_fast(fmaf(s[n][e >> 2][e & 3], c, -st.m[n]));
        p[n] = narrow8<T>(w);
        st.l[n] += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
    }
    // lane i of a quarter reads row 4 g + i / 4 at elements 4 (i % 4) .. + 3 of the block and gets
    // column i of the four rows
    const int base = again(v_at<DP>(g * 4 + (i >> 2), (i & 3) >> 1) + (i & 1) * 8);
#pragma unroll
    for (int b = 0; b < DP / 16; ++b) {
        const char* at = vl + (base ^ ((b & 7) << 5)) + (b >> 3) * 256;  // = v_at(.., 2 b + ..)
        const s16x4 lo = transposed4(at), hi = transposed4(at + 16 * DP * 2);
        const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
        for (int n = 0; n < MB; ++n) st.o[n][b] = mma<T>(v, p[n], st.o[n][b]);
        if (DP > 128 && b % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // few reads ahead: registers
    }
}

// A wave's query blocks against 32 keys of LDS.
template <typename T, int MB, int DP>
__device__ __forceinline__ void step(State<MB, DP>& st, const s16x8 (&q)[MB][DP / 32], uint32_t valid, float c, const char* kl,
                                     const char* vl) {
    const int lane = threadIdx.x & (kWave - 1);
    const int base = again(k_at<DP>(lane & 15, lane >> 4));
    f32x4 s[MB][2];
#pragma unroll
    for (int n = 0; n < MB; ++n) s[n][0] = s[n][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int kk = 0; kk < DP / 32; ++kk) {
            const s16x8 x = *reinterpret_cast<const s16x8*>(  // = k_at(16 kb + .., 4 kk + ..)
                kl + (base ^ ((kk & 3) << 6)) + (kk >> 2) * 256 + kb * 16 * DP * 2);
#pragma unroll
            for (int n = 0; n < MB; ++n) s[n][kb] = mma<T>(x, q[n][kk], s[n][kb]);
            if (DP > 128 && kk % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // few reads ahead: registers
        }
    weigh<T, MB, DP>(st, s, valid, c, vl);
}

// A cache slot's offset in elements, or -1 where there is no token.
__device__ __forceinline__ int64_t slot_offset(const Args& a, int64_t page, int in_page) {
    return page >= 0 && page < a.cache.num_pages ? page * a.cache.page_stride + in_page * a.cache.token_stride : -1;
}
__device__ __forceinline__ int64_t slot_offset(const Args& a, int slot) {
    const int page = slot >= 0 ? (a.page_shift >= 0 ? slot >> a.page_shift : slot / a.cache.page_size) : -1;
    return slot_offset(a, page, slot - page * a.cache.page_size);
}

__device__ __forceinline__ int prefix_of(const Args& a, int g) {
    const int64_t most = (int64_t)a.max_pages * a.cache.page_size;
    const int64_t n = a.max_pages ? a.prefix_len[g] : 0;
    return (int)(n < 0 ? 0 : (n > most ? most : n));
}

// Rows of group g within [0, R], first and number.
__device__ __forceinline__ int2 rows_of(const Args& a, int g) {
    int lo = a.row_start[g], hi = a.row_start[g + 1];
    lo = lo < 0 ? 0 : (lo > a.R ? a.R : lo);
    hi = hi > a.R ? a.R : hi;
    return make_int2(lo, hi > lo ? hi - lo : 0);
}

// The factor of the scores in powers of two.  A negative one goes into the queries' signs, so that
// the largest score stays the largest; zero is taken as next to nothing (masked scores are -inf).
__device__ __forceinline__ float factor_of(const Args& a, int kvh, bool* negate) {
    const float c = a.scale * (a.cache.k_scale ? a.cache.k_scale[kvh] : 1.0f) * kLog2e;
    *negate = c < 0.0f;
    const float size = fabsf(c);
    return size < 1e-37f ? 1e-37f : size;  // (NaN stays)
}

// 16 queries as the right operand of the first product: lane l has query l % 16, elements
// 32 kk + 8 (l / 16) .. + 7.
template <typename T, int DP>
__device__ __forceinline__ void load_queries(const Args& a, s16x8 (&q)[DP / 32], int row, int head, bool there, bool negate) {
    const int lane = threadIdx.x & (kWave - 1);
    const T* p = static_cast<const T*>(a.q) + (int64_t)row * a.q_row + (int64_t)head * a.q_head;
#pragma unroll
    for (int kk = 0; kk < DP / 32; ++kk) {
        const int d = kk * 32 + (lane >> 4) * 8;
        s16x8 x = {0, 0, 0, 0, 0, 0, 0, 0};
        if (there && d < a.D) x = *reinterpret_cast<const s16x8*>(p + d);
        if (negate) x ^= (short)0x8000;
        q[kk] = x;
    }
}

// ------------------------------------------------------------------------------------------
// Pieces of the prefix
// ------------------------------------------------------------------------------------------
struct Piece {
    int g, tile, begin, end;  // g < 0: none
    int first, rows;          // the group's rows
};

// What a group asks for, and where its pieces begin.
struct Share {
    int2 rows;
    int len, tiles, n;  // prefix, tiles, stretches
};

__device__ __forceinline__ Share share_of(const Args& a, int g, int mt) {
    Share s;
    s.rows = rows_of(a, g);
    s.len = prefix_of(a, g);
    s.tiles = (s.rows.y * a.per + mt - 1) / mt;
    s.n = 0;
    return s;
}

// The stretch: the groups' tiles times lengths over the pieces aimed at, less half a piece per tile
// for the stretches that end early.  (A little more than the quotient in any case: there is room for
// `want` pieces and one per tile.)
template <int KT>
__device__ __forceinline__ int stretch_of(const Args& a, long long work, long long tiles) {
    long long parts = a.want - tiles / 2;
    if (parts < a.want / 4) parts = a.want / 4;
    if (parts < 1) parts = 1;
    const float x = (float)work / (float)parts * 1.000001f + 1.0f;
    const int most = 0x7fffffff - 2 * KT;
    return (x < (float)most ? (int)x + KT - 1 : most) / KT * KT;
}

// Piece `k` of the group that `s` describes; its stretches are alike.
template <int KT>
__device__ __forceinline__ Piece piece_of(const Share& s, int g, int k) {
    Piece p;
    const int part = k / s.tiles;
    const int64_t each = (((int64_t)s.len + s.n - 1) / s.n + KT - 1) / KT * KT;
    const int64_t begin = part * each, end = begin + each;
    p.g = g;
    p.tile = k - part * s.tiles;
    p.begin = (int)(begin < s.len ? begin : s.len);
    p.end = (int)(end < s.len ? end : s.len);
    p.first = s.rows.x;
    p.rows = s.rows.y;
    return p;
}

__device__ __forceinline__ int stretches(const Share& s, int stretch) {
    return s.tiles ? (int)(((unsigned)s.len + stretch - 1u) / (unsigned)stretch) : 0;
}

// Every group's first piece and count, for more groups than a wave has lanes.
template <int MT, int KT>
__global__ __launch_bounds__(kThreads) void attention_plan_kernel(Args a) {
    __shared__ long long red64[kThreads / kWave];
    __shared__ int red[kThreads / kWave];
    long long work = 0, tiles = 0;
    for (int g = threadIdx.x; g < a.G; g += kThreads) {
        const Share s = share_of(a, g, MT);
        work += (long long)s.tiles * s.len;
        tiles += s.tiles;
    }
    work = block_sum(work, red64);
    tiles = block_sum(tiles, red64);
    const int stretch = stretch_of<KT>(a, work, tiles);
    int base = 0;
    for (int g0 = 0; g0 < a.G; g0 += kThreads) {
        const int g = g0 + threadIdx.x;
        Share s{make_int2(0, 0), 0, 0, 0};
        if (g < a.G) s = share_of(a, g, MT);
        s.n = stretches(s, stretch);
        int all;
        const int at = base + block_exclusive_scan(s.tiles * s.n, red, &all);
        if (g < a.G) a.groups[g] = make_int2(at, s.n);
        base += all;
    }
}

// Piece number x of a cache head, by every wave for itself.  Up to 64 groups lie in its lanes (the first
// workgroup leaves every group's first piece and count for the join); more are planned by a launch of
// their own, and the wave looks its group up, 64 ways at a time (2048 groups of 150 tokens: 597 us with
// every workgroup and every row going through all groups, 381 so).
template <int MT, int KT>
__device__ __forceinline__ Piece find_piece(const Args& a, int x, bool leave) {
    const int lane = threadIdx.x & (kWave - 1);
    if (a.G <= kWave) {
        Share s{make_int2(0, 0), 0, 0, 0};
        if (lane < a.G) s = share_of(a, lane, MT);
        s.n = stretches(s, stretch_of<KT>(a, wave_sum((long long)s.tiles * s.len), wave_sum(s.tiles)));
        int at;
        wave_scan(s.tiles * s.n, &at);
        if (leave && lane < a.G && threadIdx.x < kWave) a.groups[lane] = make_int2(at, s.n);
        const uint64_t mine = __ballot(x >= at && x < at + s.tiles * s.n);
        if (mine == 0) return Piece{-1, 0, 0, 0, 0, 0};
        const int g = __builtin_ctzll(mine);
        const Share t{make_int2(wave_bcast(s.rows.x, g), wave_bcast(s.rows.y, g)), wave_bcast(s.len, g), wave_bcast(s.tiles, g),
                      wave_bcast(s.n, g)};
        return piece_of<KT>(t, g, x - wave_bcast(at, g));
    }
    // the last group that begins at or before x
    int lo = 0, n = a.G;
    while (n > 1) {
        const int step = (n + kWave - 1) / kWave;
        const bool before = lane * step < n && a.groups[lo + lane * step].x <= x;
        const int c = __popcll(__ballot(before)) - 1;  // (the first always does)
        lo += c * step;
        n = n - c * step < step ? n - c * step : step;
    }
    const int g = __builtin_amdgcn_readfirstlane(lo);
    const int2 span = a.groups[g];
    Share s = share_of(a, g, MT);
    s.n = span.y;
    const auto one = [](int v) { return __builtin_amdgcn_readfirstlane(v); };  // scalar registers
    const int k = x - one(span.x);
    if (k >= one(s.tiles) * one(s.n)) return Piece{-1, 0, 0, 0, 0, 0};
    const Share t{make_int2(one(s.rows.x), one(s.rows.y)), one(s.len), one(s.tiles), one(s.n)};
    return piece_of<KT>(t, g, k);
}

// Keys a workgroup takes per step, as far as the registers that hold the next step's go: 32 for heads
// of 256, and for tiles of 128 queries, where the products bound the time and three workgroups per
// compute unit instead of two are worth more (320 queries per cache head over 8192 keys 190 -> 143 us;
// where reading bounds it, 128 queries over 6144, 112 -> 117 us).
constexpr int keys_of(int dp, int mb, int wq) { return dp > 128 || (dp == 128 && mb * wq == 8) ? 32 : 64; }
constexpr int groups_per_cu(int dp, int mb, int wq) { return dp == 128 && mb * wq == 8 ? 3 : 2; }

template <typename T, typename C, int DP, int MB, int WQ>
struct PieceLds {
    static constexpr int KT = keys_of(DP, MB, WQ);
    static constexpr int kTileBytes = KT * DP * 2;
    static constexpr int kWK = 4 / WQ;
    // the waves over the same queries meet in the same memory at the end
    static constexpr int kMeet = (kWK - 1) * WQ * MB * (16 * DP * 4 + 16 * 4 * 2);
    static constexpr int kBytes = 2 * kTileBytes > kMeet ? 2 * kTileBytes : kMeet;
};

template <typename T, typename C, int DP, int MB, int WQ>
__device__ __forceinline__ void prefix_piece(const Args& a, int index, char* lds) {
    typedef PieceLds<T, C, DP, MB, WQ> L;
    constexpr int KT = L::KT, WK = L::kWK, MT = 16 * MB * WQ;
    constexpr int kChunks = DP / 8;                    // 16-byte chunks of a row in LDS
    constexpr int kLoads = KT * kChunks / kThreads;    // of K, and of V, per thread
    constexpr int kStep = kThreads / kChunks;          // keys between a thread's loads
    typedef typename Raw<T, C>::type raw;
    __shared__ int64_t offs[2][KT];        // where a key lies (a key that does not exist: at the start)
    __shared__ uint32_t exists[2][KT / 32];  // which keys exist
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wq = wave % WQ, wk = wave / WQ;
    const int kvh = index % a.heads;
    const Piece pc = find_piece<MT, KT>(a, index / a.heads, index == 0);
    if (pc.g < 0) return;
    const int M = pc.rows * a.per;
    bool negate;
    const float c = factor_of(a, kvh, &negate);

    // the wave's query blocks, dealt out in turn so that a group that does not fill the tile still
    // occupies all waves
    s16x8 q[MB][DP / 32];
    State<MB, DP> st;
    st.clear();
    int nb = 0;
#pragma unroll
    for (int n = 0; n < MB; ++n) {
        const int base = pc.tile * MT + (n * WQ + wq) * 16, mq = base + (lane & 15);
        if (base < M) nb = n + 1;
        const bool there = mq < M;
        const int row = there ? mq / a.per : 0, h = there ? mq - row * a.per : 0;
        load_queries<T, DP>(a, q[n], pc.first + row, kvh * a.per + h, there, negate);
    }

    const int32_t* table = a.table + (int64_t)pc.g * a.max_pages;
    const int chunk = tid % kChunks, key0 = tid / kChunks;
    const bool inside = chunk * 8 < a.D;  // a chunk past head_dim is zero in LDS
    const int chunk0 = inside ? chunk * 8 : 0;
    raw kr[kLoads], vr[kLoads];

    // Where the keys of the step at t lie, by the first KT threads: the page is asked for ahead of the
    // keys and values loaded in the same step (loads return in order, so what waits for the page
    // does not wait for those), the offset is left in LDS after the step's products.
    auto page_of = [&](int t) {
        const int at = t + tid;
        return tid < KT && at < pc.end ? table[a.page_shift >= 0 ? at >> a.page_shift : at / a.cache.page_size] : -1;
    };
    auto leave = [&](int t, int page, int buf) {
        if (tid < KT) {
            const int at = t + tid;
            const int in_page = a.page_shift >= 0 ? at & (a.cache.page_size - 1) : at % a.cache.page_size;
            const int64_t o = slot_offset(a, page, in_page);
            offs[buf][tid] = (o < 0 ? 0 : o) * (int64_t)sizeof(C);
            const uint64_t there = __ballot(o >= 0);
            if ((lane & 31) == 0) exists[buf][tid >> 5] = (uint32_t)(there >> lane);
        }
    };
    // (of a key that does not exist the cache's first token is loaded: its score is masked, its value
    // zeroed on the way into LDS).  Non-temporal: a prefix is read once, or by its group's few tiles at
    // about the same time (512 single rows over up to 2000 tokens 598 -> 550 us, 16 groups of 16 queries
    // 82 -> 73; 64 groups of 64 queries whose 100 MB the last cache holds, 32.1 -> 33.1).
    const char* kc = reinterpret_cast<const char*>(static_cast<const C*>(a.cache.k) + (int64_t)kvh * a.cache.head_stride + chunk0);
    const char* vc = reinterpret_cast<const char*>(static_cast<const C*>(a.cache.v) + (int64_t)kvh * a.cache.head_stride + chunk0);
    auto load = [&](int buf) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int64_t o = offs[buf][key0 + j * kStep];
            kr[j] = __builtin_nontemporal_load(reinterpret_cast<const raw*>(kc + o));
            vr[j] = __builtin_nontemporal_load(reinterpret_cast<const raw*>(vc + o));
        }
    };
    char* kl = lds;
    char* vl = lds + L::kTileBytes;

    int page = page_of(pc.begin + KT);
    leave(pc.begin, page_of(pc.begin), 0);
    __syncthreads();
    load(0);
    leave(pc.begin + KT, page, 1);
    int buf = 0;
    for (int t = pc.begin; t < pc.end; t += KT, buf ^= 1) {
        // which keys exist (read before that is overwritten): the wave's own, and whether all do
        uint32_t valid[KT / (32 * WK)], all = 0xffffffffu;
#pragma unroll
        for (int w = 0; w < KT / 32; ++w) all &= __builtin_amdgcn_readfirstlane(exists[buf][w]);
#pragma unroll
        for (int sub = 0; sub < KT / (32 * WK); ++sub) valid[sub] = __builtin_amdgcn_readfirstlane(exists[buf][sub * WK + wk]);
        uint32_t mine = 0xffffffffu;  // of this thread's, by load
        if (all != 0xffffffffu) {
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int key = key0 + j * kStep;
                if (!((exists[buf][key >> 5] >> (key & 31)) & 1)) mine &= ~(1u << j);
            }
        }
        __syncthreads();  // the last step's tile has been read
        if (all != 0xffffffffu || a.D != DP) {
#pragma unroll
            for (int j = 0; j < kLoads; ++j)
                if (!inside || !((mine >> j) & 1)) kr[j] = vr[j] = raw{};
        }
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int key = key0 + j * kStep;
            *reinterpret_cast<s16x8*>(kl + k_at<DP>(key, chunk)) = Raw<T, C>::widen(kr[j]);
            *reinterpret_cast<s16x8*>(vl + v_at<DP>(key, chunk)) = Raw<T, C>::widen(vr[j]);
        }
        __syncthreads();
        if (t + KT < pc.end) {
            page = page_of(t + 2 * KT);
            load(buf ^ 1);
        }
#pragma unroll
        for (int sub = 0; sub < KT / (32 * WK); ++sub) {
            const int key = (sub * WK + wk) * 32;
            if (nb > 0 && valid[sub] != 0) step<T, MB, DP>(st, q, valid[sub], c, kl + key * DP * 2, vl + key * DP * 2);
        }
        leave(t + 2 * KT, page, buf);
    }
#pragma unroll
    for (int n = 0; n < MB; ++n) st.l[n] = sum_over_quarters(st.l[n]);

    // join the waves over different keys: all but the first leave theirs in LDS
    if constexpr (WK > 1) {
        __syncthreads();
        float* mo = reinterpret_cast<float*>(lds);
        float2* mm = reinterpret_cast<float2*>(lds + (WK - 1) * WQ * MB * 16 * DP * 4);
        if (wk > 0) {
#pragma unroll
            for (int n = 0; n < MB; ++n) {
                const int at = ((wk - 1) * WQ + wq) * MB + n;
                if (lane < 16) mm[at * 16 + lane] = make_float2(st.m[n], st.l[n]);
#pragma unroll
                for (int b = 0; b < DP / 16; ++b)
                    *reinterpret_cast<f32x4*>(mo + ((at * (DP / 16) + b) * 64 + lane) * 4) = st.o[n][b];
            }
        }
        __syncthreads();
        if (wk > 0) return;
#pragma unroll
        for (int n = 0; n < MB; ++n) {
#pragma unroll 1
            for (int w = 0; w < WK - 1; ++w) {
                const int at = (w * WQ + wq) * MB + n;
                const float2 ml = mm[at * 16 + (lane & 15)];
                const float m = fmaxf(st.m[n], ml.x);
                const float keep = exp2_fast(st.m[n] - m), f = exp2_fast(ml.x - m);
                st.m[n] = m;
                st.l[n] = st.l[n] * keep + ml.y * f;
#pragma unroll
                for (int b = 0; b < DP / 16; ++b)
                    st.o[n][b] = st.o[n][b] * keep + *reinterpret_cast<const f32x4*>(mo + ((at * (DP / 16) + b) * 64 + lane) * 4) * f;
            }
        }
    }
#pragma unroll
    for (int n = 0; n < MB; ++n) {
        const int in_tile = (n * WQ + wq) * 16 + (lane & 15);
        if (pc.tile * MT + in_tile >= M) continue;
        const int64_t at = (int64_t)index * MT + in_tile;
        if (lane < 16) a.piece_ml[at] = make_float2(st.m[n], st.l[n]);
#pragma unroll
        for (int b = 0; b < DP / 16; ++b) {
            const int d = b * 16 + (lane >> 4) * 4;
            if (d < a.D) *reinterpret_cast<f32x4*>(a.piece_o + at * a.D + d) = st.o[n][b];
        }
    }
}

// The group of row r, or -1, looked up by `width` lanes that share the row (a power of two; `lane` <
// width), as many ways at a time: the last group that begins at or before r, if it holds r.
__device__ __forceinline__ int group_of(const Args& a, int r, int lane, int width) {
    if (a.row_start[0] > r) return -1;
    int lo = 0, n = a.G;
    while (n > 1) {
        const int step = (n + width - 1) / width;
        const bool before = lane * step < n && a.row_start[lo + lane * step] <= r;
        const uint64_t set = __ballot(before) >> ((threadIdx.x & (kWave - 1)) - lane);
        const int c = __popcll(width < kWave ? set & ((1ull << width) - 1) : set) - 1;  // (the first always does)
        lo += c * step;
        n = n - c * step < step ? n - c * step : step;
    }
    return r < a.row_start[lo + 1] ? lo : -1;
}

// ------------------------------------------------------------------------------------------
// The suffix lists: one wave per (row, cache head, block of 16 of its query heads), 32 slots at a
// time.  Keys go from memory into the first product's operand as they lie; values through the
// wave's own part of LDS.
// ------------------------------------------------------------------------------------------
template <typename T, typename C, int DP>
__device__ __forceinline__ void suffix_wave(const Args& a, int64_t task, char* lds) {
    typedef typename Raw<T, C>::type raw;
    const int lane = threadIdx.x & (kWave - 1), g = lane >> 4, i = lane & 15;
    const int blocks = (a.per + 15) / 16;
    if (task >= (int64_t)a.R * a.heads * blocks) return;
    const int block = (int)(task % blocks), kvh = (int)(task / blocks % a.heads), r = (int)(task / blocks / a.heads);
    if (group_of(a, r, lane, kWave) < 0) return;
    int S = a.suffix_len[r];
    S = S < 0 ? 0 : (S > a.max_suffix ? a.max_suffix : S);
    const int32_t* list = a.lists + (int64_t)r * a.max_suffix;
    bool negate;
    const float c = factor_of(a, kvh, &negate);
    s16x8 q[1][DP / 32];
    const int h = block * 16 + i;
    load_queries<T, DP>(a, q[0], r, kvh * a.per + h, h < a.per, negate);
    const C* kc = static_cast<const C*>(a.cache.k) + (int64_t)kvh * a.cache.head_stride;
    const C* vc = static_cast<const C*>(a.cache.v) + (int64_t)kvh * a.cache.head_stride;
    State<1, DP> st;
    st.clear();
    for (int t = 0; t < S; t += 32) {
        // keys and values are asked for together, or 16 by 16 where that is too many registers; a slot
        // that holds no token and the elements past head_dim are read from where there are some, and
        // taken as zeros
        constexpr bool kTogether = DP <= 128;
        raw x[2][DP / 32], y[2][DP / 32];
        int64_t o[2];
        uint32_t valid = 0;
        const auto fetch = [&](const C* from, int kb, raw (&to)[DP / 32]) {
            const C* p = from + (o[kb] >= 0 ? o[kb] : 0);
#pragma unroll
            for (int kk = 0; kk < DP / 32; ++kk) {
                const int d = kk * 32 + g * 8;
                to[kk] = *reinterpret_cast<const raw*>(p + (d < a.D ? d : 0));
            }
        };
        const auto taken = [&](const raw& r, int kb, int kk) {
            const s16x8 w = Raw<T, C>::widen(r);
            return o[kb] >= 0 && kk * 32 + g * 8 < a.D ? w : s16x8{};
        };
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            const int at = t + kb * 16 + i;
            o[kb] = at < S ? slot_offset(a, list[at]) : -1;
            valid |= ((uint32_t)__ballot(o[kb] >= 0) & 0xffffu) << (kb * 16);
        }
        if (valid == 0) continue;
        if (kTogether) {
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                fetch(kc, kb, x[kb]);
                fetch(vc, kb, y[kb]);
            }
        }
        f32x4 s[1][2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            if (!kTogether) {
                __builtin_amdgcn_sched_barrier(0);
                fetch(kc, kb, x[kb]);
            }
            s[0][kb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int kk = 0; kk < DP / 32; ++kk) s[0][kb] = mma<T>(taken(x[kb][kk], kb, kk), q[0][kk], s[0][kb]);
            if (!kTogether) {
                __builtin_amdgcn_sched_barrier(0);
                fetch(vc, kb, y[kb]);
            }
#pragma unroll
            for (int kk = 0; kk < DP / 32; ++kk) {
                *reinterpret_cast<s16x8*>(lds + v_at<DP>(kb * 16 + i, kk * 4 + g)) = taken(y[kb][kk], kb, kk);
            }
        }
        __builtin_amdgcn_wave_barrier();
        weigh<T, 1, DP>(st, s, valid, c, lds);
        __builtin_amdgcn_wave_barrier();
    }
    const float sum = sum_over_quarters(st.l[0]);
    if (h >= a.per) return;
    const int64_t at = (int64_t)r * a.q_heads + kvh * a.per + h;
    if (g == 0) a.suffix_ml[at] = make_float2(st.m[0], sum);
#pragma unroll
    for (int b = 0; b < DP / 16; ++b) {
        const int d = b * 16 + g * 4;
        if (d < a.D) *reinterpret_cast<f32x4*>(a.suffix_o + at * a.D + d) = st.o[0][b];
    }
}

template <typename T, typename C, int DP, int MB, int WQ>
__global__ __launch_bounds__(kThreads, groups_per_cu(DP, MB, WQ)) void attention_pieces_kernel(Args a) {
    constexpr int kSuffixBytes = 4 * 32 * DP * 2;
    constexpr int kPieceBytes = PieceLds<T, C, DP, MB, WQ>::kBytes;
    __shared__ __align__(16) char lds[kPieceBytes > kSuffixBytes ? kPieceBytes : kSuffixBytes];
    const int pieces = a.slots * a.heads;
    if ((int)blockIdx.x < pieces) {
        prefix_piece<T, C, DP, MB, WQ>(a, blockIdx.x, lds);
    } else {
        const int wave = threadIdx.x >> 6;
        suffix_wave<T, C, DP>(a, (int64_t)(blockIdx.x - pieces) * 4 + wave, lds + wave * 32 * DP * 2);
    }
}

// ------------------------------------------------------------------------------------------
// The join: DP / 4 lanes per (row, query head), four elements each.  The lanes first take the
// maxima and sums, one part per lane, so that the parts' outputs can then be asked for without
// waiting for one another.  With few rows (`ways`) a whole workgroup shares one pair and each of
// its groups of lanes takes every kWays-th part.
// ------------------------------------------------------------------------------------------
template <typename T, int DP>
__global__ __launch_bounds__(kThreads) void attention_join_kernel(Args a, int mt, int shared) {
    constexpr int kLanes = DP / 4, kWays = kThreads / kLanes;
    __shared__ f32x4 meet[kWays][kLanes];
    const int lane = threadIdx.x % kLanes, set = threadIdx.x / kLanes;
    const int ways = shared ? kWays : 1, way = shared ? set : 0;
    const int64_t pair = shared ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * kWays + set;
    const bool there = pair < (int64_t)a.R * a.q_heads;
    const int r = there ? (int)(pair / a.q_heads) : 0, h = there ? (int)(pair % a.q_heads) : 0, kvh = h / a.per;
    const int g = there ? group_of(a, r, lane, kLanes) : -1;
    const int d = lane * 4;
    float m = kNone, l = 0.0f;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    if (g >= 0) {
        // part 0 is the suffix, then the pieces along the prefix
        const int first = a.max_suffix ? 1 : 0;
        int parts = first;
        int64_t at0 = 0, step = 0;
        if (a.slots) {
            const int2 rows = rows_of(a, g), span = a.groups[g];
            const int q = (r - rows.x) * a.per + h - kvh * a.per;
            const int tiles = (rows.y * a.per + mt - 1) / mt, tile = q / mt;
            at0 = ((int64_t)(span.x + tile) * a.heads + kvh) * mt + (q - tile * mt);
            step = (int64_t)tiles * a.heads * mt;
            // (there is room for all of them as long as row_start does not decrease)
            const int room = a.slots - span.x - tile;
            parts += room <= 0 ? 0 : min(span.y, (room - 1) / tiles + 1);
        }
        const auto ml_of = [&](int p) { return p < first ? a.suffix_ml[pair] : a.piece_ml[at0 + (p - first) * step]; };
        const auto o_of = [&](int p) { return (p < first ? a.suffix_o + pair * a.D : a.piece_o + (at0 + (p - first) * step) * a.D) + d; };
        for (int p = lane; p < parts; p += kLanes) {
            const float2 ml = ml_of(p);
            const float top = fmaxf(m, ml.x);
            l = l * exp2_fast(m - top) + ml.y * exp2_fast(ml.x - top);
            m = top;
        }
        float top = m;
#pragma unroll
        for (int s = 1; s < kLanes; s <<= 1) top = fmaxf(top, __shfl_xor(top, s));
        l *= exp2_fast(m - top);
#pragma unroll
        for (int s = 1; s < kLanes; s <<= 1) l += __shfl_xor(l, s);
        m = top;
        if (d < a.D) {
            int p = way;
            for (; p + 3 * ways < parts; p += 4 * ways) {
                f32x4 x[4];
                float f[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(o_of(p + e * ways)));
                    f[e] = ml_of(p + e * ways).x;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) o += x[e] * exp2_fast(f[e] - m);
            }
            for (; p < parts; p += ways) o += __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(o_of(p))) * exp2_fast(ml_of(p).x - m);
        }
    }
    if (shared) {
        meet[set][lane] = o;
        __syncthreads();
        if (set > 0 || g < 0) return;
#pragma unroll
        for (int w = 1; w < kWays; ++w) o += meet[w][lane];
    } else if (g < 0) {
        return;
    }
    if (d < a.D) {
        const float f = (a.cache.v_scale ? a.cache.v_scale[kvh] : 1.0f) / l;
        typedef T v4 __attribute__((ext_vector_type(4)));
        v4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = (T)(l == 0.0f ? 0.0f : o[e] * f);
        *reinterpret_cast<v4*>(static_cast<T*>(a.out) + (int64_t)r * a.out_row + (int64_t)h * a.out_head + d) = y;
    }
    if (a.lse && lane == 0) a.lse[pair] = l == 0.0f ? -__builtin_inff() : (m + log2f(l)) * kLn2;
}

template <typename T, typename C, int DP, int MB, int WQ>
static void launch_tile(const Args& a, hipStream_t stream) {
    if (a.slots && a.G > kWave)
        hipLaunchKernelGGL((attention_plan_kernel<16 * MB * WQ, keys_of(DP, MB, WQ)>), dim3(1), dim3(kThreads), 0, stream, a);
    const unsigned blocks = (unsigned)(a.slots * a.heads + a.suffix_blocks);
    if (blocks)
        hipLaunchKernelGGL((attention_pieces_kernel<T, C, DP, MB, WQ>), dim3(blocks), dim3(kThreads), 0, stream, a);
    // few rows against a long prefix have many pieces each: a workgroup per pair then
    const int64_t per = kThreads / (DP / 4), pairs = (int64_t)a.R * a.q_heads;
    const int shared = pairs <= 1024 && a.slots / a.G > 8;
    hipLaunchKernelGGL((attention_join_kernel<T, DP>), dim3((unsigned)(shared ? pairs : (pairs + per - 1) / per)),
                       dim3(kThreads), 0, stream, a, 16 * MB * WQ, shared);
}

template <typename T, typename C, int DP>
static void launch_head(const Args& a, const Tile& t, hipStream_t stream) {
    if constexpr (DP > 128) {
        launch_tile<T, C, DP, 1, 4>(a, stream);
    } else {
        if (t.mb == 1 && t.wq == 2) launch_tile<T, C, DP, 1, 2>(a, stream);
        else if (t.wq == 2) launch_tile<T, C, DP, 2, 2>(a, stream);
        else launch_tile<T, C, DP, 2, 4>(a, stream);
    }
}

template <typename T, typename C>
static void launch_typed(const Args& a, const Tile& t, hipStream_t stream) {
    if (a.D > 128) launch_head<T, C, 256>(a, t, stream);
    else if (a.D > 64) launch_head<T, C, 128>(a, t, stream);
    else launch_head<T, C, 64>(a, t, stream);
}

void launch(const Args& a, const Tile& t, int dtype, hipStream_t stream) {
    const bool eight = a.cache.dtype == SPEC_E4M3;
    if (dtype == SPEC_BF16) {
        if (eight) launch_typed<__bf16, uint8_t>(a, t, stream);
        else launch_typed<__bf16, __bf16>(a, t, stream);
    } else {
        if (eight) launch_typed<_Float16, uint8_t>(a, t, stream);
        else launch_typed<_Float16, _Float16>(a, t, stream);
    }
}

}  // namespace attn
}  // namespace sv
