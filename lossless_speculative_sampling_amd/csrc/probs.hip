// Verification from given probabilities: the acceptance scan, the mass of the row the token t* is
// drawn from, and the draw by inverse CDF in token order.
//
// What bounds it: of each request's K + 1 pairs of rows only the pair of the first rejected
// position (or the target's row after the last accepted token) is read, once, for the chunk
// masses; the draw re-reads one chunk.  So the floor is two rows per request at HBM rate, and for
// few requests the chain of dependent loads (token, its two probabilities, the row).
//
// Every workgroup of a request repeats the scan (K gathers, one wave) instead of waiting for a
// launch of its own that would publish it.
//
// Masses are differences of fp32 (or narrower) values taken and summed in fp64: the differences
// are exact unless the two values are 2^29 apart, so the running mass compared with v times the
// total carries no rounding that matters and does not depend on how a row is cut.
#include "probs.h"

namespace sv {
namespace probs {

template <typename T>
__device__ __forceinline__ float widen(T x) {
    return (float)x;
}

// Eight elements from an address with the element's alignment only.
template <typename T>
struct Eight {
    T x[8];
};
template <typename T>
__device__ __forceinline__ Eight<T> load8(const T* p) {
    Eight<T> e;
    __builtin_memcpy(&e, p, sizeof(e));
    return e;
}

__device__ __forceinline__ double random_at(const void* p, int u64, size_t i) {
    return u64 ? static_cast<const double*>(p)[i] : (double)static_cast<const float*>(p)[i];
}

struct Decision {
    int k;            // accepted tokens; -1: bad request
    int len;
    uint32_t status;
};

// A probability that may enter a sum: not negative, not NaN, not infinite.
__device__ __forceinline__ bool fine(float x) { return x >= 0.0f && x < __builtin_inff(); }

// The scan of request b by one whole wave: 64 positions at a time, each lane one position.
template <typename T>
__device__ __forceinline__ Decision decide(const Args& a, int b) {
    const int lane = threadIdx.x & (kWave - 1);
    Decision d{0, a.lens ? a.lens[b] : a.K, 0u};
    if (d.len < 0 || d.len > a.K) return Decision{-1, 0, kStBadParam};
    const T* p = static_cast<const T*>(a.draft) + (a.draft ? (int64_t)b * a.draft_req : 0);
    const T* q = static_cast<const T*>(a.target) + (int64_t)b * a.target_req;
    for (int j0 = 0; j0 < d.len; j0 += kWave) {
        const int j = j0 + lane;
        uint32_t bad = 0u;
        bool accept = false, outside = false;
        if (j < d.len) {
            const int s = a.tokens[(size_t)b * a.K + j];
            const double u = random_at(a.u, a.u64, (size_t)b * a.K + j);
            if (s < 0 || s >= a.V) {
                bad = kStBadToken;
            } else {
                const float qs = widen(q[(int64_t)j * a.target_row + s]);
                double ps = 1.0;
                if (a.flags & SPEC_UNIFORM_DRAFT) {
                    ps = 1.0 / (double)a.V;
                } else if (!(a.flags & SPEC_POINT_DRAFT)) {
                    const float x = widen(p[(int64_t)j * a.draft_row + s]);
                    ps = (double)x;
                    outside = x == 0.0f;
                    if (!fine(x)) bad = SPEC_ST_BAD_PROB;
                }
                if (!fine(qs)) bad = SPEC_ST_BAD_PROB;
                if (!(u >= 0.0 && u <= 1.0)) bad = kStBadParam;
                accept = bad == 0u && u * ps < (double)qs;
            }
        }
        const uint64_t stops = __ballot(j < d.len && !accept);
        const int first = stops ? __builtin_ctzll(stops) : kWave;  // lanes up to it were reached
        if (__ballot(outside && lane <= first)) d.status |= kStOutside;
        if (first < kWave) {
            const uint32_t why = (uint32_t)__builtin_amdgcn_readlane((int)bad, first);
            if (why) return Decision{-1, d.len, d.status | why};
            d.k = j0 + first;
            return d;
        }
    }
    d.k = d.len;
    return d;
}

// The masses of eight neighbouring tokens of the row t* is drawn from; NaN marks a bad value.
template <typename T>
struct Row {
    const T* q;
    const T* p;      // null: no draft row enters
    int point;       // token that had probability 1 (-1: none)
    double flat;     // probability of every token of a uniform draft (0: none)
    int V;

    __device__ __forceinline__ double mass(float x, float y, int i) const {
        if (!fine(x) || !fine(y)) return __builtin_nan("");
        const double w = (double)x - (double)y - flat - (i == point ? 1.0 : 0.0);
        return w > 0.0 ? w : 0.0;
    }
    __device__ __forceinline__ void eight(int i, double (&w)[8]) const {
        if (i + 8 <= V) {
            const Eight<T> x = load8(q + i);
            Eight<T> y;
            if (p) y = load8(p + i);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = mass(widen(x.x[e]), p ? widen(y.x[e]) : 0.0f, i + e);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                w[e] = i + e < V ? mass(widen(q[i + e]), p ? widen(p[i + e]) : 0.0f, i + e) : 0.0;
        }
    }
};

template <typename T>
__device__ __forceinline__ Row<T> row_of(const Args& a, int b, int k, int len, bool residual) {
    Row<T> r;
    r.q = static_cast<const T*>(a.target) + (int64_t)b * a.target_req + (int64_t)k * a.target_row;
    r.p = nullptr;
    r.point = -1;
    r.flat = 0.0;
    r.V = a.V;
    if (residual && k < len) {
        if (a.flags & SPEC_UNIFORM_DRAFT) r.flat = 1.0 / (double)a.V;
        else if (a.flags & SPEC_POINT_DRAFT) r.point = a.tokens[(size_t)b * a.K + k];
        else r.p = static_cast<const T*>(a.draft) + (int64_t)b * a.draft_req + (int64_t)k * a.draft_row;
    }
    return r;
}

// Mass of [lo, hi) (lo a multiple of kTile), in every thread.
template <typename T>
__device__ __forceinline__ double range_mass(const Row<T>& r, int lo, int hi, double* red) {
    double s = 0.0;
    for (int64_t t = lo; t < hi; t += kTile) {
        const int64_t i = t + (int64_t)threadIdx.x * 8;
        if (i < hi) {
            double w[8];
            r.eight((int)i, w);
            s += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
        }
    }
    return block_sum(s, red);
}

// The first token of [lo, hi) whose running mass, from `before` on, exceeds `at`; the last one with
// mass where none does (the running mass here and the sums `at` comes from may differ in their
// last bits); -1 where none has mass.
template <typename T>
__device__ __forceinline__ int pick(const Row<T>& r, int lo, int hi, double before, double at, double* red, int* found) {
    double run = before;
    if (threadIdx.x == 0) found[0] = 0x7fffffff, found[1] = -1;
    for (int64_t t = lo; t < hi; t += kTile) {
        const int64_t i = t + (int64_t)threadIdx.x * 8;
        double w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (i < hi) r.eight((int)i, w);
        double mine = 0.0;
        int last = -1;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            mine += w[e];
            if (w[e] > 0.0) last = (int)i + e;
        }
        double total;
        const double prior = block_exclusive_scan(mine, red, &total);  // its barriers order `found` too
        if (last >= 0) atomicMax(&found[1], last);
        double c = run + prior;
        int hit = -1;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            c += w[e];
            if (hit < 0 && w[e] > 0.0 && c > at) hit = (int)i + e;
        }
        if (hit >= 0) atomicMin(&found[0], hit);
        __syncthreads();
        if (found[0] != 0x7fffffff) break;
        run += total;
    }
    __syncthreads();
    const int f = found[0], l = found[1];
    __syncthreads();
    return f != 0x7fffffff ? f : l;
}

__device__ __forceinline__ void emit(const Args& a, int b, int k, int t, double mass, uint32_t status) {
    if (threadIdx.x == 0) {
        a.out_k[b] = k;
        a.out_tstar[b] = t;
        if (a.out_mass) a.out_mass[b] = (float)mass;
        if (a.out_status) a.out_status[b] = status;
    }
    if (a.out_emitted)
        for (int j = threadIdx.x; j <= a.K; j += kThreads)
            a.out_emitted[(size_t)b * (a.K + 1) + j] = t >= 0 && j < k ? a.tokens[(size_t)b * a.K + j] : (j == k ? t : -1);
}

// The draw of request b given its chunk masses (in LDS or global memory) by a whole workgroup.
template <typename T>
__device__ __forceinline__ void draw(const Args& a, int b, int k, int len, uint32_t status, const double* sums, double* red, int* found) {
    if (k < 0) {
        emit(a, b, 0, -1, 0.0, status);
        return;
    }
    // running mass of the chunks, four neighbours per thread
    double s[4], mine = 0.0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int c = threadIdx.x * 4 + e;
        s[e] = c < a.chunks ? sums[c] : 0.0;
        mine += s[e];
    }
    double total;
    const double before = block_exclusive_scan(mine, red, &total);
    const double v = random_at(a.v, a.u64, b);
    const bool rejected = k < len;
    if (!(v >= 0.0 && v <= 1.0)) {
        emit(a, b, 0, -1, 0.0, status | kStBadParam);
        return;
    }
    if (!(total < __builtin_inf()) || (total == 0.0 && !rejected)) {
        emit(a, b, 0, -1, 0.0, status | SPEC_ST_BAD_PROB);
        return;
    }
    Row<T> r = row_of<T>(a, b, k, len, true);
    int t;
    if (total == 0.0) {  // p >= q everywhere: t* ~ q_k, over the whole row (never on a path that counts)
        r = row_of<T>(a, b, k, len, false);
        const double all = range_mass(r, 0, a.V, red);
        if (!(all > 0.0 && all < __builtin_inf())) {
            emit(a, b, 0, -1, 0.0, status | SPEC_ST_BAD_PROB);
            return;
        }
        status |= kStEmptyResidual;
        t = pick(r, 0, a.V, 0.0, v * all, red, found);
    } else {
        const double at = v * total;
        // the chunk whose running mass first exceeds `at`, or the last one with mass
        __syncthreads();
        if (threadIdx.x == 0) found[0] = 0x7fffffff, found[1] = -1;
        __syncthreads();
        double c = before;
        int hit = -1, last = -1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            c += s[e];
            if (s[e] > 0.0) {
                last = threadIdx.x * 4 + e;
                if (hit < 0 && c > at) hit = last;
            }
        }
        if (hit >= 0) atomicMin(&found[0], hit);
        if (last >= 0) atomicMax(&found[1], last);
        __syncthreads();
        const int chunk = found[0] != 0x7fffffff ? found[0] : found[1];
        // the thread that holds the chunk says what came before it
        if (threadIdx.x == chunk / 4) {
            double x = before;
            for (int e = 0; e < 4; ++e)
                if (threadIdx.x * 4 + e < chunk) x += s[e];
            red[0] = x;
        }
        __syncthreads();
        const double ahead = red[0];
        __syncthreads();
        const int64_t lo = (int64_t)chunk * a.chunk, hi = lo + a.chunk;
        t = pick(r, (int)lo, (int)(hi < a.V ? hi : a.V), ahead, at, red, found);
    }
    emit(a, b, k, t, rejected ? total : 0.0, status);
}

// One workgroup per (chunk, request): the scan, then the chunk's mass.  With one chunk per row the
// same workgroup draws as well.
template <typename T>
__global__ __launch_bounds__(kThreads) void probs_scan_kernel(Args a) {
    __shared__ double red[kThreads / kWave];
    __shared__ int found[2];
    __shared__ Decision shared;
    const int b = blockIdx.x / a.chunks, c = blockIdx.x % a.chunks;
    if (threadIdx.x < kWave) {
        const Decision d = decide<T>(a, b);
        if (threadIdx.x == 0) shared = d;
    }
    __syncthreads();
    const Decision d = shared;
    double s = 0.0;
    if (d.k >= 0) {
        const int64_t lo = (int64_t)c * a.chunk, hi = lo + a.chunk;
        s = range_mass(row_of<T>(a, b, d.k, d.len, true), (int)lo, (int)(hi < a.V ? hi : a.V), red);
    }
    if (a.chunks == 1) {
        draw<T>(a, b, d.k, d.len, d.status, &s, red, found);
        return;
    }
    if (threadIdx.x == 0) {
        a.sums[(size_t)b * a.chunks + c] = s;
        if (c == 0) a.recs[b] = Rec{d.k, d.len, d.status, 0};
    }
}

// One workgroup per request: the chunk the draw falls into, then the token within it.
template <typename T>
__global__ __launch_bounds__(kThreads) void probs_draw_kernel(Args a) {
    __shared__ double red[kThreads / kWave];
    __shared__ int found[2];
    const int b = blockIdx.x;
    const Rec r = a.recs[b];
    draw<T>(a, b, r.k, r.len, r.status, a.sums + (size_t)b * a.chunks, red, found);
}

template <typename T>
static void launch_type(const Args& a, hipStream_t stream) {
    hipLaunchKernelGGL(probs_scan_kernel<T>, dim3((unsigned)a.chunks * (unsigned)a.B), dim3(kThreads), 0, stream, a);
    if (a.chunks > 1) hipLaunchKernelGGL(probs_draw_kernel<T>, dim3((unsigned)a.B), dim3(kThreads), 0, stream, a);
}

void launch(const Args& a, int dtype, hipStream_t stream) {
    if (dtype == SPEC_FP32) launch_type<float>(a, stream);
    else if (dtype == SPEC_BF16) launch_type<__bf16>(a, stream);
    else launch_type<_Float16>(a, stream);
}

}  // namespace probs
}  // namespace sv
