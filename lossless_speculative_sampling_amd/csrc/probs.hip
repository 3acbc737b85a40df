// Verification from given probabilities: the acceptance scan, the mass of the row the token t* is
// drawn from, and the draw by inverse CDF in token order.
//
// What bounds it: of each request's K + 1 pairs of rows only the pair of the first rejected
// position (or the target's row after the last accepted token) is read, once, for the masses of its
// cells; the draw re-reads one cell.  So the floor is two rows per request at HBM rate, and for
// few requests the chain of dependent loads (token, its two probabilities, the row).
//
// Measured: 512 requests of V = 151936 in bf16 66 us, the scan 60 (5.2 TB/s of the 5.6 a plain read of
// that size reaches) and the draw 7; 16 of V = 128256 in fp32 5.3 and 5.7 us; one of V = 1024 5.2 us.
// More cells per workgroup (8, 16: 2% and 8% more) and all of a workgroup's loads ahead of its sums (5%
// more) did not help, nor did cheaper arithmetic: it is bound by its reads.
//
// Every workgroup of a request repeats the scan (K gathers, one wave) instead of waiting for a
// launch of its own that would publish it.
//
// Masses are differences of fp32 (or narrower) values taken and summed in fp64: the differences
// are exact unless the two values are 2^29 apart, so the running mass compared with v times the
// total carries no rounding that matters and does not depend on how a row is cut.
#include <type_traits>

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
// (ONCE: read once, not to be kept in the caches)
template <bool ONCE, typename T>
__device__ __forceinline__ Eight<T> load8(const T* p) {
    typedef uint32_t words4 __attribute__((ext_vector_type(4), aligned(4)));
    typedef uint32_t words2 __attribute__((ext_vector_type(4), aligned(2)));
    typedef std::conditional_t<sizeof(T) == 4, words4, words2> words;
    words w[sizeof(Eight<T>) / 16];
#pragma unroll
    for (unsigned i = 0; i < sizeof(Eight<T>) / 16; ++i) 
        w[i] = ONCE ? __builtin_nontemporal_load(reinterpret_cast<const words*>(p) + i) : reinterpret_cast<const words*>(p)[i];
    Eight<T> e;
    __builtin_memcpy(&e, w, sizeof(e));
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
    template <bool ONCE>
    __device__ __forceinline__ void eight(int i, double (&w)[8]) const {
        if (i + 8 <= V) {
            const Eight<T> x = load8<ONCE>(q + i);
            Eight<T> y;
            if (p) y = load8<ONCE>(p + i);
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

// The thread's part of the mass of [lo, hi) (lo a multiple of kTile).
template <bool ONCE, typename T>
__device__ __forceinline__ double part_of_mass(const Row<T>& r, int64_t lo, int64_t hi) {
    double s = 0.0;
    for (int64_t t = lo; t < hi; t += kTile) {
        const int64_t i = t + (int64_t)threadIdx.x * 8;
        if (i < hi) {
            double w[8];
            r.template eight<ONCE>((int)i, w);
            s += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
        }
    }
    return s;
}

constexpr int kWaves = kThreads / kWave;
constexpr int kAhead = kOneLaunchV / kTile;  // most tiles a draw holds at once

struct DrawShared {
    double red[kWaves];
    double tot[kAhead][kWaves];
    int hit[kWaves], last[kWaves];
    int cell, found;
    double ahead;
};

struct Pick {
    int token;      // -1: no token of the range has mass
    double total;   // mass of the range
};

// The first token of [lo, hi) whose running mass, from `before` on, exceeds `at` (WHOLE: exceeds
// v times the range's own mass; the range is then at most A tiles); the last one with mass
// where none does (the running mass here and the sums `at` comes from may differ in their last
// bits).  A tiles are loaded at once, so that their loads do not wait for each other.
template <typename T, bool WHOLE, int A>
__device__ __forceinline__ Pick pick(const Row<T>& r, int lo, int hi, double before, double at_or_v, DrawShared& sh) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    double run = before, at = at_or_v, all = 0.0;
    int last = -1;
    for (int64_t t0 = lo; t0 < hi; t0 += A * kTile) {
        double w[A][8], prior[A];
#pragma unroll
        for (int q = 0; q < A; ++q) {
            const int64_t i = t0 + q * kTile + (int64_t)threadIdx.x * 8;
            if (i < hi) {
                r.template eight<false>((int)i, w[q]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) w[q][e] = 0.0;
            }
        }
        __syncthreads();  // the last round's (or caller's) words have been read
#pragma unroll
        for (int q = 0; q < A; ++q) {
            const double mine = ((w[q][0] + w[q][1]) + (w[q][2] + w[q][3])) + ((w[q][4] + w[q][5]) + (w[q][6] + w[q][7]));
            const double upto = wave_scan(mine, &prior[q]);
            if (lane == kWave - 1) sh.tot[q][wave] = upto;
        }
        __syncthreads();
        if (WHOLE) {
            all = 0.0;
#pragma unroll
            for (int q = 0; q < A; ++q)
#pragma unroll
                for (int v = 0; v < kWaves; ++v) all += sh.tot[q][v];
            at = at_or_v * all;
        }
        int hit = 0x7fffffff, mine_last = -1;
#pragma unroll
        for (int q = 0; q < A; ++q) {
            double c = run;
#pragma unroll
            for (int v = 0; v < kWaves; ++v) {
                const double x = sh.tot[q][v];
                if (v < wave) c += x;
                run += x;
            }
            c += prior[q];
            const int i = (int)(t0 + q * kTile) + (int)threadIdx.x * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                c += w[q][e];
                if (w[q][e] > 0.0) {
                    mine_last = i + e;
                    if (hit == 0x7fffffff && c > at) hit = i + e;
                }
            }
        }
        hit = wave_min(hit);
        mine_last = wave_max(mine_last);
        if (lane == 0) {
            sh.hit[wave] = hit;
            sh.last[wave] = mine_last;
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
            hit = sh.hit[v] < hit ? sh.hit[v] : hit;
            last = sh.last[v] > last ? sh.last[v] : last;
        }
        if (hit != 0x7fffffff) return Pick{hit, all};
    }
    return Pick{last, all};
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

// t* of a request whose residual is empty: p >= q everywhere, so t* ~ q_k over the whole row (never
// on a path that counts).
template <typename T>
__device__ __forceinline__ void draw_from_target(const Args& a, int b, const Decision& d, double v, DrawShared& sh) {
    const Row<T> r = row_of<T>(a, b, d.k, d.len, false);
    const double all = block_sum(part_of_mass<false>(r, 0, a.V), sh.red);
    if (!(all > 0.0 && all < __builtin_inf())) {
        emit(a, b, 0, -1, 0.0, d.status | SPEC_ST_BAD_PROB);
        return;
    }
    emit(a, b, d.k, pick<T, false, 1>(r, 0, a.V, 0.0, v * all, sh).token, 0.0, d.status | kStEmptyResidual);
}

// The requests nothing is drawn for, given the mass of the row to draw from.
__device__ __forceinline__ bool refused(const Args& a, int b, const Decision& d, double v, double total) {
    uint32_t why = 0u;
    if (d.k < 0) why = d.status;
    else if (!(v >= 0.0 && v <= 1.0)) why = d.status | kStBadParam;
    else if (!(total < __builtin_inf()) || (total == 0.0 && d.k >= d.len)) why = d.status | SPEC_ST_BAD_PROB;
    if (why) emit(a, b, 0, -1, 0.0, why);
    return why != 0u;
}

// The scan by the first wave, handed to the others.
template <typename T>
__device__ __forceinline__ Decision decide_for_all(const Args& a, int b, Decision* shared) {
    if (threadIdx.x < kWave) {
        const Decision d = decide<T>(a, b);
        if (threadIdx.x == 0) *shared = d;
    }
    __syncthreads();
    return *shared;
}

// Rows of at most kOneLaunchV tokens: one workgroup per request does all, the draw from the masses it
// holds in registers (V = 1024: 5.0 us, 15 in two launches).
template <typename T>
__global__ __launch_bounds__(kThreads) void probs_whole_kernel(Args a) {
    __shared__ DrawShared sh;
    __shared__ Decision shared;
    const int b = blockIdx.x;
    const double v = random_at(a.v, a.u64, b);
    const Decision d = decide_for_all<T>(a, b, &shared);
    Pick p{-1, 0.0};
    if (d.k >= 0) p = pick<T, true, kAhead>(row_of<T>(a, b, d.k, d.len, true), 0, a.V, 0.0, v, sh);
    if (refused(a, b, d, v, p.total)) return;
    if (p.total == 0.0) draw_from_target<T>(a, b, d, v, sh);
    else emit(a, b, d.k, p.token, d.k < d.len ? p.total : 0.0, d.status);
}

// One workgroup per (`per` cells, request): the scan, then the cells' masses.  ONCE for rows of more
// than the last cache holds in all (512 requests of V = 151936 in bf16 70.5 -> 66 us; 64 of 128256 in
// fp32, which it holds, 19 -> 20.5 us).
template <typename T, bool ONCE>
__global__ __launch_bounds__(kThreads) void probs_scan_kernel(Args a) {
    __shared__ double red[kCellsAtOnce][kWaves];
    __shared__ Decision shared;
    const int groups = (a.cells + a.per - 1) / a.per, b = blockIdx.x / groups, c0 = blockIdx.x % groups * a.per;
    const Decision d = decide_for_all<T>(a, b, &shared);
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    if (d.k >= 0) {
        const Row<T> r = row_of<T>(a, b, d.k, d.len, true);
#pragma unroll
        for (int q = 0; q < kCellsAtOnce; ++q) {
            if (q >= a.per) break;
            const int64_t lo = (int64_t)(c0 + q) * a.cell, hi = lo + a.cell;
            const double s = wave_sum(part_of_mass<ONCE>(r, lo, hi < a.V ? hi : a.V));
            if (lane == 0) red[q][wave] = s;
        }
    }
    __syncthreads();
    const int q = threadIdx.x;
    if (q < a.per && c0 + q < a.cells) {
        double s = 0.0;
        for (int w = 0; w < kWaves && d.k >= 0; ++w) s += red[q][w];
        a.sums[(size_t)b * a.cells + c0 + q] = s;
    }
    if (threadIdx.x == 0 && c0 == 0) a.recs[b] = Rec{d.k, d.len, d.status, 0};
}

// One workgroup per request: the cell the draw falls into, then the token within it.
template <typename T>
__global__ __launch_bounds__(kThreads) void probs_draw_kernel(Args a) {
    __shared__ DrawShared sh;
    const int b = blockIdx.x;
    const Rec rec = a.recs[b];
    const double v = random_at(a.v, a.u64, b);
    // running mass of the cells, four neighbours per thread (at most kMaxCells)
    double s[4], mine = 0.0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int c = threadIdx.x * 4 + e;
        s[e] = c < a.cells ? a.sums[(size_t)b * a.cells + c] : 0.0;
        mine += s[e];
    }
    if (threadIdx.x == 0) {
        sh.cell = 0x7fffffff;
        sh.found = -1;
    }
    double total;
    const double before = block_exclusive_scan(mine, sh.red, &total);
    const Decision d{rec.k, rec.len, rec.status};
    if (refused(a, b, d, v, total)) return;
    if (total == 0.0) {
        draw_from_target<T>(a, b, d, v, sh);
        return;
    }
    // the cell whose running mass first exceeds v times the total, or the last one with mass
    const double at = v * total;
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
    if (hit >= 0) atomicMin(&sh.cell, hit);
    if (last >= 0) atomicMax(&sh.found, last);
    __syncthreads();
    const int cell = sh.cell != 0x7fffffff ? sh.cell : sh.found;
    if ((int)threadIdx.x == cell / 4) {  // the thread that holds the cell says what comes before it
        double x = before;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if ((int)threadIdx.x * 4 + e < cell) x += s[e];
        sh.ahead = x;
    }
    __syncthreads();
    const int64_t lo = (int64_t)cell * a.cell, hi = lo + a.cell;
    const Row<T> r = row_of<T>(a, b, d.k, d.len, true);
    const Pick p = pick<T, false, 1>(r, (int)lo, (int)(hi < a.V ? hi : a.V), sh.ahead, at, sh);
    emit(a, b, d.k, p.token, d.k < d.len ? total : 0.0, d.status);
}

template <typename T>
static void launch_type(const Args& a, hipStream_t stream) {
    if (a.V <= kOneLaunchV) {
        hipLaunchKernelGGL(probs_whole_kernel<T>, dim3((unsigned)a.B), dim3(kThreads), 0, stream, a);
        return;
    }
    const unsigned groups = (unsigned)((a.cells + a.per - 1) / a.per) * (unsigned)a.B;
    const size_t bytes = (size_t)a.B * a.V * sizeof(T) * (a.draft ? 2 : 1);
    if (bytes > kCacheBytes)
        hipLaunchKernelGGL((probs_scan_kernel<T, true>), dim3(groups), dim3(kThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((probs_scan_kernel<T, false>), dim3(groups), dim3(kThreads), 0, stream, a);
    hipLaunchKernelGGL(probs_draw_kernel<T>, dim3((unsigned)a.B), dim3(kThreads), 0, stream, a);
}

void launch(const Args& a, int dtype, hipStream_t stream) {
    if (dtype == SPEC_FP32) launch_type<float>(a, stream);
    else if (dtype == SPEC_BF16) launch_type<__bf16>(a, stream);
    else launch_type<_Float16>(a, stream);
}

}  // namespace probs
}  // namespace sv
