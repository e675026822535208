// beam_kernel.cuh -- beam search's selection: per group of beams the K best
// continuations (beam i, column v) by c = score_i + x_iv - lse_i, best first, ties to the lower
// (beam, column).
//
// Two kernels.  The first reads every logit once: a CTA takes a run of one row's
// columns, tile by tile, and leaves the run's (m, d) normalizer state and its K
// best logits, best first.  Within a row c has the order of x, so a row's K best
// are all that can matter.  The second, one CTA per group, joins the runs' states
// into lse and ranks the runs' lists by c.
//
// A run's K best: a bound that at least K of the tile's values reach is the least
// of the maxima of K (or a few more) equal parts of the tile; the values that
// reach it (some K ln K) go to a list in shared memory and are ranked by counting.
// From then on a value has to pass the K-th of the list, which few do; every few
// tiles the list is ranked again.
//
// Exact choices.  Values of different beams compare through their lse, which the
// first kernel's fp32 sums give within eps (below).  Where two values of different
// beams next to one another in the order, up to the first that is not chosen,
// are nearer than both errors, the rows of these beams are summed again with the
// sampler's weights (38 bits, added as integers) and the order is taken from those
// sums in 64 bits.
#pragma once

#include "sample_kernel.cuh"

namespace os {
namespace beam {

using sample::key_value;
using sample::order_key;
using sample::widen;
using u64 = unsigned long long;

constexpr int kThreads = 256;   // of a run's CTA
constexpr int kPer = 16;        // columns per thread and tile
constexpr int kTile = kThreads * kPer;
constexpr int kChunk = 4;       // tiles between two looks at the list
constexpr int kList = 512;      // values that reach the bound; more go another way
constexpr int kMergeThreads = 512;
constexpr int kCandidates = 1024;
constexpr int kMaxBeams = 64;
constexpr int kMaxK = 64;
constexpr float kLog2e = 1.442695022e+00f;

struct BeamArgs {
    const void* x;
    const float* scores;           // [groups][beams]
    const unsigned char* ended;    // [groups][beams] or NULL
    float* out;                    // [groups][K]
    int* parents;
    int* tokens;
    u64* lists;                    // [groups * beams][runs][K]: keys, best first, 0 behind them
    float2* states;                // [groups * beams][runs]: m, d
    int64_t cols;
    int beams, K, runs;
    int64_t run_tiles;             // tiles of a run
    int pad;
    float eps;                     // bound of lse's error
};

// A live beam's candidates are its row's columns.
__device__ __forceinline__ bool has_row(const BeamArgs& a, int64_t row) {
    return a.scores[row] > -INFINITY && !(a.ended && a.ended[row]);
}

// value and column in one number: larger is better, no two alike, 0 is none
__device__ __forceinline__ u64 make_key(float x, int64_t col) {
    return (static_cast<u64>(order_key(x)) << 32) | (0xffffffffu - static_cast<uint32_t>(col));
}

__device__ __forceinline__ float ex2f(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// e^(x - m) for merges of states (accurate; m >= x, m may be +-inf)
__device__ __forceinline__ float factor(float x, float m) {
    return x == m ? 1.f : exp1(x - m);
}

// The best KP parts' least maximum; every thread gets it.  KP is a power of two
// of 8 to 64: the threads' maxima are joined in parts of kThreads / KP threads.
template <int KP, int THREADS, typename V, typename Max>
__device__ __forceinline__ V parts_bound(V v, V* sh, Max larger) {
    constexpr int kPart = THREADS / KP;
    static_assert(KP <= 64, "parts");
    const int tid = threadIdx.x;
    if constexpr (kPart <= 32) {
#pragma unroll
        for (int o = kPart / 2; o > 0; o >>= 1) v = larger(v, __shfl_xor_sync(kFullMask, v, o));
        if (tid % kPart == 0) sh[tid / kPart] = v;
    } else {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v = larger(v, __shfl_xor_sync(kFullMask, v, o));
        if (tid % 32 == 0) sh[tid / 32] = v;
        __syncthreads();
        // parts of several warps: their first ones' places take the maximum
        if (tid < KP)
            for (int i = 1; i < kPart / 32; ++i)
                sh[64 + tid] = i == 1 ? larger(sh[tid * (kPart / 32)], sh[tid * (kPart / 32) + 1])
                                      : larger(sh[64 + tid], sh[tid * (kPart / 32) + i]);
        sh += 64;
    }
    __syncthreads();
    V least = sh[(tid & 31) % KP];
    if (KP > 32) {
        const V other = sh[32 + (tid & 31) % (KP > 32 ? KP - 32 : 1)];
        least = larger(least, other) == least ? other : least;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const V other = __shfl_xor_sync(kFullMask, least, o);
        least = larger(least, other) == least ? other : least;
    }
    return least;
}

struct RunShared {
    u64 list[kList];
    u64 sorted[kMaxK];
    uint32_t bound[128];
    u64 best[kThreads / 32];
    float m[kThreads / 32], d[kThreads / 32];
    int count;
};

// Columns of the tile's thread, as 16-byte blocks: value i of the thread belongs
// to column col(i).  Rows start anywhere, so block 0 is the aligned one that the
// row's first column lies in; a block that the row covers in part is read by elements.
template <typename T>
struct Tile {
    static constexpr int kVec = 16 / sizeof(T);
    static constexpr int kBlocks = kPer / kVec;
    const T* row;
    int64_t cols, base;  // base: first column of the tile's block 0 (may be below 0)
    int head;            // columns between the row's start and the block boundary before it

    __device__ __forceinline__ int64_t col(int i) const {
        return base + (static_cast<int64_t>(i / kVec) * kThreads + threadIdx.x) * kVec + i % kVec;
    }
    __device__ __forceinline__ void fetch(uint4 (&w)[kBlocks]) const {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            const int64_t c = base + (static_cast<int64_t>(b) * kThreads + threadIdx.x) * kVec;
            if (c >= 0 && c + kVec <= cols) {
                asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(w[b].x), "=r"(w[b].y), "=r"(w[b].z), "=r"(w[b].w)
                             : "l"(row + c));
            } else {
                T e[kVec];
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    e[i] = c + i >= 0 && c + i < cols ? row[c + i] : T(-INFINITY);
                w[b] = *reinterpret_cast<const uint4*>(e);
            }
        }
    }
    static __device__ __forceinline__ void values(const uint4 (&w)[kBlocks], float (&v)[kPer]) {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            const T* e = reinterpret_cast<const T*>(&w[b]);
#pragma unroll
            for (int i = 0; i < kVec; ++i) v[b * kVec + i] = static_cast<float>(e[i]);
        }
    }
};

// NaN counts as -inf.
__device__ __forceinline__ void clean(float (&v)[kPer]) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) v[e] = fmaxf(v[e], -INFINITY);
}

// A tile's share of the row's normalizer state, in the thread: m, and d + lost.  Values
// that are no numbers are cleaned out of v.  Returns the values' maximum.
struct State {
    float m = -INFINITY, d = 0.f, lost = 0.f;

    static __device__ __forceinline__ float weights(const float (&v)[kPer], float up) {
        float part[4] = {};
        if (fabsf(up) < 1e30f) {
            // base-2 exponents with one rounding each, below the rounded maximum; the
            // factor between it and the maximum comes at once
            const float c = up * kLog2e;
#pragma unroll
            for (int e = 0; e < kPer; ++e) part[e & 3] += ex2f(fmaf(v[e], kLog2e, -c));
            return ((part[0] + part[1]) + (part[2] + part[3])) * ex2f(fmaf(up, -kLog2e, c));
        }
        // a maximum of +-inf or near the largest number
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            part[e & 3] += v[e] == up ? 1.f : ex2f((v[e] - up) * kLog2e);
        return (part[0] + part[1]) + (part[2] + part[3]);
    }
    __device__ __forceinline__ float add(float (&v)[kPer]) {
        float top = fmaxf(v[0], -INFINITY);
#pragma unroll
        for (int e = 1; e < kPer; ++e) top = fmaxf(top, v[e]);
        const float up = fmaxf(m, top);
        if (up == -INFINITY) return top;
        if (up > m) {
            const float f = factor(m, up);
            d *= f;
            lost *= f;
            m = up;
        }
        float sum = weights(v, up);
        if (!(sum == sum)) {
            clean(v);
            sum = weights(v, up);
        }
        // the running sum keeps what its rounding loses
        const float s = d + sum;
        lost += d >= sum ? (d - s) + sum : (sum - s) + d;
        d = s;
        return top;
    }
};

// The list's first n keys ranked by counting; the K best, in order, to sh.sorted and
// back to the list.  Returns how many there are.
__device__ __forceinline__ int rank_list(RunShared& sh, int n, int K) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const u64 mine = sh.list[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += sh.list[j] > mine;
        if (rank < K) sh.sorted[rank] = mine;
    }
    __syncthreads();
    const int left = min(n, K);
    if (threadIdx.x < left) sh.list[threadIdx.x] = sh.sorted[threadIdx.x];
    return left;
}

// The same for any number of values (many may be equal): the best in turn, of the sorted
// list's `held` keys and a tile.
template <typename T>
__device__ __noinline__ int best_in_turn(RunShared& sh, const Tile<T> tile, int held, int K) {
    const int tid = threadIdx.x;
    uint4 w[Tile<T>::kBlocks];
    float v[kPer];
    tile.fetch(w);
    Tile<T>::values(w, v);
    clean(v);
    const u64 before = tid < held ? sh.sorted[tid] : 0;
    u64 below = ~0ull;
    int k = 0;
    __syncthreads();
    for (; k < K; ++k) {
        u64 best = before < below ? before : 0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const u64 key = make_key(v[e], tile.col(e));
            if (v[e] > -INFINITY && key < below && key > best) best = key;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const u64 other = __shfl_xor_sync(kFullMask, best, o);
            best = other > best ? other : best;
        }
        if (tid % 32 == 0) sh.best[tid / 32] = best;
        __syncthreads();
        for (int i = 0; i < kThreads / 32; ++i) best = max(best, sh.best[i]);
        __syncthreads();
        if (best == 0) break;
        if (tid == 0) sh.sorted[k] = best;
        below = best;
    }
    __syncthreads();
    if (tid < k) sh.list[tid] = sh.sorted[tid];
    return k;
}

template <typename T, int KP>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 3)
    beam_runs_kernel(const __grid_constant__ BeamArgs a) {
    __shared__ RunShared sh;
    const int64_t row = blockIdx.x / a.runs;
    const int run = static_cast<int>(blockIdx.x % a.runs);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;");
    if (!has_row(a, row)) return;
    Tile<T> tile;
    tile.row = static_cast<const T*>(a.x) + row * a.cols;
    tile.cols = a.cols;
    const int head = static_cast<int>(reinterpret_cast<uintptr_t>(tile.row) % 16 / sizeof(T));
    State state;
    int held = 0;  // keys in the list, best first
    const int64_t tiles = (a.cols + head + kTile - 1) / kTile;
    const int64_t first = run * a.run_tiles, last = min(tiles, first + a.run_tiles);
    uint4 w[Tile<T>::kBlocks];
    float v[kPer];
    auto place = [&](int64_t i) { tile.base = i * kTile - head; };
    // the next tile's values are asked for before this one's are worked on
    auto step = [&](int64_t i) {
        Tile<T>::values(w, v);
        if (i + 1 < last) {
            place(i + 1);
            tile.fetch(w);
        }
        place(i);
        return order_key(state.add(v));
    };
    auto push = [&](uint32_t bound) {
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            if (order_key(v[e]) >= bound) {
                const int at = atomicAdd(&sh.count, 1);
                if (at < kList) sh.list[at] = make_key(v[e], tile.col(e));
            }
    };
    if (tid == 0) sh.count = 0;
    if (first < last) {
        place(first);
        tile.fetch(w);
    }
#pragma unroll 1
    for (int64_t i = first; i < last;) {
        // until the list is full a tile's own bound, from then on the K-th of the list
        const bool full = held == a.K;
        const int64_t end = full ? min(last, i + kChunk) : i + 1;
        uint32_t bound = full ? static_cast<uint32_t>(sh.list[a.K - 1] >> 32) + 1 : 0;
#pragma unroll 1
        for (int64_t j = i; j < end; ++j) {
            const uint32_t top = step(j);
            if (!full)
                bound = max(parts_bound<KP, kThreads>(
                                top, sh.bound, [](uint32_t x, uint32_t y) { return max(x, y); }),
                            sample::kKeyNegInf + 1);
            if (top >= bound) push(bound);
        }
        __syncthreads();
        const int n = sh.count;
        if (n > held) {
            if (n <= kList) {
                held = rank_list(sh, n, a.K);
            } else {
#pragma unroll 1
                for (int64_t j = i; j < end; ++j) {
                    place(j);
                    held = best_in_turn(sh, tile, held, a.K);
                }
            }
        }
        __syncthreads();
        if (tid == 0) sh.count = held;
        __syncthreads();
        i = end;
    }
    float m = state.m, d = state.d + state.lost;
    // ---- the run's state
    float top = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
    if (lane == 0) sh.m[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) top = fmaxf(top, sh.m[w]);
    d = m > -INFINITY ? d * factor(m, top) : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(kFullMask, d, o);
    if (lane == 0) sh.d[warp] = d;
    __syncthreads();
    const int64_t at = row * a.runs + run;
    if (tid == 0) {
        float all = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) all += sh.d[w];
        a.states[at] = make_float2(top, all);
    }
    if (tid < a.K) a.lists[at * a.K + tid] = tid < held ? sh.sorted[tid] : 0;
}

// ------------------------------------------------------------------ the groups
struct MergeShared {
    u64 order[kCandidates], at[kCandidates];  // of a value; beam and column
    u64 best[kMaxK], best_at[kMaxK];          // the chosen, in order
    double offset[kMaxBeams];       // score - lse, to add to x - m
    double lse[kMaxBeams];          // ln of the summed weights
    double m64[kMaxBeams];
    double score[kMaxBeams];
    float m[kMaxBeams];
    unsigned char kind[kMaxBeams];  // 0 no candidates, 1 a row, 2 ended
    unsigned char again[kMaxBeams]; // its sum is wanted in 38 bits
    u64 bound[128];
    u64 warp_order[kMergeThreads / 32], warp_at[kMergeThreads / 32];
    u64 sum[kMergeThreads / 32];
    float pow2[64];
    int count;
};

// Doubles as integers of their order: 64-bit comparisons on the integer pipe (the
// FP64 pipe takes one per SM and cycle or so).  No NaN comes here.
__device__ __forceinline__ u64 order64(double v) {
    const u64 b = static_cast<u64>(__double_as_longlong(v + 0.0));
    return b >> 63 ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ double value64(u64 o) {
    return __longlong_as_double(static_cast<long long>(o >> 63 ? o & ~(1ull << 63) : ~o));
}
constexpr u64 kNone = 0x000fffffffffffffull;  // order64(-inf)

// (order, place) pairs: larger value first, then the lower place
__device__ __forceinline__ bool better(u64 c, u64 at, u64 c2, u64 at2) {
    return c > c2 || (c == c2 && at < at2);
}

// ln of a row's summed weights e^(x - m), the weights added as integers; thread 0 has it.
template <typename T>
__device__ double exact_log_sum(MergeShared& sh, const T* row, int64_t cols, float m) {
    int bits = 62;
    while ((int64_t(1) << (62 - bits)) < cols) --bits;
    sample::Weight w;
    w.set(m, 1.f, min(44, bits), sh.pow2);
    u64 sum = 0;
    for (int64_t c = threadIdx.x; c < cols; c += kMergeThreads) {
        const float x = widen(row[c]);
        if (x > -INFINITY) sum += w(x);
    }
    sum = sample::warp_sum64(sum);
    __syncthreads();
    if (threadIdx.x % 32 == 0) sh.sum[threadIdx.x / 32] = sum;
    __syncthreads();
    if (threadIdx.x != 0) return 0.0;
    sum = 0;
    for (int i = 0; i < kMergeThreads / 32; ++i) sum += sh.sum[i];
    return log(static_cast<double>(sum)) - log(static_cast<double>(w(m)));
}

template <typename T, int KP>
__global__ void __launch_bounds__(kMergeThreads)
    beam_merge_kernel(const __grid_constant__ BeamArgs a) {
    __shared__ MergeShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.beams;
    for (int i = tid; i < a.beams; i += kMergeThreads) {
        const float s = a.scores[row0 + i];
        sh.score[i] = s;
        sh.kind[i] = !(s > -INFINITY) ? 0 : a.ended && a.ended[row0 + i] ? 2 : 1;
        sh.again[i] = 0;
    }
    if (tid < 64) sh.pow2[tid] = sample::kPow2[tid];
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = warp; i < a.beams; i += kMergeThreads / 32) {
        if (sh.kind[i] != 1) continue;
        const float2* st = a.states + (row0 + i) * a.runs;
        float top = -INFINITY;
        for (int r = lane; r < a.runs; r += 32) top = fmaxf(top, st[r].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
        float d = 0.f;
        for (int r = lane; r < a.runs; r += 32)
            if (st[r].x > -INFINITY) d += st[r].y * factor(st[r].x, top);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(kFullMask, d, o);
        if (lane == 0) {
            sh.m[i] = top;
            // ln d by parts: the power of two's share is exact in 64 bits
            const int e = d > 0.f ? ilogbf(d) : 0;
            const double ln_d = static_cast<double>(logf(scalbnf(d, -e))) + e * 0.6931471805599453;
            sh.lse[i] = ln_d;
            sh.m64[i] = top;
        }
    }
    const int lists = a.beams * a.runs;
    const double eps = a.eps;
    // entry e of list j (a beam's run): its key, 0 where there is none
    auto key_of = [&](int list, int e) -> u64 {
        const int beam = list / a.runs;
        if (sh.kind[beam] == 1) return a.lists[((row0 + beam) * a.runs + list % a.runs) * a.K + e];
        // an ended beam goes on with `pad` alone
        return sh.kind[beam] == 2 && list % a.runs == 0 && e == 0
                   ? (1ull << 63) | (0xffffffffu - static_cast<uint32_t>(a.pad)) : 0;
    };
    auto order_of = [&](u64 key, int beam) -> u64 {
        if (key == 0) return kNone;
        if (sh.kind[beam] == 2) return order64(sh.score[beam]);
        const float x = key_value(static_cast<uint32_t>(key >> 32));
        if (sh.m[beam] == INFINITY) return x == INFINITY ? order64(sh.offset[beam]) : kNone;
        return order64(sh.offset[beam] + (static_cast<double>(x) - sh.m64[beam]));
    };
    auto at_of = [](u64 key, int beam) {
        return (static_cast<u64>(beam) << 32) | (0xffffffffu - static_cast<uint32_t>(key));
    };
    int found = 0;
    for (int round = 0; round < 2; ++round) {
        __syncthreads();
        if (tid == 0) sh.count = 0;
        for (int i = tid; i < a.beams; i += kMergeThreads)
            if (sh.kind[i] == 1)
                sh.offset[i] = sh.score[i] - sh.lse[i];
        __syncthreads();
        // ---- a bound that K of the lists' first entries reach, dealt out to the parts in turn
        u64 top = kNone;
        {
            constexpr int kPart = kMergeThreads / KP;
            const int all = max(lists, min(kMergeThreads, lists * a.K));
            for (int i = tid / kPart + KP * (tid % kPart); i < all; i += kMergeThreads) {
                const u64 c = order_of(key_of(i % lists, i / lists), i % lists / a.runs);
                top = c > top ? c : top;
            }
        }
        u64 bound = parts_bound<KP, kMergeThreads>(top, sh.bound,
                                                   [](u64 x, u64 y) { return x > y ? x : y; });
        // (one that the errors may have put below another is not lost)
        if (round == 0 && bound > kNone) bound = order64(value64(bound) - 4 * eps);
        if (bound == kNone) ++bound;
        for (int i = tid; i < lists * a.K; i += kMergeThreads) {
            const int list = i / a.K, beam = list / a.runs;
            const u64 key = key_of(list, i % a.K);
            const u64 c = order_of(key, beam);
            if (c >= bound) {
                const int at = atomicAdd(&sh.count, 1);
                if (at < kCandidates) {
                    sh.order[at] = c;
                    sh.at[at] = at_of(key, beam);
                }
            }
        }
        __syncthreads();
        const int n = sh.count;
        if (n <= kCandidates) {
            for (int i = tid; i < n; i += kMergeThreads) {
                const u64 c = sh.order[i], at = sh.at[i];
                int rank = 0;
                for (int j = 0; j < n; ++j) rank += better(sh.order[j], sh.at[j], c, at);
                if (rank < a.K) {
                    sh.best[rank] = c;
                    sh.best_at[rank] = at;
                }
            }
            found = min(n, a.K);
        } else {
            // many equal values: the best of what is left in turn
            u64 c0 = ~0ull, at0 = 0;
            for (found = 0; found < a.K; ++found) {
                u64 c1 = kNone, at1 = ~0ull;
                for (int i = tid; i < lists * a.K; i += kMergeThreads) {
                    const int beam = i / a.K / a.runs;
                    const u64 key = key_of(i / a.K, i % a.K);
                    const u64 c = order_of(key, beam), at = at_of(key, beam);
                    if (c > kNone && (found == 0 || better(c0, at0, c, at)) &&
                        better(c, at, c1, at1))
                        c1 = c, at1 = at;
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const u64 c = __shfl_xor_sync(kFullMask, c1, o);
                    const u64 at = __shfl_xor_sync(kFullMask, at1, o);
                    if (better(c, at, c1, at1)) c1 = c, at1 = at;
                }
                if (lane == 0) sh.warp_order[warp] = c1, sh.warp_at[warp] = at1;
                __syncthreads();
                for (int w = 0; w < kMergeThreads / 32; ++w)
                    if (better(sh.warp_order[w], sh.warp_at[w], c1, at1))
                        c1 = sh.warp_order[w], at1 = sh.warp_at[w];
                __syncthreads();
                if (c1 == kNone) break;
                if (tid == 0) sh.best[found] = c1, sh.best_at[found] = at1;
                c0 = c1, at0 = at1;
            }
        }
        __syncthreads();
        if (round || found == 0) break;
        // ---- values of different beams that the sums cannot tell apart: neighbours in the
        // order, and of what is not chosen all that come near the last chosen
        bool near = false;
        auto mark = [&](u64 at0, u64 at1) {
            const uint32_t b0 = at0 >> 32, b1 = at1 >> 32;
            if (b0 == b1) return;
            near = true;
            sh.again[b0] = sh.again[b1] = 1;
        };
        for (int i = tid; i + 1 < found; i += kMergeThreads)
            if (value64(sh.best[i]) - value64(sh.best[i + 1]) <= 2 * eps)
                mark(sh.best_at[i], sh.best_at[i + 1]);
        const u64 last = sh.best[found - 1], last_at = sh.best_at[found - 1];
        const u64 low = order64(value64(last) - 2 * eps);
        auto behind = [&](u64 c, u64 at) {
            if (c >= low && better(last, last_at, c, at)) mark(last_at, at);
        };
        if (n <= kCandidates)
            for (int i = tid; i < n; i += kMergeThreads) behind(sh.order[i], sh.at[i]);
        else
            for (int i = tid; i < lists * a.K; i += kMergeThreads) {
                const int beam = i / a.K / a.runs;
                const u64 key = key_of(i / a.K, i % a.K);
                if (key) behind(order_of(key, beam), at_of(key, beam));
            }
        if (!__syncthreads_or(near)) break;
        for (int b = 0; b < a.beams; ++b) {
            if (!sh.again[b] || sh.kind[b] != 1 || sh.m[b] == INFINITY) continue;
            const double log_sum = exact_log_sum(
                sh, static_cast<const T*>(a.x) + (row0 + b) * a.cols, a.cols, sh.m[b]);
            if (tid == 0) sh.lse[b] = log_sum;
        }
    }
    if (tid < a.K) {
        const bool is = tid < found;
        const int64_t at = static_cast<int64_t>(blockIdx.x) * a.K + tid;
        a.out[at] = is ? static_cast<float>(value64(sh.best[tid])) : -INFINITY;
        a.parents[at] = is ? static_cast<int>(sh.best_at[tid] >> 32) : -1;
        a.tokens[at] = is ? static_cast<int>(sh.best_at[tid] & 0xffffffffu) : -1;
    }
}

}  // namespace beam
}  // namespace os
