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
// From then on a value has to pass the K-th of the list, which few do.
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
    __device__ __forceinline__ void load(float (&v)[kPer]) const {
        uint4 w[kBlocks];
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
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            const T* e = reinterpret_cast<const T*>(&w[b]);
#pragma unroll
            for (int i = 0; i < kVec; ++i) v[b * kVec + i] = widen(e[i]);
        }
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

template <typename T, int KP>
__global__ void __launch_bounds__(kThreads) beam_runs_kernel(const __grid_constant__ BeamArgs a) {
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
    float m = -INFINITY, d = 0.f, lost = 0.f;
    int held = 0;  // keys in the list, best first
    const int64_t tiles = (a.cols + head + kTile - 1) / kTile;
    const int64_t first = run * a.run_tiles, last = min(tiles, first + a.run_tiles);
#pragma unroll 1
    for (int64_t i = first; i < last; ++i) {
        tile.base = i * kTile - head;
        float v[kPer];
        tile.load(v);
        if (tid == 0) sh.count = held;
        float top = v[0];
#pragma unroll
        for (int e = 1; e < kPer; ++e) top = fmaxf(top, v[e]);
        // ---- (m, d): weights below the thread's running maximum
        const float up = fmaxf(m, top);
        if (up > -INFINITY) {
            float sum;
            if (fabsf(up) < 1e30f) {
                // base-2 exponents with one rounding each, below the rounded
                // maximum; the factor between it and the maximum comes at once
                const float c = up * kLog2e;
                float part[4] = {};
#pragma unroll
                for (int e = 0; e < kPer; ++e) part[e & 3] += ex2f(fmaf(v[e], kLog2e, -c));
                sum = ((part[0] + part[1]) + (part[2] + part[3])) * ex2f(fmaf(up, -kLog2e, c));
            } else {
                // a maximum of +-inf or near the largest number
                sum = 0.f;
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    sum += v[e] == up ? 1.f : ex2f((v[e] - up) * kLog2e);
            }
            const float f = factor(m, up);
            d *= f;
            lost *= f;
            m = up;
            // the running sum keeps what its rounding loses
            const float s = d + sum;
            lost += d >= sum ? (d - s) + sum : (sum - s) + d;
            d = s;
        }
        // ---- the K best so far
        uint32_t bound;
        if (held < a.K)
            bound = parts_bound<KP, kThreads>(order_key(top), sh.bound,
                                              [](uint32_t x, uint32_t y) { return max(x, y); });
        else
            bound = static_cast<uint32_t>(sh.list[a.K - 1] >> 32) + 1;
        bound = max(bound, sample::kKeyNegInf + 1);
        const bool any = order_key(top) >= bound;
        if (!__syncthreads_or(any)) continue;
        if (any) {
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (order_key(v[e]) >= bound) {
                    const int at = atomicAdd(&sh.count, 1);
                    if (at < kList) sh.list[at] = make_key(v[e], tile.col(e));
                }
        }
        __syncthreads();
        const int n = sh.count;
        if (n <= kList) {
            held = rank_list(sh, n, a.K);
        } else {
            // many equal values: the best in turn, from the tile and the old list
            u64 mine_before = tid < held ? sh.sorted[tid] : 0, below = ~0ull;
            int k = 0;
            __syncthreads();
            for (; k < a.K; ++k) {
                u64 best = mine_before < below ? mine_before : 0;
#pragma unroll 1
                for (int e = 0; e < kPer; ++e) {
                    float x = v[0];
#pragma unroll
                    for (int j = 1; j < kPer; ++j) x = j == e ? v[j] : x;
                    const u64 key = make_key(x, tile.col(e));
                    if (x > -INFINITY && key < below && key > best) best = key;
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const u64 other = __shfl_xor_sync(kFullMask, best, o);
                    best = other > best ? other : best;
                }
                if (lane == 0) sh.best[warp] = best;
                __syncthreads();
                for (int w = 0; w < kThreads / 32; ++w) best = max(best, sh.best[w]);
                __syncthreads();
                if (best == 0) break;
                if (tid == 0) sh.sorted[k] = best;
                below = best;
            }
            __syncthreads();
            held = k;
            if (tid < held) sh.list[tid] = sh.sorted[tid];
        }
        __syncthreads();
    }
    // ---- the run's state
    d += lost;
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
    double value[kCandidates];
    uint32_t beam[kCandidates], col[kCandidates];
    double best[kMaxK];             // the chosen, in order
    uint32_t best_beam[kMaxK], best_col[kMaxK];
    double offset[kMaxBeams];       // score - lse + m
    double score[kMaxBeams];
    float m[kMaxBeams];
    unsigned char kind[kMaxBeams];  // 0 no candidates, 1 a row, 2 ended
    unsigned char again[kMaxBeams]; // its sum is wanted in 38 bits
    double bound[128];
    double warp_value[kMergeThreads / 32];
    u64 warp_at[kMergeThreads / 32];
    u64 sum[kMergeThreads / 32];
    float pow2[64];
    int count;
};

// (value, place) pairs: larger value first, then the lower place
__device__ __forceinline__ bool better(double c, u64 at, double c2, u64 at2) {
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
            sh.offset[i] = sh.score[i] - ln_d;
        }
    }
    const int lists = a.beams * a.runs;
    const double eps = a.eps;
    // candidate e of list j: its value, or -inf where there is none
    auto value = [&](u64 key, int beam) -> double {
        if (sh.kind[beam] == 2) return key ? sh.score[beam] : -INFINITY;
        if (key == 0) return -INFINITY;
        const float x = key_value(static_cast<uint32_t>(key >> 32)), m = sh.m[beam];
        return sh.offset[beam] + (x == m ? 0.0 : static_cast<double>(x) - static_cast<double>(m));
    };
    auto key_of = [&](int list, int e) -> u64 {
        const int beam = list / a.runs;
        if (sh.kind[beam] == 1) return a.lists[((row0 + beam) * a.runs + list % a.runs) * a.K + e];
        // an ended beam goes on with `pad` alone
        return sh.kind[beam] == 2 && list % a.runs == 0 && e == 0
                   ? (1ull << 63) | (0xffffffffu - static_cast<uint32_t>(a.pad)) : 0;
    };
    int found = 0;
    for (int round = 0; round < 2; ++round) {
        __syncthreads();
        if (tid == 0) sh.count = 0;
        // ---- a bound that K of the lists' first values reach
        double top = -INFINITY;
        for (int j = tid; j < lists; j += kMergeThreads) {
            const double c = value(key_of(j, 0), j / a.runs);
            top = c > top ? c : top;
        }
        double bound = parts_bound<KP, kMergeThreads>(
            top, sh.bound, [](double x, double y) { return x > y ? x : y; });
        // (one that the errors may have put below another is not lost)
        if (round == 0) bound -= 4 * eps;
        __syncthreads();
        for (int i = tid; i < lists * a.K; i += kMergeThreads) {
            const int list = i / a.K, beam = list / a.runs;
            const u64 key = key_of(list, i % a.K);
            const double c = value(key, beam);
            if (c > -INFINITY && c >= bound) {
                const int at = atomicAdd(&sh.count, 1);
                if (at < kCandidates) {
                    sh.value[at] = c;
                    sh.beam[at] = beam;
                    sh.col[at] = 0xffffffffu - static_cast<uint32_t>(key);
                }
            }
        }
        __syncthreads();
        const int n = sh.count, want = a.K;
        if (n <= kCandidates) {
            for (int i = tid; i < n; i += kMergeThreads) {
                const double c = sh.value[i];
                const u64 at = (static_cast<u64>(sh.beam[i]) << 32) | sh.col[i];
                int rank = 0;
                for (int j = 0; j < n; ++j)
                    rank += better(sh.value[j], (static_cast<u64>(sh.beam[j]) << 32) | sh.col[j],
                                   c, at);
                if (rank < want) {
                    sh.best[rank] = c;
                    sh.best_beam[rank] = sh.beam[i];
                    sh.best_col[rank] = sh.col[i];
                }
            }
            found = min(n, want);
        } else {
            // many equal values: the best of what is left in turn
            double c0 = INFINITY;
            u64 at0 = 0;
            for (found = 0; found < want; ++found) {
                double c1 = -INFINITY;
                u64 at1 = ~0ull;
                for (int i = tid; i < lists * a.K; i += kMergeThreads) {
                    const int beam = i / a.K / a.runs;
                    const u64 key = key_of(i / a.K, i % a.K);
                    const double c = value(key, beam);
                    const u64 at = (static_cast<u64>(beam) << 32) |
                                   (0xffffffffu - static_cast<uint32_t>(key));
                    if (c > -INFINITY && (found == 0 || better(c0, at0, c, at)) &&
                        better(c, at, c1, at1))
                        c1 = c, at1 = at;
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const double c = __shfl_xor_sync(kFullMask, c1, o);
                    const u64 at = __shfl_xor_sync(kFullMask, at1, o);
                    if (better(c, at, c1, at1)) c1 = c, at1 = at;
                }
                if (lane == 0) sh.warp_value[warp] = c1, sh.warp_at[warp] = at1;
                __syncthreads();
                for (int w = 0; w < kMergeThreads / 32; ++w)
                    if (better(sh.warp_value[w], sh.warp_at[w], c1, at1))
                        c1 = sh.warp_value[w], at1 = sh.warp_at[w];
                __syncthreads();
                if (!(c1 > -INFINITY)) break;
                if (tid == 0) {
                    sh.best[found] = c1;
                    sh.best_beam[found] = static_cast<uint32_t>(at1 >> 32);
                    sh.best_col[found] = static_cast<uint32_t>(at1);
                }
                c0 = c1, at0 = at1;
            }
        }
        __syncthreads();
        if (round || found == 0) break;
        // ---- values of different beams that the sums cannot tell apart: neighbours in the
        // order, and of what is not chosen all that come near the last chosen
        bool near = false;
        auto mark = [&](uint32_t b0, uint32_t b1) {
            if (b0 == b1) return;
            near = true;
            sh.again[b0] = sh.again[b1] = 1;
        };
        for (int i = tid; i + 1 < found; i += kMergeThreads)
            if (sh.best[i] - sh.best[i + 1] <= 2 * eps) mark(sh.best_beam[i], sh.best_beam[i + 1]);
        const uint32_t last_beam = sh.best_beam[found - 1];
        const u64 last_at = (static_cast<u64>(last_beam) << 32) | sh.best_col[found - 1];
        const double last = sh.best[found - 1];
        auto behind = [&](double c, uint32_t beam, uint32_t col) {
            if (c >= last - 2 * eps && better(last, last_at, c, (static_cast<u64>(beam) << 32) | col))
                mark(last_beam, beam);
        };
        if (n <= kCandidates)
            for (int i = tid; i < n; i += kMergeThreads) behind(sh.value[i], sh.beam[i], sh.col[i]);
        else
            for (int i = tid; i < lists * a.K; i += kMergeThreads) {
                const u64 key = key_of(i / a.K, i % a.K);
                const int beam = i / a.K / a.runs;
                const double c = value(key, beam);
                if (c > -INFINITY) behind(c, beam, 0xffffffffu - static_cast<uint32_t>(key));
            }
        if (!__syncthreads_or(near)) break;
        for (int b = 0; b < a.beams; ++b) {
            if (!sh.again[b] || sh.kind[b] != 1 || sh.m[b] == INFINITY) continue;
            const double log_sum = exact_log_sum(
                sh, static_cast<const T*>(a.x) + (row0 + b) * a.cols, a.cols, sh.m[b]);
            if (tid == 0) sh.offset[b] = sh.score[b] - log_sum;
        }
    }
    if (tid < a.K) {
        const bool is = tid < found;
        const int64_t at = static_cast<int64_t>(blockIdx.x) * a.K + tid;
        a.out[at] = is ? static_cast<float>(sh.best[tid]) : -INFINITY;
        a.parents[at] = is ? static_cast<int>(sh.best_beam[tid]) : -1;
        a.tokens[at] = is ? static_cast<int>(sh.best_col[tid]) : -1;
    }
}

}  // namespace beam
}  // namespace os
