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
// A run's K best: every thread keeps the largest value of its columns of each tile
// (64 bytes; one store).  At the end of the run a bound that at least K values reach is
// the least of the largest values of K (or a few more) equal parts of the threads;
// the shares that reach it (some K ln K) are read again, their values that reach it go
// to a list in shared memory, and the list is ranked by counting.  So the pass over
// memory has no branch, no barrier and no atomic for the selection.
//
// Exact choices.  Values of different beams compare through their lse, which the
// first kernel's fp32 sums give within eps.  Where two values of different
// beams next to one another in the order, up to the first that is not chosen,
// are nearer than both errors, the rows of these beams are summed again with the
// sampler's weights (38 bits, added as integers), by the CTAs of a cluster, and the
// order is taken from those sums in 64 bits.
//
// What bounds it: 32 groups of 8 beams of 128256 bf16 columns, K = 16, take 29 us in a
// graph, with one beam in eight ended too (the one read at the rate of memory: 9.7 and 8.5).
// Alone and cold the first kernel takes 23, with memory at a third of its rate and schedulers
// that issue in 42 % of their cycles: on SMs with one CTA or two, the start, the stream (about
// 8 instructions per column, of which one on the SFU) and the selection at its end, when the
// CTA's memory stands idle, follow one another.  The second takes 10, the latency of its
// steps on one SM per group (issue 4 %).  Where a group needs exact sums (5 calls in 300 at
// these sizes) it takes 18 more: two rows of 43 instructions per column on eight SMs.  4
// beams of 50257 fp32: 11 us.
#pragma once

#include "../beam_error.h"
#include "paged_common.cuh"
#include "sample_kernel.cuh"

namespace os {
namespace beam {

using sample::key_value;
using sample::order_key;
using sample::widen;
using u64 = unsigned long long;

constexpr int kThreads = 256;   // of a run's CTA
constexpr int kBlocks = 4;      // 16-byte blocks per thread and tile
constexpr int kSegmentCols = 1 << 16;  // columns between two selections
constexpr int kList = 1024;     // values that reach the bound; more go another way
constexpr int kGroups = 512;    // threads' shares of a tile that do
constexpr int kMergeThreads = kThreads;
constexpr int kHelpers = 8;     // CTAs of a group, at most: four equal beams of 50257 columns
                                // take 27 us with eight and 74 with one, beams that need no
                                // exact sums 10.9 and 10.5
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
    u64* lists;                    // [groups][K][beams * runs]: the runs' keys, best first, then 0
    float2* states;                // [groups * beams][runs]: m, d
    int64_t cols;
    int beams, K, runs;
    int run_tiles;                 // tiles of a run
    int helpers;                   // CTAs of a group
    int pad;
    float eps;                     // bound of lse's error (and kFarError)
};

// value and column in one number: larger is better, no two alike, 0 is none
__device__ __forceinline__ u64 make_key(float x, uint32_t col) {
    return (static_cast<u64>(order_key(x)) << 32) | (0xffffffffu - col);
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

// The least of the maxima of KP parts of the CTA's values (as order keys); every thread
// gets it.  Thread t is of part t mod KP, so that neighbouring columns are of different
// parts and a short row fills them all.  sh: a word per thread.
template <int KP>
__device__ __forceinline__ uint32_t parts_bound(uint32_t v, uint32_t* sh) {
    constexpr int kLanes = KP < 32 ? KP : 32, kWarps = kThreads / 32;
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int o = 16; o >= kLanes; o >>= 1) v = max(v, __shfl_xor_sync(kFullMask, v, o));
    sh[threadIdx.x] = v;
    __syncthreads();
    // 64 parts: the even warps have the first 32 of them, the odd ones the others
    constexpr int kSets = KP > 32 ? 2 : 1;
    uint32_t least = 0xffffffffu;
#pragma unroll
    for (int set = 0; set < kSets; ++set) {
        uint32_t top = 0;
#pragma unroll
        for (int w = set; w < kWarps; w += kSets) top = max(top, sh[w * 32 + lane]);
        least = min(least, top);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) least = min(least, __shfl_xor_sync(kFullMask, least, o));
    return least;
}

// Tiles on their way to a CTA, what it keeps of them, and its list: 75 KB for fp32, 67 for
// bf16, so that three CTAs fit an SM.
template <typename T>
struct RunShared {
    static constexpr int kStages = 3;
    static constexpr int kSegment = kSegmentCols / (kThreads * kBlocks * 16 / int(sizeof(T)));
    uint4 tile[kStages][kBlocks][kThreads];
    float top[kSegment][kThreads];  // the largest of a thread's columns of a tile
    u64 list[kList];
    u64 sorted[kMaxK];
    uint32_t bound[kThreads];
    u64 best[kThreads / 32];
    float m[kThreads / 32], d[kThreads / 32];
    uint16_t group[kGroups];
    int count, groups;
};

// Columns of the tile's thread, as 16-byte blocks: value i of the thread belongs
// to column col(i).  Rows start anywhere, so block 0 is the aligned one that the
// row's first column lies in; a block that the row covers in part is read by elements.
// Columns count modulo 2^32: what lies before the row is past its end.
template <typename T>
struct Tile {
    static constexpr int kVec = 16 / sizeof(T);
    static constexpr int kPer = kBlocks * kVec;  // columns per thread
    static constexpr int kTile = kThreads * kPer;
    const T* row;
    uint32_t cols, base;  // base: column of the thread's first value

    __device__ __forceinline__ uint32_t col(int i) const {
        return base + (i / kVec) * (kThreads * kVec) + i % kVec;
    }
    __device__ __forceinline__ bool whole(uint32_t c) const { return c < cols && cols - c >= kVec; }
    // The tile on its way to the thread's places in shared memory, which no other thread
    // reads or writes; -inf where there is no column.  `inside`: the row covers it all.
    __device__ __forceinline__ void fetch(uint4 (&to)[kBlocks][kThreads], bool inside) const {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            const uint32_t c = base + b * (kThreads * kVec);
            uint4* at = &to[b][threadIdx.x];
            if (inside || whole(c)) {
                asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;"
                             :: "r"(static_cast<uint32_t>(__cvta_generic_to_shared(at))),
                                "l"(row + c) : "memory");
            } else {
#pragma unroll 1
                for (int i = 0; i < kVec; ++i)
                    reinterpret_cast<T*>(at)[i] = c + i < cols ? row[c + i] : T(-INFINITY);
            }
        }
    }
    // The block from column c on, read anew.
    __device__ __forceinline__ uint4 block(uint32_t c) const {
        if (whole(c)) return *reinterpret_cast<const uint4*>(row + c);
        uint32_t words[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            constexpr int kEach = 4 / sizeof(T);
            words[j] = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const uint32_t at = c + j * kEach + i;
                const T v = at < cols ? row[at] : T(-INFINITY);
                if constexpr (sizeof(T) == 4) words[j] = __float_as_uint(v);
                else words[j] |= static_cast<uint32_t>(__bfloat16_as_ushort(v)) << (16 * i);
            }
        }
        return make_uint4(words[0], words[1], words[2], words[3]);
    }
    static __device__ __forceinline__ void values(const uint4& w, float* v) {
        const uint32_t bits[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            v[i] = __uint_as_float(sizeof(T) == 4 ? bits[i % 4]
                                   : i & 1        ? bits[i / 2 % 4] & 0xffff0000u
                                                  : bits[i / 2 % 4] << 16);
    }
};

// The largest of a thread's columns, NaN passed over.
template <typename T>
__device__ __forceinline__ float largest_of(const uint4 (&w)[kBlocks]) {
    if constexpr (sizeof(T) == 4) {
        float top = -INFINITY;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            top = max3(top, __uint_as_float(w[b].x), __uint_as_float(w[b].y));
            top = max3(top, __uint_as_float(w[b].z), __uint_as_float(w[b].w));
        }
        return top;
    } else {
        // two at a time, as they lie
        uint32_t top = 0xff80ff80u;  // -inf, -inf
        auto larger = [&](uint32_t v) {
            asm("max.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(v));
        };
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) larger(w[b].x), larger(w[b].y), larger(w[b].z), larger(w[b].w);
        return fmaxf(__uint_as_float(top << 16), __uint_as_float(top & 0xffff0000u));
    }
}

// A thread's share of the row's normalizer state: weights e^(x - m) summed as d + lost,
// and the largest value so far.  m follows the largest only when that has passed it by
// more than one, so what has been through many changes of m weighs little beside what
// came later, and the changes' roundings add up to the logarithm of the share's columns
// (beam_error.h).
template <typename T>
struct State {
    float m = -INFINITY, d = 0.f, lost = 0.f, largest = -INFINITY;

    __device__ __forceinline__ float weights(const uint4 (&w)[kBlocks]) const {
        // base-2 exponents with one rounding each, below the rounded reference; the
        // factor between it and the reference comes at once
        const float c = m * kLog2e;
        float2 part[2] = {};
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            float v[Tile<T>::kVec];
            Tile<T>::values(w[b], v);
#pragma unroll
            for (int e = 0; e < Tile<T>::kVec; e += 2) {
                const float2 t = fma2(make_float2(v[e], v[e + 1]), splat2(kLog2e), splat2(-c));
                part[e/2&1] = add2(part[e/2&1], make_float2(ex2f(t.x), ex2f(t.y)));
            }
        }
        return ((part[0].x + part[0].y) + (part[1].x + part[1].y)) * ex2f(fmaf(m, -kLog2e, c));
    }
    // Returns the tile's largest value.
    __device__ __forceinline__ float add(const uint4 (&w)[kBlocks]) {
        const float top = largest_of<T>(w);
        if (top > m + 1.f) {
            const float f = factor(m, top);
            d *= f;
            lost *= f;
            m = top;
        }
        largest = fmaxf(largest, top);
        const float sum = m > -INFINITY ? weights(w) : 0.f;
        // the running sum keeps what its rounding loses
        const float s = d + sum;
        lost += d >= sum ? (d - s) + sum : (sum - s) + d;
        d = s;
        return top;
    }
    // Not so where a value was NaN, or the reference is infinite or so large that it and
    // its product with log2 e are too far apart (the sum is then NaN, or this is asked).
    __device__ __forceinline__ bool good() const {
        return d < INFINITY && (m == -INFINITY || fabsf(m) < 0x1p28f);
    }
    // the sum below another reference of at least `largest`
    __device__ __forceinline__ float below(float top) const {
        return m > -INFINITY ? (d + lost) * (m == top ? 1.f : exp1(m - top)) : 0.f;
    }
};

// The list's first n keys ranked by counting; the K best, in order, to sh.sorted and
// back to the list.  Returns how many there are.
template <typename T>
__device__ __forceinline__ int rank_list(RunShared<T>& sh, int n, int K) {
    const auto* pairs = reinterpret_cast<const ulonglong2*>(sh.list);
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const u64 mine = sh.list[i];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n / 2; ++j) {
            const ulonglong2 p = pairs[j];
            rank += (p.x > mine) + (p.y > mine);
        }
        if (n & 1) rank += sh.list[n - 1] > mine;
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
__device__ __noinline__ int best_in_turn(RunShared<T>& sh, const Tile<T> tile, int held, int K) {
    const int tid = threadIdx.x;
    constexpr int kPer = Tile<T>::kPer;
    float v[kPer];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
        Tile<T>::values(tile.block(tile.col(b * Tile<T>::kVec)), v + b * Tile<T>::kVec);
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
    __syncthreads();
    return k;
}

// A thread's weights of tiles [first, last) below their largest value `top`, one by one:
// for the rows that State cannot sum.
template <typename T>
__device__ __noinline__ float careful_sum(Tile<T> tile, int first, int last, int head, float top) {
    float d = 0.f, lost = 0.f;
    for (int i = first; i < last; ++i) {
        tile.base = static_cast<uint32_t>(i) * Tile<T>::kTile - head + threadIdx.x * Tile<T>::kVec;
        for (int b = 0; b < kBlocks; ++b) {
            float v[Tile<T>::kVec];
            Tile<T>::values(tile.block(tile.col(b * Tile<T>::kVec)), v);
#pragma unroll
            for (int e = 0; e < Tile<T>::kVec; ++e) {
                const float x = !(v[e] > -INFINITY) ? 0.f : v[e] == top ? 1.f : exp1(v[e] - top);
                const float s = d + x;
                lost += d >= x ? (d - s) + x : (x - s) + d;
                d = s;
            }
        }
    }
    return d + lost;
}

template <typename T, int KP>
__global__ void __launch_bounds__(kThreads, 3)
    beam_runs_kernel(const __grid_constant__ BeamArgs a) {
    using Tiles = Tile<T>;
    constexpr int kTile = Tiles::kTile, kSegment = RunShared<T>::kSegment;
    constexpr int kStages = RunShared<T>::kStages, kVec = Tiles::kVec;
    extern __shared__ __align__(16) unsigned char raw[];
    auto& sh = *reinterpret_cast<RunShared<T>*>(raw);
    const int64_t row = blockIdx.x / a.runs;
    const int run = static_cast<int>(blockIdx.x % a.runs);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    wait_before();
    // a beam that is not there or has ended has no continuations of its own (known only
    // after the first tiles are asked for, so as not to wait twice)
    const float score = a.scores[row];
    const bool ended = a.ended && a.ended[row];
    Tiles tile;
    tile.row = static_cast<const T*>(a.x) + row * a.cols;
    tile.cols = static_cast<uint32_t>(a.cols);
    const int head = static_cast<int>(reinterpret_cast<uintptr_t>(tile.row) % 16 / sizeof(T));
    const int tiles = static_cast<int>((a.cols + head + kTile - 1) / kTile);
    const int first = run * a.run_tiles, last = min(tiles, first + a.run_tiles);
    auto place = [&](int i, int thread) {
        tile.base = static_cast<uint32_t>(i) * kTile - head + thread * kVec;
    };
    auto fetch = [&](int i, int stage) {
        place(i, tid);
        const uint32_t begin = static_cast<uint32_t>(i) * kTile - head;
        if (i < last) tile.fetch(sh.tile[stage], begin < tile.cols && tile.cols - begin >= kTile);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(first + i, i);
    if (!(score > -INFINITY) || ended) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        return;
    }
    State<T> state;
    int held = 0;  // keys in the list, best first
    bool many = false;  // more values reached a bound than the list holds: many are equal
    int stage = 0;
#pragma unroll 1
    for (int from = first; from < last; from += kSegment) {
        const int to = min(last, from + kSegment);
        float largest = -INFINITY;
#pragma unroll 1
        for (int i = from; i < to; ++i) {
            fetch(i + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
            asm volatile("cp.async.wait_group %0;" :: "n"(kStages - 1) : "memory");
            uint4 w[kBlocks];
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) w[b] = sh.tile[stage][b][tid];
            stage = stage + 1 == kStages ? 0 : stage + 1;
            const float top = state.add(w);
            sh.top[i - from][tid] = top;
            largest = fmaxf(largest, top);
        }
        if (to == last) {
            // the row's state, warp by warp (NaN where a thread could not sum)
            float top = state.largest;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
            float d = state.good() ? state.below(top) : NAN;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(kFullMask, d, o);
            if (lane == 0) sh.m[warp] = top, sh.d[warp] = d;
        }
        // ---- the K best so far: a bound that K values of the segment reach (-inf is no
        // continuation); with a full list, one past its K-th (a later column has to be larger)
        if (tid == 0) sh.count = held, sh.groups = 0;
        uint32_t least = parts_bound<KP>(order_key(largest), sh.bound);
        least = max(least, sample::kKeyNegInf + 1);
        if (held == a.K) least = max(least, static_cast<uint32_t>(sh.list[a.K - 1] >> 32) + 1);
        const float bound = key_value(least);
        if (largest >= bound)
            for (int i = 0; i < to - from; ++i)
                if (sh.top[i][tid] >= bound) {
                    const int at = atomicAdd(&sh.groups, 1);
                    if (at < kGroups) sh.group[at] = static_cast<uint16_t>(i * kThreads + tid);
                }
        __syncthreads();
        const int groups = sh.groups;
        if (groups <= kGroups) {
            for (int i = tid; i < groups * kBlocks; i += kThreads) {
                const int group = sh.group[i / kBlocks];
                place(from + group / kThreads, group % kThreads);
                const uint32_t c = tile.col(i % kBlocks * kVec);
                float v[kVec];
                Tiles::values(tile.block(c), v);
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if (v[e] >= bound) {
                        const int at = atomicAdd(&sh.count, 1);
                        if (at < kList) sh.list[at] = make_key(v[e], c + e);
                    }
            }
            __syncthreads();
        }
        const int n = sh.count;
        if (groups > kGroups || n > kList) {
            many = true;
            __syncthreads();
        } else {
            if (n > held) held = rank_list(sh, n, a.K);
            __syncthreads();
        }
    }
    if (many) {
        held = 0;
#pragma unroll 1
        for (int i = first; i < last; ++i) {
            place(i, tid);
            held = best_in_turn(sh, tile, held, a.K);
        }
    }
    // ---- the run's state
    const int64_t at = row * a.runs + run;
    if (first < last) {
        constexpr int kWarps = kThreads / 32;
        auto join = [&](float& top) {
            float m = sh.m[lane % kWarps], d = sh.d[lane % kWarps];
            top = m;
#pragma unroll
            for (int o = kWarps / 2; o > 0; o >>= 1)
                top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
            d = m > -INFINITY ? d * factor(m, top) : 0.f;
#pragma unroll
            for (int o = kWarps / 2; o > 0; o >>= 1) d += __shfl_xor_sync(kFullMask, d, o);
            return d;
        };
        float top, d = join(top);
        if (!(d == d)) {
            __syncthreads();
            float mine = careful_sum(tile, first, last, head, top);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(kFullMask, mine, o);
            if (lane == 0) sh.m[warp] = top, sh.d[warp] = mine;
            __syncthreads();
            d = join(top);
        }
        if (tid == 0) a.states[at] = make_float2(top, d);
    } else if (tid == 0) {
        a.states[at] = make_float2(-INFINITY, 0.f);
    }
    const int64_t group = row / a.beams, list = at - group * a.beams * a.runs;
    if (tid < a.K)
        a.lists[(group * a.K + tid) * a.beams * a.runs + list] = tid < held ? sh.sorted[tid] : 0;
}

// ------------------------------------------------------------------ the groups
// A sum of integers of 64 bits: high * 2^32 + low, each the sum of the halves.
struct Sum {
    u64 high, low;
    __device__ __forceinline__ void add(Sum s) { high += s.high, low += s.low; }
    // (from the parts' only form with low below 2^32, so that equal sums are equal doubles)
    __device__ __forceinline__ double value() const {
        return static_cast<double>(high + (low >> 32)) * 4294967296.0 +
               static_cast<double>(low & 0xffffffffu);
    }
};

struct MergeShared {
    ulonglong2 found[kCandidates];            // a value's order; its beam and column
    u64 best[kMaxK], best_at[kMaxK];          // the chosen, in order
    double offset[kMaxBeams];       // score - lse, to add to x - m
    double lse[kMaxBeams];          // ln of the summed weights
    double m64[kMaxBeams];
    double score[kMaxBeams];
    float m[kMaxBeams], near[kMaxBeams];  // near: the offset in fp32
    unsigned char kind[kMaxBeams];  // 0 no candidates, 1 a row, 2 ended
    uint32_t bound[kMergeThreads];
    u64 warp_order[kMergeThreads / 32], warp_at[kMergeThreads / 32];
    Sum sum[kMergeThreads / 32];
    Sum slice[kMaxBeams][kHelpers];  // a row's summed weights, from each CTA of the cluster
    u64 todo;                        // rows to be summed again
    float pow2[64];
    int count, far;                  // far: a row's maximum is beyond 2^24
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

// A row's weights as multiples of 2^-bits, so that a thread's sum of its share of the
// columns stays below 2^62: 44 bits up to 2^25 columns, 38 for 2^31 - 1 without helpers.
__device__ __forceinline__ sample::Weight row_weights(float m, int64_t cols, int helpers,
                                                      const float* pow2) {
    const int64_t share = cols / (int64_t(kMergeThreads) * helpers) + 1;
    int bits = 44;
    while (share >> (62 - bits)) --bits;
    sample::Weight w;
    w.set(m, 1.f, bits, pow2);
    return w;
}

// The weights e^(x - m) of columns [from, to) of a row, summed as integers; thread 0 has
// the result.
template <typename T>
__device__ Sum exact_sum(MergeShared& sh, const sample::Weight& w, const T* row, int64_t from,
                         int64_t to) {
    constexpr int kAtOnce = 16;
    u64 mine = 0;
#pragma unroll 1
    for (int64_t c = from + threadIdx.x; c < to; c += kAtOnce * kMergeThreads) {
        float x[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            x[i] = c + i * kMergeThreads < to ? static_cast<float>(row[c + i * kMergeThreads])
                                              : -INFINITY;
        mine += w.sum_from(x, -FLT_MAX);
    }
    Sum sum = {sample::warp_sum64(mine >> 32), sample::warp_sum64(mine & 0xffffffffu)};
    __syncthreads();
    if (threadIdx.x % 32 == 0) sh.sum[threadIdx.x / 32] = sum;
    __syncthreads();
    for (int i = 1; threadIdx.x == 0 && i < kMergeThreads / 32; ++i) sum.add(sh.sum[i]);
    return sum;
}

// All CTAs of a group (threads come from branches, so the form that counts them).
__device__ __forceinline__ void group_sync(int helpers) {
    if (helpers == 1) __syncthreads();
    else
        asm volatile("barrier.cluster.arrive.release;\n\t"
                     "barrier.cluster.wait.acquire;" ::: "memory");
}

template <typename T, int KP>
__global__ void __launch_bounds__(kMergeThreads)
    beam_merge_kernel(const __grid_constant__ BeamArgs a) {
    __shared__ MergeShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t group = blockIdx.x / a.helpers, row0 = group * a.beams;
    const int rank = static_cast<int>(blockIdx.x % a.helpers);
    // this CTA's share of the rows whose sums have to be exact, into the first CTA
    auto sum_rows = [&](u64 todo) {
        const int64_t each = (a.cols + a.helpers - 1) / a.helpers;
        for (; todo; todo &= todo - 1) {
            const int i = __ffsll(static_cast<long long>(todo)) - 1;
            float m = sh.m[i];
            if (rank) {
                const uint32_t at = map_to_rank(&sh.m[i], 0);
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(m) : "r"(at) : "memory");
            }
            const sample::Weight w = row_weights(m, a.cols, a.helpers, sh.pow2);
            const Sum sum =
                exact_sum(sh, w, static_cast<const T*>(a.x) + (row0 + i) * a.cols, rank * each,
                          min(a.cols, (rank + 1) * each));
            if (tid) continue;
            if (rank) {
                const uint32_t at = map_to_rank(&sh.slice[i][rank], 0);
                asm volatile("st.shared::cluster.u64 [%0], %1;" :: "r"(at), "l"(sum.high) : "memory");
                asm volatile("st.shared::cluster.u64 [%0], %1;"
                             :: "r"(at + 8), "l"(sum.low) : "memory");
            } else {
                sh.slice[i][0] = sum;
            }
        }
    };
    if (tid == 0) sh.todo = 0, sh.far = 0;
    // (a CTA's shared memory may be written from outside once it has started)
    if (a.helpers > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    if (rank) {
        if (tid < 64) sh.pow2[tid] = sample::kPow2[tid];
        asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
        group_sync(a.helpers);
        if (sh.todo == 0) return;
        sum_rows(sh.todo);
        group_sync(a.helpers);
        return;
    }
    for (int i = tid; i < a.beams; i += kMergeThreads) {
        const float s = a.scores[row0 + i];
        sh.score[i] = s;
        sh.kind[i] = !(s > -INFINITY) ? 0 : a.ended && a.ended[row0 + i] ? 2 : 1;
    }
    if (tid < 64) sh.pow2[tid] = sample::kPow2[tid];
    __syncthreads();
    if (a.helpers > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    // ---- the lists' entries, entry by entry of all lists: a thread's first ones stay in
    // registers.
    const int lists = a.beams * a.runs, entries = lists * a.K;
    const u64* keys = a.lists + group * entries;
    constexpr int kHeld = 4;
    // (entry e of the lists begins with list e, so that a part's entries are of many lists)
    auto list_of = [&](int i) {
        const int e = i / lists;
        return (i - e * lists + e) % lists;
    };
    u64 mine[kHeld];
    int mine_of[kHeld];
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
        const int i = tid + j * kMergeThreads;
        mine_of[j] = i < entries ? list_of(i) : -1;
        mine[j] = i < entries ? __ldcg(keys + i / lists * lists + mine_of[j]) : 0;
    }
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
            if (fabsf(top) >= 0x1p24f && fabsf(top) < INFINITY) sh.far = 1;
        }
    }
    // the order of an entry's value, kNone where there is none
    auto order_of = [&](u64 key, int beam) -> u64 {
        if (key == 0) return kNone;
        if (sh.kind[beam] == 2) return order64(sh.offset[beam]);
        const float x = key_value(static_cast<uint32_t>(key >> 32));
        if (sh.m[beam] == INFINITY) return x == INFINITY ? order64(sh.offset[beam]) : kNone;
        return order64(sh.offset[beam] + (static_cast<double>(x) - sh.m64[beam]));
    };
    // f(key, beam) of the thread's entries that are continuations
    auto each = [&](auto f) {
        auto one = [&](int i, int list, u64 key) {
            const int beam = list / a.runs;
            if (sh.kind[beam] != 1) {
                // an ended beam goes on with `pad` alone
                key = sh.kind[beam] == 2 && i == beam * a.runs
                          ? (1ull << 63) | (0xffffffffu - static_cast<uint32_t>(a.pad)) : 0;
            }
            if (key) f(key, beam);
        };
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
            if (mine_of[j] >= 0) one(tid + j * kMergeThreads, mine_of[j], mine[j]);
#pragma unroll 1
        for (int i = tid + kHeld * kMergeThreads; i < entries; i += kMergeThreads) {
            const int list = list_of(i);
            one(i, list, __ldcg(keys + i / lists * lists + list));
        }
    };
    auto place_of = [](u64 key, int beam) {
        return (static_cast<u64>(beam) << 32) | (0xffffffffu - static_cast<uint32_t>(key));
    };
    // a value in fp32, and how far it may be off (its own three roundings)
    auto rough = [&](u64 key, int beam, float& slack) {
        const float off = sh.near[beam];
        float t = 0.f;
        if (sh.kind[beam] == 1) {
            const float x = key_value(static_cast<uint32_t>(key >> 32)), m = sh.m[beam];
            t = x == m ? 0.f : x - m;
        }
        slack = (fabsf(off) + fabsf(t)) * 0x1p-22f;
        return off + t;
    };
    int found = 0;
    for (int round = 0; round < 2; ++round) {
        __syncthreads();
        if (tid == 0) sh.count = 0;
        for (int i = tid; i < a.beams; i += kMergeThreads)
            if (sh.kind[i]) {
                sh.offset[i] = sh.kind[i] == 1 ? sh.score[i] - sh.lse[i] : sh.score[i];
                sh.near[i] = static_cast<float>(sh.offset[i]);
            }
        __syncthreads();
        const float eps = sh.far ? a.eps + kFarError : a.eps;
        // ---- a bound that K entries reach, less what the roundings and (in the first
        // round) the sums' errors may have taken from others
        float top = -INFINITY, slack;
        each([&](u64 key, int beam) {
            const float c = rough(key, beam, slack) - slack;
            top = fmaxf(top, c);
        });
        float bound = key_value(parts_bound<KP>(order_key(top), sh.bound));
        bound -= 4 * eps + fabsf(bound) * 0x1p-22f;
        each([&](u64 key, int beam) {
            const float c = rough(key, beam, slack) + slack;
            if (c < bound) return;
            const u64 order = order_of(key, beam);
            if (order == kNone) return;
            const int i = atomicAdd(&sh.count, 1);
            if (i < kCandidates) sh.found[i] = make_ulonglong2(order, place_of(key, beam));
        });
        __syncthreads();
        const int n = sh.count;
        if (n <= kCandidates) {
            for (int i = tid; i < n; i += kMergeThreads) {
                const ulonglong2 c = sh.found[i];
                int rank = 0;
#pragma unroll 8
                for (int j = 0; j < n; ++j) {
                    const ulonglong2 other = sh.found[j];
                    rank += better(other.x, other.y, c.x, c.y);
                }
                if (rank < a.K) {
                    sh.best[rank] = c.x;
                    sh.best_at[rank] = c.y;
                }
            }
            found = min(n, a.K);
        } else {
            // many equal values: the best of what is left in turn
            u64 c0 = ~0ull, at0 = 0;
            for (found = 0; found < a.K; ++found) {
                u64 c1 = kNone, at1 = ~0ull;
                each([&](u64 key, int beam) {
                    const u64 c = order_of(key, beam), at = place_of(key, beam);
                    if (c > kNone && (found == 0 || better(c0, at0, c, at)) &&
                        better(c, at, c1, at1))
                        c1 = c, at1 = at;
                });
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
        if (round) break;
        // ---- values of different beams that the sums cannot tell apart: neighbours in the
        // order, and of what is not chosen all that come near the last chosen
        auto mark = [&](u64 at0, u64 at1) {
            const int b0 = static_cast<int>(at0 >> 32), b1 = static_cast<int>(at1 >> 32);
            if (b0 != b1) atomicOr(&sh.todo, (1ull << b0) | (1ull << b1));
        };
        if (found > 0) {
            for (int i = tid; i + 1 < found; i += kMergeThreads)
                if (value64(sh.best[i]) - value64(sh.best[i + 1]) <= 2 * eps)
                    mark(sh.best_at[i], sh.best_at[i + 1]);
            const u64 last = sh.best[found - 1], last_at = sh.best_at[found - 1];
            const u64 low = order64(value64(last) - 2 * eps);
            auto behind = [&](u64 c, u64 at) {
                if (c >= low && better(last, last_at, c, at)) mark(last_at, at);
            };
            if (n <= kCandidates)
                for (int i = tid; i < n; i += kMergeThreads) behind(sh.found[i].x, sh.found[i].y);
            else
                each([&](u64 key, int beam) { behind(order_of(key, beam), place_of(key, beam)); });
        }
        __syncthreads();
        // what has a sum, for every CTA of the group
        u64 todo = sh.todo;
        for (u64 left = todo; left; left &= left - 1) {
            const int i = __ffsll(static_cast<long long>(left)) - 1;
            if (sh.kind[i] != 1 || sh.m[i] == INFINITY) todo &= ~(1ull << i);
        }
        if (todo && tid > 0 && tid < a.helpers) {
            const uint32_t at = map_to_rank(&sh.todo, tid);
            asm volatile("st.shared::cluster.u64 [%0], %1;" :: "r"(at), "l"(todo) : "memory");
        }
        group_sync(a.helpers);
        if (todo == 0) break;
        sum_rows(todo);
        group_sync(a.helpers);
        if (tid < a.beams && (todo >> tid & 1)) {
            const sample::Weight w = row_weights(sh.m[tid], a.cols, a.helpers, sh.pow2);
            Sum sum = {0, 0};
            for (int i = 0; i < a.helpers; ++i) sum.add(sh.slice[tid][i]);
            sh.lse[tid] = log(sum.value() / static_cast<double>(w(sh.m[tid])));
        }
    }
    if (tid < a.K) {
        const bool is = tid < found;
        const int64_t at = group * a.K + tid;
        a.out[at] = is ? static_cast<float>(value64(sh.best[tid])) : -INFINITY;
        a.parents[at] = is ? static_cast<int>(sh.best_at[tid] >> 32) : -1;
        a.tokens[at] = is ? static_cast<int>(sh.best_at[tid] & 0xffffffffu) : -1;
    }
}

}  // namespace beam
}  // namespace os
