// sample_kernel.cuh -- one draw per row of logits: temperature, top-k, top-p and
// min-p from given uniform numbers.
//
// With m the row's maximum, weights w_c = e^((x_c - m) / T).  Sorted by (logit
// descending, column ascending) the filters each keep a prefix: top-k the
// first k; top-p the shortest prefix of those whose weight reaches p times
// theirs; min-p the columns with w >= min_p.  So what stays is the columns
// with x > cut, and those with x == cut up to a last column.  The draw is the
// lowest kept column whose running sum, in column order, exceeds u times the
// kept weight.
//
// Exact draws.  Where a cut or a draw falls depends on sums of up to 2^31
// weights compared with a border, so the sums are kept as integers: a weight
// is a multiple of 2^-B (B = 62 - log2 cols, at most 44), computed in two fp32
// parts to about 2^-38 relative, and a sum of them is a 64-bit integer.  Sums
// then do not depend on how the row was split or in which order atomics came,
// and a draw that differs from the one in real arithmetic needs u within about
// 2^-38 of a border.
//
// Passes.  The row is read from memory once (maximum, and bounds for the
// cuts); what else is needed is read again from L2, where a batch's rows in
// flight stay:
//   no filter, min-p:  the kept columns' weights are summed per warp, the
//                      border's warp is found, its run summed again in pieces,
//                      and the border's piece element by element;
//   top-k (<= 1024):   the columns at or above a bound that k of them reach
//                      are listed in shared memory (a few times k), sorted,
//                      and everything else happens on the list;
//   top-p alone:       a histogram of weight in fp32, over 2048 equal steps of
//                      the logit down to where the rest could not matter, says
//                      within what few steps the border lies; one pass sums the
//                      weights above and below them per warp and lists their
//                      columns, which are sorted and complete the sums;
//   else (k larger, too many equal logits for the lists): the cut is found
//                      digit by digit of the logits' order keys over the row.
//
// One row is shared by a cluster of S CTAs (1 to 8, by the number of rows),
// each with a run of columns, which exchange through distributed shared memory.
//
// What bounds it: 256 rows of 128256 bf16 columns with one temperature take 91 us
// (0.75 TB/s of the one read; 10 us at the rate of memory) and are bound by
// instructions, 43 per column, 16 of them packed pairs that take the FMA pipe two
// cycles; top-p 0.9 150 us, a histogram more.  256 x 50257 fp32: 45 us, top-p 78, top-k 50 29.
// One row: 13 us, top-p 27, the latency of its steps over eight CTAs.  Temperature
// 0: 42 us, 24 and 10.  Rows of one value throughout, where the general cut meets
// all its atomics on one word: 256 x 50257 top-k 50 310 us, top-p 0.9 760.
#pragma once

#include <cuda_bf16.h>

#include <cfloat>
#include <climits>
#include <cstdint>

#include "ops.cuh"

namespace os {
namespace sample {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kRuns = kMaxCluster * kWarps;  // runs of columns of a row, one per warp
constexpr int kList = 2048;   // columns that a list holds
constexpr int kBins = 2048;   // steps of the top-p histogram
constexpr int kTopK = 1024;   // top-k up to here is settled on a list
constexpr float kColdest = 5e-29f;  // colder rows would leave fp32's range with 32 log2 e / T
using u64 = unsigned long long;

// 2^(j/32) in two fp32 parts, j = 0..31: the high parts, then the low ones
__device__ const float kPow2[64] = {
    0x1p+0f, 0x1.059b0ep+0f, 0x1.0b5586p+0f, 0x1.11301ep+0f, 0x1.172b84p+0f, 0x1.1d4874p+0f,
    0x1.2387a6p+0f, 0x1.29e9ep+0f, 0x1.306fep+0f, 0x1.371a74p+0f, 0x1.3dea64p+0f, 0x1.44e086p+0f,
    0x1.4bfdaep+0f, 0x1.5342b6p+0f, 0x1.5ab07ep+0f, 0x1.6247ecp+0f, 0x1.6a09e6p+0f, 0x1.71f75ep+0f,
    0x1.7a1148p+0f, 0x1.82589ap+0f, 0x1.8ace54p+0f, 0x1.93737cp+0f, 0x1.9c4918p+0f, 0x1.a5503cp+0f,
    0x1.ae89fap+0f, 0x1.b7f77p+0f, 0x1.c199bep+0f, 0x1.cb720ep+0f, 0x1.d5818ep+0f, 0x1.dfc974p+0f,
    0x1.ea4afap+0f, 0x1.f50766p+0f,
    0.f, -0x1.9d4f52p-25f, 0x1.9f3122p-25f, -0x1.fdb496p-25f, -0x1.c15742p-27f, -0x1.d2e8cap-25f,
    0x1.ceac48p-25f, -0x1.5c0424p-25f, 0x1.4636e2p-25f, -0x1.18aac6p-25f, 0x1.824684p-25f, 0x1.8624b4p-30f,
    -0x1.593abcp-25f, -0x1.2c561p-25f, -0x1.5bd5ecp-27f, -0x1.f8b55p-25f, 0x1.9fcef4p-26f, 0x1.1d8beep-25f,
    -0x1.829fdp-25f, -0x1.accc7cp-26f, 0x1.15506ep-27f, -0x1.e64744p-25f, 0x1.51f848p-27f, -0x1.b83b54p-25f,
    -0x1.a94b14p-26f, -0x1.a09438p-25f, -0x1.3d56b2p-27f, -0x1.8837ccp-27f, -0x1.822dbcp-27f, -0x1.908c94p-25f,
    0x1.52486cp-27f, -0x1.246ebp-26f};

struct Settings {
    const float* temperature;
    const int* top_k;
    const float* top_p;
    const float* min_p;
    float temperature_all;
    int top_k_all;
    float top_p_all, min_p_all;
};

__device__ __forceinline__ float widen(float v) { return fmaxf(v, -INFINITY); }  // NaN -> -inf
__device__ __forceinline__ float widen(__nv_bfloat16 v) {
    return fmaxf(__bfloat162float(v), -INFINITY);
}
// Order-preserving key; -0 counts as +0.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
constexpr uint32_t kKeyNegInf = 0x007fffffu;  // order_key(-inf)

// p 2^64 as an integer, p in [0, 1).
__device__ __forceinline__ u64 fraction64(float p) {
    const uint32_t b = __float_as_uint(p);
    const int shift = int(b >> 23) - 127 + 41;  // p = mantissa 2^(shift - 64)
    const u64 mantissa = (b & 0x7fffffu) | 0x800000u;
    if (shift < -23) return 0;  // also 0 and subnormal numbers
    return shift >= 0 ? mantissa << shift : mantissa >> -shift;
}

// A row's weight function: w(x) = e^((x - m) / T) up to a constant factor of the
// row, as a multiple of 2^-bits.
//
// With c = 32 log2 e / T in two fp32 parts, the exponent is 32 n + j + g, |g| <=
// 1/2, and 2^(g/32) = e^y with y = g ln 2 / 32; w = 2^n 2^(j/32) (1 + (e^y -
// 1)): the table-driven exponential, reduced to 1/32 of an octave.  Every product
// whose rounding would show at 2^-38 carries its residual, and the two parts of w
// are turned into integers by adding a constant whose last bit is their unit (on
// the FMA and integer pipes: the conversion instructions run at an eighth of their
// rate).  Two ways:
//   plain rows (nearly all): the exponent is x c - base with an integer base >
//     m c, two values at a time on packed pairs, 32 FMA-pipe operations per
//     column, which bound the sums' passes;
//   any row: the exponent is (x / 2 - m / 2) 2 c, the difference in two parts;
//     w(m) = 1.
struct Weight {
    float m, c_hi, c_lo;  // maximum; c
    float unit;           // 1.5 * 2^(23 - bits): its last bit is 2^-bits
    float origin;         // plain rows: the rounding constant less the base
    float clamp;          // plain rows: a lower x may stand in for any lower one
    int bits;             // 31..44
    bool plain;
    const float* table;   // kPow2 in shared memory

    __device__ __forceinline__ void set(float m_, float temperature, int bits_, const float* t) {
        constexpr float kHi = 0x1.715476p+5f, kLo = 0x1.4ae0cp-21f;  // 32 log2 e
        m = m_;
        c_hi = __fdiv_rn(kHi, temperature);
        c_lo = c_hi > 1e-30f
                   ? __fdiv_rn(fmaf(-c_hi, temperature, kHi) + kLo, temperature) : 0.f;
        bits = bits_;
        unit = 1.5f * __int_as_float((23 - bits + 127) << 23);
        table = t;
        clamp = m - __fdiv_rn(1920.f, c_hi);  // 2^-60
        // the clamp, as rounded, still far below every weight that counts, and
        // exponents small enough for their residuals
        plain = c_hi > 1e-30f && fabsf(m) * c_hi < 12000.f && fabsf(clamp) * c_hi < 14000.f &&
                (m - clamp) * c_hi > 1600.f;
        origin = expc::kRound - (ceilf(m * c_hi) + 1.f);
    }

    // 2^g/32 times the table's value: t (1 + (e^y - 1)) = wh + wl
    static __device__ __forceinline__ void scale(float g, float gl, float t, float t_lo, float& wh,
                                                 float& wl) {
        constexpr float kL = 0x1.62e43p-6f, kLLo = -0x1.05c61p-34f;  // ln 2 / 32
        const float yh = __fmul_rn(g, kL);
        const float yl = fmaf(g, kL, -yh) + fmaf(gl, kL, g * kLLo);
        const float poly = fmaf(yh, fmaf(yh, 0x1.555556p-5f, 0x1.555556p-3f), 0.5f);
        const float q = __fmul_rn(yh * yh, poly);
        const float eh = yh + q, el = (q - (eh - yh)) + yl;  // e^y - 1
        wh = fmaf(t, eh, t);
        wl = fmaf(t, el, fmaf(t, eh, t - wh) + fmaf(t_lo, eh, t_lo));
    }
    // e^((x - m) / T) = (wh + wl) 2^n by the second way; n below -60 is -200
    __device__ __forceinline__ void relative(float x, float& wh, float& wl, int& n) const {
        // halves, since x - m may be past the largest number (and still be a small
        // multiple of the temperature)
        const float xh = 0.5f * x, mh = 0.5f * m, ch = 2.f * c_hi;
        const float dh = xh - mh;
        const float bb = dh - xh;
        const float dl = (xh - (dh - bb)) + (-mh - bb);  // x / 2 - m / 2 = dh + dl exactly
        const float th = __fmul_rn(dh, ch);  // its residual is added below
        const float tl = fmaf(dh, ch, -th) + fmaf(dh, 2.f * c_lo, dl * ch);
        const float uf = th + expc::kRound;
        const float gh = th - (uf - expc::kRound);
        const float g = gh + tl;
        const int i = __float_as_int(uf);  // the constant's bits are a multiple of 32
        scale(g, tl - (g - gh), table[i & 31], table[32 + (i & 31)], wh, wl);
        n = (i - __float_as_int(expc::kRound)) >> 5;
        if (!(th > -4000.f)) n = -200;                // below 2^-125, -inf
        if (x == m) wh = 1.f, wl = 0.f, n = 0;        // also m = +inf
    }
    // (wh + wl) 2^n = hi 2^-22 + lo 2^-bits
    __device__ __forceinline__ void fix(float wh, float wl, int n, uint32_t& hi, int& lo) const {
        const float s = __int_as_float((max(n, -100) + 127) << 23);
        const float big = fmaf(wh, s, 3.f);  // last bit 2^-22
        const float rest = fmaf(wl, s, fmaf(wh, s, -(big - 3.f)));
        hi = __float_as_uint(big) - __float_as_uint(3.f);
        lo = __float_as_int(rest + unit) - __float_as_int(unit);
    }
    // The first way, two values at a time, for x in [clamp, m].  Negated values
    // save the sign changes that the packed forms lack.
    __device__ __forceinline__ void parts2(float2 x, uint32_t (&hi)[2], int (&lo)[2]) const {
        raw2(x, hi, lo);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            hi[i] -= __float_as_uint(3.f);
            lo[i] -= __float_as_int(unit);
        }
    }
    // The same with the constants that the parts were added to still in them.
    __device__ __forceinline__ void raw2(float2 x, uint32_t (&hi)[2], int (&lo)[2]) const {
        const float2 minus = splat2(-1.f), K = splat2(origin);
        const float2 np = mul2(x, splat2(-c_hi));
        const float2 pl = fma2(x, splat2(c_lo), fma2(x, splat2(c_hi), np));
        const float2 uf = fma2(np, minus, K);
        const float2 gh = fma2(np, minus, fma2(uf, minus, K));
        const float2 g = add2(gh, pl);
        const float2 gl = fma2(fma2(gh, minus, g), minus, pl);
        constexpr float kL = 0x1.62e43p-6f, kLLo = -0x1.05c61p-34f;  // ln 2 / 32
        const float2 yh = mul2(g, splat2(kL));
        const float2 nyl = fma2(g, splat2(-kL), yh);
        const float2 yl = fma2(nyl, minus, fma2(g, splat2(kLLo), mul2(gl, splat2(kL))));
        const float2 poly = fma2(yh, fma2(yh, splat2(0x1.555556p-5f), splat2(0x1.555556p-3f)),
                                 splat2(0.5f));
        const float2 yy = mul2(yh, yh);
        const float2 eh = fma2(yy, poly, yh);  // e^y - 1
        const float2 el = add2(fma2(yy, poly, fma2(eh, minus, yh)), yl);
        const int i0 = __float_as_int(uf.x), i1 = __float_as_int(uf.y);
        const float2 t = make_float2(table[i0 & 31], table[i1 & 31]);
        const float2 t_lo = make_float2(table[32 + (i0 & 31)], table[32 + (i1 & 31)]);
        const float2 wh = fma2(t, eh, t);
        const float2 wl = fma2(t, el, add2(fma2(t, eh, fma2(wh, minus, t)), fma2(t_lo, eh, t_lo)));
        // 2^n: n is the rounding constant's distance, moved to the exponent field
        const float2 s = make_float2(__int_as_float(((i0 & ~31) << 18) + 0x3f800000),
                                     __int_as_float(((i1 & ~31) << 18) + 0x3f800000));
        const float2 big = fma2(wh, s, splat2(3.f));
        const float2 rest = fma2(wl, s, fma2(wh, s, fma2(big, minus, splat2(3.f))));
        const float2 end = add2(rest, splat2(unit));
        hi[0] = __float_as_uint(big.x);
        hi[1] = __float_as_uint(big.y);
        lo[0] = __float_as_int(end.x);
        lo[1] = __float_as_int(end.y);
    }
    __device__ __forceinline__ void parts(float x, uint32_t& hi, int& lo) const {
        if (plain) {  // the same operations as a pair's, so that sums agree to the bit
            uint32_t h[2];
            int l[2];
            const float y = fmaxf(x, clamp);
            parts2(make_float2(y, y), h, l);
            hi = h[0], lo = l[0];
        } else {
            float wh, wl;
            int n;
            relative(x, wh, wl, n);
            fix(wh, wl, n, hi, lo);
            if (n < -60) hi = 0, lo = 0;
        }
    }
    __device__ __forceinline__ u64 join(uint32_t hi, int lo) const {
        const long long w = static_cast<long long>(u64(hi) << (bits - 22)) + lo;
        return w > 0 ? u64(w) : 0;
    }
    __device__ __forceinline__ u64 operator()(float x) const {
        uint32_t hi;
        int lo;
        parts(x, hi, lo);
        return join(hi, lo);
    }
    // The share of x in a sum of weights, rounded once; a weight below the
    // sums' last bit keeps its digits.
    __device__ __forceinline__ float share(float x, u64 total) const {
        float wh, wl;
        int n;
        relative(x, wh, wl, n);
        const float e = n < -126 ? 0.f : (wh + wl) * __int_as_float((n + 127) << 23);
        return float(double(e) * double((*this)(m)) / double(total));
    }

    // parts() of two values, in whichever way the row takes.
    __device__ __forceinline__ void pair(float x, float y, uint32_t (&hi)[2], int (&lo)[2]) const {
        if (plain) {
            parts2(make_float2(fmaxf(x, clamp), fmaxf(y, clamp)), hi, lo);
        } else {
            parts(fmaxf(x, -INFINITY), hi[0], lo[0]);
            parts(fmaxf(y, -INFINITY), hi[1], lo[1]);
        }
    }

    // What sums of parts amount to.
    __device__ __forceinline__ u64 sum_of(uint32_t hi, int lo) const {
        return static_cast<u64>(static_cast<long long>(u64(hi) << (bits - 22)) + lo);
    }
    // The summed weights of N values of at least `from` (finite).
    template <int N>
    __device__ __forceinline__ u64 sum_from(const float (&v)[N], float from) const {
        uint32_t hi = 0;
        int lo = 0;
        if (plain) {
            // values that do not count become the clamp, whose parts are 0;
            // sums of the parts' bits wrap, and the constants come off at once
            const float least = fmaxf(from, clamp);
            uint32_t lo_bits = 0;
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                uint32_t h[2];
                int l[2];
                raw2(make_float2(v[i] >= least ? v[i] : clamp, v[i + 1] >= least ? v[i + 1] : clamp),
                     h, l);
                hi += h[0] + h[1];
                lo_bits += uint32_t(l[0]) + uint32_t(l[1]);
            }
            hi -= uint32_t(N) * __float_as_uint(3.f);
            lo = int(lo_bits - uint32_t(N) * __float_as_uint(unit));
        } else {
#pragma unroll 1
            for (int i = 0; i < N; ++i) {
                float x = v[0];
#pragma unroll
                for (int j = 1; j < N; ++j) x = j == i ? v[j] : x;
                uint32_t h;
                int l;
                parts(x, h, l);
                if (x >= from) hi += h, lo += l;
            }
        }
        return sum_of(hi, lo);
    }
};

__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}
__device__ __forceinline__ u64 warp_prefix64(u64 v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 t = __shfl_up_sync(kFullMask, v, o);
        if (lane >= o) v += t;
    }
    return v;
}

// What stays of a row: x > value, and x == value up to column `last`.
struct alignas(8) Cut {
    float value;
    int last;
    __device__ __forceinline__ bool keeps(float x, int64_t col) const {
        return x > value || (x == value && col <= last);
    }
};

struct Shared {
    float table[64];
    // one value per warp of the row, every CTA's in each of them
    uint32_t top[kRuns], bound[kRuns];
    float near[kRuns];  // weights of a warp's run, in fp32, to its own maximum
    u64 sum[kRuns];     // weights of a warp's run outside the list
    u64 draw[kRuns];    // kept weights of a warp's run (top-p: those above the list)
    uint32_t slice[kMaxCluster];  // histogram's weight in each CTA's steps
    uint32_t bin_lo, bin_hi;  // first and last step that may hold the border
    u64 piece[kWarps];  // kept weights of a piece of the border's run
    float floor_p;
    // rank 0's findings, read by the others
    uint32_t listed;    // columns put on the list (it may be more than fit)
    Cut cut;
    uint32_t fine;      // the border's step when the listed ones are divided again
    u64 fine_above;     // weight above it
    u64 want;           // weight that the border reaches
    u64 extra[kRuns];   // kept weights of a run's listed columns
    // scratch of one CTA
    u64 warp[kWarps];
    u64 result[2];
    uint32_t found[2];
    uint32_t count[256];
    u64 list[kList];    // (order key << 32) | ~column
    union {
        u64 mass[kBins];
        uint32_t steps[kBins];
        u64 sorted[kList];
    };
};

// This CTA's address of the shared object `local` in CTA `rank` of the cluster.
template <int S, typename V>
__device__ __forceinline__ V remote(const V* local, int rank) {
    if constexpr (S == 1) {
        return *local;
    } else {
        const uint32_t a = map_to_rank(local, rank);
        V v;
        if constexpr (sizeof(V) == 8) {
            u64 t;
            asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(t) : "r"(a) : "memory");
            memcpy(&v, &t, 8);
        } else {
            uint32_t t;
            asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(t) : "r"(a) : "memory");
            memcpy(&v, &t, 4);
        }
        return v;
    }
}
// Stores a value in the row's CTA `to` (nowhere where there is none); called by a
// warp's lanes with their own numbers it stores in every CTA.  Written before a
// barrier, the value is read after it as shared memory of one's own: reads of
// other CTAs' by all their warps queue up for thousands of cycles.
template <int S, typename V>
__device__ __forceinline__ void publish(V* local, V v, int to) {
    if constexpr (S == 1) {
        if (to == 0) *local = v;
    } else if (to < S) {
        const uint32_t a = map_to_rank(local, to);
        if constexpr (sizeof(V) == 8) {
            u64 t;
            memcpy(&t, &v, 8);
            asm volatile("st.shared::cluster.u64 [%0], %1;" :: "r"(a), "l"(t) : "memory");
        } else {
            uint32_t t;
            memcpy(&t, &v, 4);
            asm volatile("st.shared::cluster.u32 [%0], %1;" :: "r"(a), "r"(t) : "memory");
        }
    }
}
// Barrier over the CTAs of a row.  Threads of a warp come to it from loops that
// they left at different times, so the cluster's barrier is the form that
// counts threads, not the .aligned one, which takes a warp for converged.
template <int S>
__device__ __forceinline__ void row_sync() {
    if constexpr (S == 1) {
        __syncthreads();
    } else {
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release;\n\t"
                     "barrier.cluster.wait.acquire;" ::: "memory");
    }
}

// Puts (x, col) on rank 0's list.
template <int S>
__device__ __forceinline__ void list_push(Shared& sh, float x, uint32_t col) {
    const u64 e = (u64(order_key(x)) << 32) | (0xffffffffu - col);
    // the lanes that are here together take their places with one addition
    const uint32_t here = __activemask();
    const int lane = threadIdx.x & 31, leader = __ffs(here) - 1;
    const uint32_t mine = __popc(here & ((1u << lane) - 1)), all = __popc(here);
    uint32_t at = 0;
    if constexpr (S == 1) {
        if (lane == leader) at = atomicAdd(&sh.listed, all);
        at = __shfl_sync(here, at, leader) + mine;
        if (at < kList) sh.list[at] = e;
    } else {
        if (lane == leader)
            asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;"
                         : "=r"(at) : "r"(map_to_rank(&sh.listed, 0)), "r"(all) : "memory");
        at = __shfl_sync(here, at, leader) + mine;
        if (at < kList)
            asm volatile("st.shared::cluster.u64 [%0], %1;"
                         :: "r"(map_to_rank(&sh.list[at], 0)), "l"(e) : "memory");
    }
}

// Puts those of a block's columns on it that `which` names: few, so one after
// the other (code for all of them side by side costs more time to fetch).
template <int S, int N>
__device__ __forceinline__ void list_push_all(Shared& sh, const float (&v)[N], uint32_t which,
                                              uint32_t col) {
#pragma unroll 1
    for (; which; which &= which - 1) {
        const int i = __ffs(which) - 1;
        float y = v[0];
#pragma unroll
        for (int j = 1; j < N; ++j) y = j == i ? v[j] : y;
        list_push<S>(sh, y, col + i);
    }
}

// How many are on it while others are being put there.
template <int S>
__device__ __forceinline__ uint32_t listed_now(Shared& sh) {
    if constexpr (S == 1) return *static_cast<volatile uint32_t*>(&sh.listed);
    else return remote<S>(&sh.listed, 0);
}

// Sorts list[0, n) into sorted[0, n), best (key, lower column) first.  Up to
// 512 entries are ranked by counting (one thread per entry, no barriers); more
// by a bitonic network.  All threads of the CTA.
__device__ __forceinline__ void sort_list(Shared& sh, int n) {
    const int tid = threadIdx.x;
    if (n <= kThreads) {
        if (tid < n) {
            const u64 mine = sh.list[tid];
            int rank = 0;
#pragma unroll 8
            for (int i = 0; i < n; ++i) rank += sh.list[i] > mine;
            sh.sorted[rank] = mine;  // entries differ: each has a column of its own
        }
        __syncthreads();
        return;
    }
    int size = 1024;
    while (size < n) size *= 2;
    for (int i = tid; i < size; i += kThreads) sh.sorted[i] = i < n ? sh.list[i] : 0ull;
    for (int width = 2; width <= size; width *= 2)
        for (int step = width / 2; step > 0; step /= 2) {
            __syncthreads();
            for (int i = tid; i < size / 2; i += kThreads) {
                const int a = 2 * i - (i & (step - 1)), b = a + step;
                const u64 p = sh.sorted[a], q = sh.sorted[b];
                if ((p < q) == ((a & width) == 0)) {
                    sh.sorted[a] = q;
                    sh.sorted[b] = p;
                }
            }
        }
    __syncthreads();
}

// Adds to a 64-bit sum in shared memory by 32-bit additions, the carry handed on
// by whoever caused it (with 64-bit atomics, which try again whenever another
// thread was there first, 256 x 50257 with top-k 1025 takes 820 us, so 134).
__device__ __forceinline__ void add64(u64* sum, u64 v) {
    uint32_t* const word = reinterpret_cast<uint32_t*>(sum);
    const uint32_t lo = uint32_t(v), old = atomicAdd(word, lo);
    const uint32_t hi = uint32_t(v >> 32) + (old + lo < old);
    if (hi) atomicAdd(word + 1, hi);
}

// Inclusive prefix sum of one value per thread over the CTA.
__device__ __forceinline__ u64 cta_prefix(Shared& sh, u64 v) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = warp_prefix64(v, lane);
    __syncthreads();
    if (lane == 31) sh.warp[warp] = v;
    __syncthreads();
    for (int i = 0; i < warp; ++i) v += sh.warp[i];
    return v;
}
__device__ __forceinline__ u64 cta_sum(Shared& sh, u64 v) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = warp_sum64(v);
    __syncthreads();
    if (lane == 0) sh.warp[warp] = v;
    __syncthreads();
    u64 t = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) t += sh.warp[i];
    return t;
}

// p (in [0, 1]) times `total`, rounded up: the least integer that is at least
// the product.
__device__ __forceinline__ u64 share_of(float p, u64 total) {
    const u64 frac = fraction64(p);  // p < 1
    const u64 want = __umul64hi(frac, total) + (frac * total != 0);
    return want > 0 ? want : 1;
}

// ------------------------------------------------------------------ the general cut
// Digit by digit from the top, the largest key T such that the elements with
// key >= T amount to at least `want`, an element amounting to amount(key) (its
// count or its weight).  On return `above` is what the keys > T amount to and
// `ties` the number of elements with key T.  each(f) calls f(key, times) for
// every element of the calling thread's share.
template <typename Each, typename Amount>
__device__ uint32_t select_key(Shared& sh, u64 want, Each each, Amount amount, u64& above,
                               uint32_t& ties) {
    uint32_t prefix = 0;
    above = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        __syncthreads();
        if (threadIdx.x < 256) {
            sh.mass[threadIdx.x] = 0;
            sh.count[threadIdx.x] = 0;
        }
        __syncthreads();
        each([&](uint32_t key, uint32_t times) {
            if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8))) {
                const int b = (key >> shift) & 255;
                add64(&sh.mass[b], amount(key) * times);
                atomicAdd(&sh.count[b], times);
            }
        });
        __syncthreads();
        if (threadIdx.x < 32) {
            // bins from the top: lane l has bins 255 - 8 l .. 248 - 8 l
            const int lane = threadIdx.x;
            u64 own = 0;
            for (int i = 0; i < 8; ++i) own += sh.mass[255 - 8 * lane - i];
            const u64 upto = warp_prefix64(own, lane) + above;
            const uint32_t hit = __ballot_sync(kFullMask, upto >= want);
            const int src = hit ? __ffs(hit) - 1 : 31;
            if (lane == src) {
                u64 run = upto - own;
                int b = 255 - 8 * lane;
                for (int i = 0; i < 7 && run + sh.mass[b] < want; ++i) run += sh.mass[b--];
                sh.result[0] = run;
                sh.found[0] = b;
                sh.found[1] = sh.count[b];
            }
        }
        __syncthreads();
        above = sh.result[0];
        prefix |= sh.found[0] << shift;
        ties = sh.found[1];
    }
    return prefix;
}

// The cut of top-k and top-p by one CTA over the whole row.
template <typename T>
__device__ __noinline__ Cut general_cut(Shared& sh, const T* p, int cols, const Weight w, int k,
                                        float tp) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t cut = kKeyNegInf, room = 0;  // keys > cut stay, and `room` columns at it
    bool some = false;                    // only the first `room`, there are more
    auto each_all = [&](auto f) {
        for (int64_t i = tid; i < cols; i += kThreads) f(order_key(widen(p[i])), 1u);
    };
    if (k > 0 && k < cols) {
        u64 above;
        uint32_t ties;
        cut = select_key(sh, u64(k), each_all, [](uint32_t) { return 1ull; }, above, ties);
        room = uint32_t(k - above);
        some = room < ties;
        if (cut <= kKeyNegInf) {
            cut = kKeyNegInf;
            some = false;
            room = 0;
        }
    }
    if (tp < 1.f) {
        u64 total = 0;
        for (int64_t i = tid; i < cols; i += kThreads) {
            const float v = widen(p[i]);
            if (order_key(v) > cut) total += w(v);
        }
        const u64 w_cut = cut > kKeyNegInf ? w(key_value(cut)) : 0;
        total = cta_sum(sh, total) + w_cut * room;
        const u64 want = share_of(fmaxf(tp, 0.f), total);
        const uint32_t cut_k = cut, room_k = room;
        u64 above;
        uint32_t ties;
        auto each_kept = [&](auto f) {
            each_all([&](uint32_t key, uint32_t) {
                if (key > cut_k) f(key, 1u);
            });
            if (tid == 0 && room_k > 0) f(cut_k, room_k);
        };
        cut = select_key(sh, want, each_kept, [&](uint32_t key) { return w(key_value(key)); },
                         above, ties);
        const u64 wt = w(key_value(cut));
        room = wt > 0 ? uint32_t((want - above + wt - 1) / wt) : ties;
        if (room > ties) room = ties;
        some = cut == cut_k ? (some || room < room_k) : room < ties;
    }
    if (cut <= kKeyNegInf) return {-FLT_MAX, INT_MAX};
    if (!some) return {key_value(cut), INT_MAX};
    // the last of the first `room` columns at the cut: runs of columns per warp
    const int64_t per_warp = (int64_t(cols) + kThreads - 1) / kThreads * 32;
    const int64_t lo = min(int64_t(cols), warp * per_warp);
    const int64_t hi = min(int64_t(cols), (warp + 1) * per_warp);
    uint32_t mine = 0;
    for (int64_t i = lo + lane; i < hi; i += 32) mine += order_key(widen(p[i])) == cut;
    mine = __reduce_add_sync(kFullMask, mine);
    __syncthreads();
    if (lane == 0) sh.warp[warp] = mine;
    __syncthreads();
    uint32_t before = 0;
    for (int i = 0; i < warp; ++i) before += uint32_t(sh.warp[i]);
    if (before < room && room <= before + mine) {
        for (int64_t i0 = lo; i0 < hi; i0 += 32) {
            const bool tie = i0 + lane < hi && order_key(widen(p[i0 + lane])) == cut;
            const uint32_t b = __ballot_sync(kFullMask, tie);
            if (before + __popc(b) >= room) {
                const uint32_t upto = before + __popc(b & (0xffffffffu >> (31 - lane)));
                if (tie && upto == room) sh.found[0] = uint32_t(i0 + lane);
                break;
            }
            before += __popc(b);
        }
    }
    __syncthreads();
    return {key_value(cut), int(sh.found[0])};
}

// ------------------------------------------------------------------ the kernel
// The 16-byte blocks of memory that a row covers: block b holds columns
// b * EPV - head .. b * EPV - head + EPV - 1, those outside the row read as -inf.
template <typename T>
struct Blocks {
    static constexpr int EPV = VecTraits<T>::EPV;
    const T* base;  // 16-byte aligned, `head` elements before the row
    int head, cols;
    int64_t count;
    __device__ __forceinline__ Blocks(const T* row, int cols_) : cols(cols_) {
        head = int((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
        base = row - head;
        count = (int64_t(head) + cols + EPV - 1) / EPV;
    }
    __device__ __forceinline__ int64_t col(int64_t b) const { return b * EPV - head; }
    __device__ __forceinline__ bool whole(int64_t b) const {
        return col(b) >= 0 && col(b) + EPV <= cols;
    }
    __device__ __forceinline__ uint4 words(int64_t b) const {
        return __ldg(reinterpret_cast<const uint4*>(base) + b);
    }
    // a NaN stays one: it fails every comparison and is passed over by maxima
    __device__ __forceinline__ void load(int64_t b, float (&v)[EPV]) const {
        const int64_t c = col(b);
        if (whole(b)) {
            const uint4 w = words(b);
            const uint32_t a[4] = {w.x, w.y, w.z, w.w};
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(a[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = unpack_bf16x2(a[i]);
                    v[2 * i] = f.x;
                    v[2 * i + 1] = f.y;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPV; ++i)
                v[i] = c + i >= 0 && c + i < cols ? widen(base[b * EPV + i]) : -INFINITY;
        }
    }
    // The largest value of the blocks b, b + 32, ... below `end`.
    __device__ __forceinline__ float maximum(int64_t b, int64_t end) const {
        float top = -INFINITY;
        if constexpr (sizeof(T) == 4) {
#pragma unroll 4
            for (; b < end; b += 32) {
                float v[EPV];
                load(b, v);
                top = fmaxf(max3(top, v[0], v[1]), fmaxf(v[2], v[3]));
            }
        } else {
            __nv_bfloat162 best = __float2bfloat162_rn(-INFINITY);
#pragma unroll 4
            for (; b < end; b += 32) {
                if (whole(b)) {
                    const uint4 w = words(b);
                    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        best = __hmax2(best, *reinterpret_cast<const __nv_bfloat162*>(&a[i]));
                } else {
                    float v[EPV];
                    load(b, v);
#pragma unroll
                    for (int i = 0; i < EPV; ++i) top = fmaxf(top, v[i]);
                }
            }
            top = fmaxf(top, fmaxf(__low2float(best), __high2float(best)));
        }
        return top;
    }
    // The same with the sum d of 2^((x - maximum) c) in fp32.
    __device__ __forceinline__ float maximum_and_sum(int64_t b, int64_t end, float c, float& d) const {
        float top = -INFINITY;
        d = 0.f;
#pragma unroll 2
        for (; b < end; b += 32) {
            float v[EPV];
            load(b, v);
            float best = -INFINITY;
#pragma unroll
            for (int i = 0; i < EPV; ++i) {
                v[i] = fmaxf(v[i], -INFINITY);  // a NaN counts for nothing
                best = fmaxf(best, v[i]);
            }
            if (best == -INFINITY) continue;
            if (best > top) {
                d *= ex2_sfu((top - best) * c);  // 0 at first
                top = best;
            }
            float part = 0.f;
#pragma unroll
            for (int i = 0; i < EPV; ++i) part += ex2_sfu((v[i] - top) * c);
            d += part;
        }
        return top;
    }
};

// The weights that stay of a row, in column order.  Columns at the cut and past
// its last one are summed with the rest and taken off again; column by column
// where every kept column counts (u = 0).
template <typename T>
struct Kept {
    static constexpr int EPV = Blocks<T>::EPV;
    Blocks<T> blocks;
    Weight w;
    Cut cut;
    u64 w_cut;  // w(cut.value) where the cut goes through equal logits
    bool by_column;

    __device__ __forceinline__ u64 column(float v, int64_t c) const {
        if (!cut.keeps(v, c)) return 0;
        const u64 a = w(v);
        return by_column && a == 0 ? 1ull : a;  // u = 0: the first column, however small
    }
    __device__ __forceinline__ u64 block(int64_t b) const {
        float v[EPV];
        blocks.load(b, v);
        u64 a = 0;
        if (!by_column) {
            a = w.sum_from(v, cut.value);
            if (cut.last != INT_MAX) {
#pragma unroll
                for (int i = 0; i < EPV; ++i)
                    if (v[i] == cut.value && blocks.col(b) + i > cut.last) a -= w_cut;
            }
            return a;
        }
        bool any = false;
#pragma unroll
        for (int i = 0; i < EPV; ++i) any |= v[i] >= cut.value;
        if (any) {
#pragma unroll 1
            for (int j = 0; j < EPV; ++j) {
                float y = v[0];
#pragma unroll
                for (int i = 1; i < EPV; ++i) y = i == j ? v[i] : y;
                a += column(y, blocks.col(b) + j);
            }
        }
        return a;
    }
};

template <typename T, int S>
__global__ void __launch_bounds__(kThreads, 2)
sample_kernel(const T* __restrict__ x, const float* __restrict__ u, int* __restrict__ out,
              float* __restrict__ prob, int64_t rows, int cols, const Settings s, int bits) {
    constexpr int EPV = VecTraits<T>::EPV;
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = S == 1 ? 0 : int(cluster_rank());
    if (tid < 64) sh.table[tid] = kPow2[tid];
    // the row's other CTAs have to be there before anything is stored in them:
    // asked for here, waited for after the first pass
    if constexpr (S > 1) {
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    }
    bool first_row = true;
    const int own_run = rank * kWarps + warp;  // this warp's run of columns
    for (int64_t row = blockIdx.x / S; row < rows; row += gridDim.x / S) {
        const Blocks<T> blocks(x + row * cols, cols);
        // runs of blocks, in column order: CTA by CTA, warp by warp
        const int64_t per_warp = (blocks.count + S * kThreads - 1) / (S * kThreads) * 32;
        const int64_t lo = min(blocks.count, (rank * kWarps + warp) * per_warp);
        const int64_t hi = min(blocks.count, lo + per_warp);
        float t_row = s.temperature ? s.temperature[row] : s.temperature_all;
        if (t_row > 0.f) t_row = fmaxf(t_row, kColdest);
        const int k = s.top_k ? s.top_k[row] : s.top_k_all;
        const float tp = s.top_p ? s.top_p[row] : s.top_p_all;
        const float mp = s.min_p ? s.min_p[row] : s.min_p_all;
        float uu = u[row] > 0.f ? fminf(u[row], 0x1.fffffep-1f) : 0.f;
        const bool by_k = k > 0 && k < cols;
        // warps with a whole run: those whose thread maxima bound the k-th best
        const int full = int(blocks.count / per_warp);
        const bool list_k = by_k && k <= kTopK && k <= 32 * full;

        // ---- the only pass over memory: maxima per thread, for top-p the weight
        const bool by_p = !by_k && tp < 1.f && t_row > 0.f;
        const float c_near = __fdiv_rn(1.442695041f, t_row);
        float near = 0.f;
        const float thread_top = by_p ? blocks.maximum_and_sum(lo + lane, hi, c_near, near)
                                      : blocks.maximum(lo + lane, hi);
        uint32_t key = order_key(thread_top);
        const uint32_t warp_top = __reduce_max_sync(kFullMask, key);
        if (by_p) {
            const float t = key_value(warp_top);
            near = near == 0.f ? 0.f : near * ex2_sfu((thread_top - t) * c_near);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) near += __shfl_xor_sync(kFullMask, near, o);
            for (int i = tid; i < kBins; i += kThreads) sh.steps[i] = 0;
            if (tid < S * kWarps) sh.extra[tid] = 0;
        }
        uint32_t bound = 0xffffffffu;
        if (list_k && rank * kWarps + warp < full) {
            // every such warp's j-th best thread maximum, j = ceil(k / warps):
            // the smallest of them is reached by j threads in every warp, so by
            // k elements.  The lanes' keys are sorted descending to find it.
            const int j = (k + full - 1) / full;
#pragma unroll
            for (int width = 2; width <= 32; width *= 2)
#pragma unroll
                for (int step = width / 2; step > 0; step /= 2) {
                    const uint32_t o = __shfl_xor_sync(kFullMask, key, step);
                    const bool first = (lane & step) == 0, down = (lane & width) == 0;
                    key = first == down ? max(key, o) : min(key, o);
                }
            bound = __shfl_sync(kFullMask, key, j - 1);
        }
        if constexpr (S > 1) {
            if (first_row) {
                __syncwarp();
                asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
            }
            first_row = false;
        }
        publish<S>(&sh.top[own_run], warp_top, lane);
        if (list_k) publish<S>(&sh.bound[own_run], bound, lane);
        if (by_p) publish<S>(&sh.near[own_run], near, lane);
        if (tid == 0) {
            sh.listed = 0;
            sh.bin_lo = sh.bin_hi = kBins;  // none
            sh.cut = {NAN, 0};
        }
        row_sync<S>();
        uint32_t top_key = 0;
        bound = 0xffffffffu;
        for (int i = lane; i < S * kWarps; i += 32) {
            top_key = max(top_key, sh.top[i]);
            if (list_k) bound = min(bound, sh.bound[i]);
        }
        top_key = __reduce_max_sync(kFullMask, top_key);
        bound = __reduce_min_sync(kFullMask, bound);

        Weight w;
        const bool greedy = !(t_row > 0.f);
        w.set(key_value(top_key), greedy ? 1.f : t_row, bits, sh.table);
        // the lowest logit that min-p keeps; compared in fp32 it decides as in
        // real arithmetic, since it is rounded up
        float floor_p = -FLT_MAX;
        if (mp > 0.f && !greedy) {
            const float q = fminf(mp, 1.f);
            floor_p = w.m;
            if (q < 1.f) {  // 64-bit arithmetic, slow here: one warp does it
                if (warp == 0) {
                    const float f = __double2float_ru(double(w.m) + double(t_row) * log(double(q)));
                    if (lane == 0) sh.floor_p = f;
                }
                __syncthreads();
                floor_p = sh.floor_p;
            }
        }
        auto write = [&](int64_t c, float v, u64 total) {
            out[row] = int(c);
            if (prob) prob[row] = greedy ? 1.f : w.share(v, total);
        };
        auto target_of = [&](u64 total) {
            return __umul64hi(fraction64(uu), total);
        };

        bool done = false, have_runs = false;
        Cut cut = {-FLT_MAX, INT_MAX};
        if (top_key <= kKeyNegInf) {
            if (rank == 0 && tid == 0) {
                out[row] = -1;
                if (prob) prob[row] = 0.f;
            }
            done = true;
        } else if (greedy) {
            cut.value = w.m;
            uu = 0.f;  // the first kept column
        } else {
            bool settled = !by_k && !(tp < 1.f);
            if (list_k) {
                // ---- top-k on a list.  Where a mask leaves a warp too few
                // columns for a bound, all that are there, while they fit
                // (256 x 50257 with 100 columns left, top-k 50: 157 us by the
                // general cut, 29 so)
                const bool all = bound <= kKeyNegInf;
                const float least = all ? -FLT_MAX : key_value(bound);
#pragma unroll 2
                for (int64_t b = lo + lane; b < hi; b += 32) {
                    if (all && listed_now<S>(sh) > kList) break;
                    float v[EPV];
                    blocks.load(b, v);
                    uint32_t for_list = 0;
#pragma unroll
                    for (int i = 0; i < EPV; ++i)
                        if (v[i] >= least) for_list |= 1u << i;
                    list_push_all<S>(sh, v, for_list, uint32_t(blocks.col(b)));
                }
                row_sync<S>();
                const uint32_t n = remote<S>(&sh.listed, 0);
                if (n <= kList) {
                    const int stay = min(k, int(n));
                    settled = done = true;
                    if (rank == 0) {
                        sort_list(sh, int(n));
                        // thread t: sorted entries 2t, 2t + 1 (k <= 1024)
                        u64 e[2], a[2];
                        float v[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            e[i] = 2 * tid + i < stay ? sh.sorted[2 * tid + i] : 0;
                            v[i] = e[i] ? key_value(uint32_t(e[i] >> 32)) : -INFINITY;
                            a[i] = e[i] ? w(v[i]) : 0;
                        }
                        const u64 upto1 = cta_prefix(sh, a[0] + a[1]), upto0 = upto1 - a[1];
                        __syncthreads();
                        if (tid == kThreads - 1) sh.result[0] = upto1;
                        __syncthreads();
                        if (tp < 1.f) {
                            const u64 want = share_of(fmaxf(tp, 0.f), sh.result[0]);
                            if (upto0 - a[0] >= want) a[0] = 0, v[0] = -INFINITY;
                            if (upto0 >= want) a[1] = 0, v[1] = -INFINITY;
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (!(v[i] >= floor_p)) a[i] = 0, v[i] = -INFINITY;
                        // what stays, as (column, weight): list and sorted hold them
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if (uu == 0.f && v[i] > -INFINITY && a[i] == 0) a[i] = 1;
                            sh.list[2 * tid + i] = 0xffffffffu - uint32_t(e[i]);
                        }
                        const u64 total = cta_sum(sh, a[0] + a[1]);
                        sh.sorted[2 * tid] = a[0];
                        sh.sorted[2 * tid + 1] = a[1];
                        __syncthreads();
                        const u64 target = target_of(total);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if (a[i] == 0) continue;
                            const u64 col = 0xffffffffu - uint32_t(e[i]);
                            u64 before = 0;
                            for (int j = 0; j < stay; ++j) before += sh.list[j] < col ? sh.sorted[j] : 0;
                            if (before <= target && target < before + a[i])
                                write(int64_t(col), v[i], total);
                        }
                    }
                }
            } else if (by_p) {
                // ---- top-p.  The fp32 total says how far down the border may
                // lie: columns of at most (1 - p) total / cols cannot reach it
                // even together.
                near = 0.f;
                for (int i = lane; i < S * kWarps; i += 32) {
                    const float part = sh.near[i], t = key_value(sh.top[i]);
                    near += part == 0.f ? 0.f : part * ex2_sfu((t - w.m) * c_near);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) near += __shfl_xor_sync(kFullMask, near, o);
                // (infinite logits or temperatures make it NaN: the general cut)
                const float pc = fmaxf(tp, 0.f);
                const float log_small = 0.6931472f * __log2f((1.f - pc) * near * 0.999f / float(cols));
                const float low = w.m + t_row * log_small;
                const float least = fmaxf(
                    low - 1e-5f * (fabsf(w.m) + t_row * (1.f + fabsf(log_small))), -FLT_MAX);
                const float steps = float(kBins) / (w.m - least);
                if (w.m < INFINITY && steps > 0.f && steps < INFINITY && near < INFINITY) {
                    // weights in units of total 2^-31
                    const float scale = 0x1p31f / near;
                    for (int64_t b = lo + lane; b < hi; b += 32) {
                        float v[EPV];
                        blocks.load(b, v);
#pragma unroll
                        for (int i = 0; i < EPV; ++i)
                            if (v[i] >= least)
                                atomicAdd(&sh.steps[min(kBins - 1, int((w.m - v[i]) * steps))],
                                          __float2uint_rn(ex2_sfu((v[i] - w.m) * c_near) * scale));
                    }
                    row_sync<S>();
                    // every CTA adds up a share of the steps over the cluster;
                    // the border lies where the running weight comes within
                    // `slack` of p: every weight and the total are good to 1e-5
                    // (a difference rounded, at most 60 octaves, and the SFU's
                    // error), and half a unit per column is rounded away
                    constexpr int kShare = kBins / S;
                    constexpr int B = kShare > kThreads ? kShare / kThreads : 1;
                    uint32_t part[B], own = 0;
#pragma unroll
                    for (int i = 0; i < B; ++i) {
                        part[i] = 0;
                        if (B * tid + i < kShare)
#pragma unroll
                            for (int r = 0; r < S; ++r)
                                part[i] += remote<S>(&sh.steps[kShare * rank + B * tid + i], r);
                        own += part[i];
                    }
                    const u64 upto = cta_prefix(sh, own);
                    if (warp == kWarps - 1)
                        publish<S>(&sh.slice[rank], uint32_t(__shfl_sync(kFullMask, upto, 31)), lane);
                    row_sync<S>();
                    u64 run = upto - own;
                    for (int r = 0; r < rank; ++r) run += sh.slice[r];
                    const float slack = 3e-5f + float(cols) * 0x1p-31f;
                    const float from = (pc - slack) * 0x1p31f, to = (pc + slack) * 0x1p31f;
#pragma unroll
                    for (int i = 0; i < B; ++i) {
                        const float before = float(run), after = float(run + part[i]);
                        // steps whose end reaches `from`, and the first that reaches `to`
                        if (B * tid + i < kShare) {
                            const uint32_t step = kShare * rank + B * tid + i;
                            if (after >= from && (before < from || step == 0))
                                for (int r = 0; r < S; ++r) publish<S>(&sh.bin_lo, step, r);
                            if (after >= to && before < to)
                                for (int r = 0; r < S; ++r) publish<S>(&sh.bin_hi, step, r);
                        }
                        run += part[i];
                    }
                    row_sync<S>();
                    const int bin_lo = int(sh.bin_lo), bin_hi = int(sh.bin_hi);
                    // weights above those steps, below them, and the columns in
                    // them; not needed where min-p cuts above them
                    const float from_step = float(bin_lo);
                    const float to_step = bin_hi >= kBins - 1 ? INFINITY : float(bin_hi + 1);
                    if (bin_lo < kBins && (w.m - floor_p) * steps < from_step) settled = true;
                    u64 above = 0, rest = 0;
                    for (int64_t b = settled ? hi : lo + lane; b < hi; b += 32) {
                        float v[EPV];
                        blocks.load(b, v);
                        uint32_t hi_a = 0, hi_r = 0, for_list = 0;
                        int lo_a = 0, lo_r = 0;
#pragma unroll
                        for (int i = 0; i < EPV; i += 2) {
                            uint32_t h[2];
                            int l[2];
                            w.pair(v[i], v[i + 1], h, l);
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const float at = (w.m - v[i + j]) * steps;
                                if (v[i + j] >= least && at < to_step) {
                                    if (at < from_step) hi_a += h[j], lo_a += l[j];
                                    else for_list |= 1u << (i + j);
                                } else {
                                    hi_r += h[j], lo_r += l[j];
                                }
                            }
                        }
                        above += w.sum_of(hi_a, lo_a);
                        rest += w.sum_of(hi_r, lo_r);
                        list_push_all<S>(sh, v, for_list, uint32_t(blocks.col(b)));
                    }
                    above = warp_sum64(above);
                    rest = warp_sum64(rest);
                    publish<S>(&sh.draw[own_run], above, lane);
                    publish<S>(&sh.sum[own_run], above + rest, lane);
                    row_sync<S>();
                    const uint32_t n = remote<S>(&sh.listed, 0);
                    if (n > 0 && n <= kList) {
                        if (rank == 0) {
                            u64 total = 0, top_sum = 0;
                            for (int i = lane; i < S * kWarps; i += 32) {
                                total += sh.sum[i];
                                top_sum += sh.draw[i];
                            }
                            total = warp_sum64(total);
                            top_sum = warp_sum64(top_sum);
                            sort_list(sh, int(n));
                            // weights beside the sorted entries, in the list's place
                            u64 mine = 0;
#pragma unroll 1
                            for (int at = tid; at < int(n); at += kThreads) {
                                const u64 a = w(key_value(uint32_t(sh.sorted[at] >> 32)));
                                sh.list[at] = a;
                                mine += a;
                            }
                            const u64 want = share_of(pc, total + cta_sum(sh, mine));
                            u64 run_sum = top_sum;  // before this chunk of entries
#pragma unroll 1
                            for (int base = 0; base < int(n); base += kThreads) {
                                const int at = base + tid;
                                const u64 a = at < int(n) ? sh.list[at] : 0;
                                const u64 upto = run_sum + cta_prefix(sh, a);
                                if (at < int(n) && upto - a < want) {  // stays
                                    const u64 e = sh.sorted[at];
                                    const uint32_t col = 0xffffffffu - uint32_t(e);
                                    const uint32_t block = (col + uint32_t(blocks.head)) / EPV;
                                    add64(&sh.extra[block / uint32_t(per_warp)], a);
                                    if (want <= upto && top_sum < want)
                                        sh.cut = {key_value(uint32_t(e >> 32)), int(col)};
                                }
                                __syncthreads();
                                if (tid == kThreads - 1) sh.result[0] = upto;
                                __syncthreads();
                                run_sum = sh.result[0];
                            }
                            if (S > 1 && warp < S) {  // for the others' copies
                                for (int i = lane; i < S * kWarps; i += 32)
                                    publish<S>(&sh.extra[i], sh.extra[i], warp);
                                if (lane == 0) publish<S>(&sh.cut, sh.cut, warp);
                            }
                        }
                        row_sync<S>();
                        cut = sh.cut;
                        settled = cut.value == cut.value;  // found
                        have_runs = settled && uu != 0.f;
                    } else if (n > kList) {
                        // many small weights at the border (p close to 1):
                        // divide those steps into 2048 again, by exact weights
                        const float first = from_step;
                        const float range = fminf(to_step, (w.m - least) * steps) - first;
                        const float fine = float(kBins) / range;
                        auto fine_of = [&](float v) {
                            return min(kBins - 1, int(((w.m - v) * steps - first) * fine));
                        };
                        auto in_border = [&](float v) {
                            const float at = (w.m - v) * steps;
                            return v >= least && at < to_step && at >= from_step;
                        };
                        for (int i = tid; i < kBins; i += kThreads) sh.mass[i] = 0;
                        if (tid == 0) sh.fine = kBins;  // none
                        row_sync<S>();
                        // only now has every thread of the row read the first list's
                        // length; the barrier before the next columns orders this
                        if (tid == 0) sh.listed = 0;
                        for (int64_t b = lo + lane; b < hi; b += 32) {
                            float v[EPV];
                            blocks.load(b, v);
#pragma unroll
                            for (int i = 0; i < EPV; i += 2) {
                                uint32_t h[2];
                                int l[2];
                                w.pair(v[i], v[i + 1], h, l);
#pragma unroll
                                for (int j = 0; j < 2; ++j)
                                    if (in_border(v[i + j]))
                                        add64(&sh.mass[fine_of(v[i + j])], w.join(h[j], l[j]));
                            }
                        }
                        row_sync<S>();
                        if (rank == 0) {
                            u64 total = 0, top_sum = 0;
                            for (int i = lane; i < S * kWarps; i += 32) {
                                total += sh.sum[i];
                                top_sum += sh.draw[i];
                            }
                            total = warp_sum64(total);
                            top_sum = warp_sum64(top_sum);
                            constexpr int F = kBins / kThreads;
                            u64 part[F], mine = 0;
#pragma unroll
                            for (int i = 0; i < F; ++i) {
                                part[i] = 0;
                                for (int r = 0; r < S; ++r)
                                    part[i] += remote<S>(&sh.mass[F * tid + i], r);
                                mine += part[i];
                            }
                            const u64 upto = cta_prefix(sh, mine);
                            if (tid == kThreads - 1) sh.result[0] = upto;
                            __syncthreads();
                            const u64 want = share_of(pc, total + sh.result[0]);
                            u64 run = top_sum + upto - mine;
                            if (run < want && want <= run + mine && top_sum < want) {
                                int i = 0;
                                while (i < F - 1 && run + part[i] < want) run += part[i++];
                                sh.fine = F * tid + i;
                                sh.fine_above = run;
                                sh.want = want;
                            }
                        }
                        row_sync<S>();
                        const int step = int(remote<S>(&sh.fine, 0));
                        if (step < kBins)
                            for (int64_t b = lo + lane; b < hi; b += 32) {
                                float v[EPV];
                                blocks.load(b, v);
                                uint32_t for_list = 0;
#pragma unroll
                                for (int i = 0; i < EPV; ++i)
                                    if (in_border(v[i]) && fine_of(v[i]) == step) for_list |= 1u << i;
                                list_push_all<S>(sh, v, for_list, uint32_t(blocks.col(b)));
                            }
                        row_sync<S>();
                        const uint32_t n_fine = remote<S>(&sh.listed, 0);
                        if (n_fine > 0 && n_fine <= kList) {
                            if (rank == 0) {
                                sort_list(sh, int(n_fine));
                                constexpr int P = kList / kThreads;
                                u64 a[P], mine = 0;
#pragma unroll
                                for (int i = 0; i < P; ++i) {
                                    const int at = P * tid + i;
                                    a[i] = at < int(n_fine) ? w(key_value(uint32_t(sh.sorted[at] >> 32))) : 0;
                                    mine += a[i];
                                }
                                const u64 upto = cta_prefix(sh, mine) + sh.fine_above, want = sh.want;
                                u64 run = upto - mine;
                                if (run < want && want <= upto) {
                                    int i = 0;
                                    while (i < P - 1 && run + a[i] < want) run += a[i++];
                                    const u64 e = sh.sorted[P * tid + i];
                                    sh.cut = {key_value(uint32_t(e >> 32)),
                                              int(0xffffffffu - uint32_t(e))};
                                }
                            }
                            row_sync<S>();
                            cut = remote<S>(&sh.cut, 0);
                            settled = cut.value == cut.value;  // found
                        }
                    }
                }
            }
            if (!settled) {
                row_sync<S>();
                if (rank == 0) {
                    const Cut c = general_cut<T>(sh, x + row * cols, cols, w, k, tp);
                    __syncthreads();
                    if (tid == 0) sh.cut = c;
                }
                row_sync<S>();
                cut = remote<S>(&sh.cut, 0);
            }
            if (floor_p > cut.value) {
                cut = {floor_p, INT_MAX};
                have_runs = false;
            }
        }

        if (!done) {
            // ---- the draw, in column order
            const Kept<T> kept = {blocks, w, cut, cut.last != INT_MAX ? w(cut.value) : 0, uu == 0.f};
            if (!have_runs) {
                u64 mine = 0;
#pragma unroll 2
                for (int64_t b = lo + lane; b < hi; b += 32) mine += kept.block(b);
                mine = warp_sum64(mine);
                publish<S>(&sh.draw[own_run], mine, lane);
                row_sync<S>();
            }
            // the run that holds the border: before <= target < before + its sum
            constexpr int R = (S * kWarps + 31) / 32;  // runs per lane, in order
            u64 part[R], own = 0;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int g = R * lane + i;
                part[i] = g < S * kWarps ? sh.draw[g] : 0;
                if (have_runs && g < S * kWarps) part[i] += sh.extra[g];
                own += part[i];
            }
            const u64 upto = warp_prefix64(own, lane);
            const u64 total = __shfl_sync(kFullMask, upto, 31), target = target_of(total);
            const int src = __ffs(__ballot_sync(kFullMask, upto > target)) - 1;
            int run_id = R * lane;
            u64 before = upto - own;
#pragma unroll
            for (int i = 0; i < R - 1; ++i)
                if (before + part[i] <= target && run_id == R * lane + i) {
                    before += part[i];
                    ++run_id;
                }
            run_id = __shfl_sync(kFullMask, run_id, src);
            before = __shfl_sync(kFullMask, before, src);
            if (run_id / kWarps == rank) {
                // its columns again
                if constexpr (S > 1) {
                    // few rows: a piece per warp, then that piece's, until a warp can
                    // walk the rest, column by column, the same few instructions
                    // throughout (their fetch is what a row of its own waits for:
                    // 1 x 128256, top-p, 44 us with the blocks' code below, 38 so)
                    int64_t from = max(int64_t(0), blocks.col(run_id * per_warp));
                    int64_t to = min(int64_t(cols), blocks.col((run_id + 1) * per_warp));
                    for (;;) {
                        const int64_t per = (to - from + kThreads - 1) / kThreads * 32;
                        const int64_t end = min(to, from + (warp + 1) * per);
                        u64 mine = 0;
                        for (int64_t c = from + warp * per + lane; c < end; c += 128) {
                            float v[4];  // four loads at a time
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                v[j] = c + 32 * j < end ? widen(x[row * cols + c + 32 * j]) : -INFINITY;
#pragma unroll 1
                            for (int j = 0; j < 4; ++j) {
                                mine += kept.column(v[0], c + 32 * j);
                                v[0] = v[1], v[1] = v[2], v[2] = v[3];
                            }
                        }
                        mine = warp_sum64(mine);
                        __syncthreads();  // the last round's have been read
                        if (lane == 0) sh.piece[warp] = mine;
                        __syncthreads();
                        int p = 0;  // the last one takes what is left
                        for (; p < kWarps - 1 && before + sh.piece[p] <= target; ++p) before += sh.piece[p];
                        from += p * per;
                        to = min(to, from + per);
                        if (per <= 128) break;
                    }
                    if (warp == 0) {
                        for (int64_t c0 = from; c0 < to; c0 += 32) {
                            const int64_t c = c0 + lane;
                            const float v = c < to ? widen(x[row * cols + c]) : -INFINITY;
                            const u64 a = kept.column(v, c);
                            const u64 upto = before + warp_prefix64(a, lane);
                            const uint32_t found = __ballot_sync(kFullMask, a > 0 && upto > target);
                            if (found) {
                                if (lane == __ffs(found) - 1) write(c, v, total);
                                break;
                            }
                            before = __shfl_sync(kFullMask, upto, 31);
                        }
                    }
                } else {
                    // many rows: a piece per warp, block by block (256 x 128256, one
                    // temperature: 91 us, column by column 97)
                    const int64_t from = run_id * per_warp;
                    const int64_t to = min(blocks.count, from + per_warp);
                    const int64_t per_piece = (per_warp / 32 + kWarps - 1) / kWarps * 32;
                    const int64_t plo = min(to, from + warp * per_piece), phi = min(to, plo + per_piece);
                    u64 piece = 0;
                    for (int64_t b = plo + lane; b < phi; b += 32) piece += kept.block(b);
                    piece = warp_sum64(piece);
                    if (lane == 0) sh.piece[warp] = piece;
                    __syncthreads();
                    for (int i = 0; i < warp; ++i) before += sh.piece[i];
                    if (before <= target && target < before + piece) {
                        for (int64_t b0 = plo; b0 < phi; b0 += 32) {
                            const u64 a = b0 + lane < phi ? kept.block(b0 + lane) : 0;
                            const u64 end = before + warp_prefix64(a, lane);
                            const uint32_t hit = __ballot_sync(kFullMask, end > target);
                            if (hit) {
                                // the block that holds the border: a lane per column
                                const int at = __ffs(hit) - 1;
                                const u64 start = __shfl_sync(kFullMask, end - a, at);
                                const int64_t c = blocks.col(b0 + at) + lane;
                                const bool in = lane < EPV && c >= 0 && c < cols;
                                const float v = in ? widen(x[row * cols + c]) : -INFINITY;
                                const u64 a_c = in ? kept.column(v, c) : 0;
                                const u64 upto_c = start + warp_prefix64(a_c, lane);
                                uint32_t found = __ballot_sync(kFullMask, a_c > 0 && upto_c > target);
                                if (lane == __ffs(found) - 1) write(c, v, total);
                                break;
                            }
                            before = __shfl_sync(kFullMask, end, 31);
                        }
                    }
                }
            }
        }
        row_sync<S>();  // the next row's values may be written; peers may leave
    }
}

}  // namespace sample
}  // namespace os
