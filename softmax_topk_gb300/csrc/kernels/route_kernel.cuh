// route_kernel.cuh -- routing of tokens to experts and its gradient, one warp
// per token.
//
// A row of E logits x gives scores s = softmax(x) or s_e = 1 / (1 + e^-x_e).
// The choice is made on c_e = s_e + bias_e (bias only steers the choice): with
// groups, the E experts are `groups` runs of equal length, a group is worth the
// sum of its `group_top` largest c, and only experts of the topk_groups best
// groups take part; then the K largest c, ties to the lower expert.  The
// weights are s of the chosen experts, divided by their sum when renormalised,
// times a scale.
//
// What bounds it: E logits are read and K pairs written per token, a few
// instructions per logit, so memory for large batches and one launch for small
// ones.  A token's row lives in the registers of one warp: lane l holds a run
// of consecutive experts, runs in lane order inside a group and groups in lane
// order, so the lowest expert among ties is the lowest lane's lowest element
// and a maximum over the warp is one redux instruction.  65536 rows, inputs past
// L2: 64 experts, K = 6, softmax 24 us, 128 experts, K = 8, 31 us; 256 experts,
// sigmoid, bias and groups 68 us by the kernel for large batches below (64
// instructions per logit, the ALU pipe 56 % busy; 10.5 us is what the bytes take).
// The gradient of the last: 21 us for 73 MB.
//
// Exact choices.  Without a bias s rises with x, so logits are compared and
// the choice is exact.  With a bias (and for sums of two scores) c is computed
// in fp32 with bounds (score_bounds), and the addition of the bias rounds once.
// Three steps, each for the tokens that the one before could not settle: choices
// by 32-bit keys, a value with its low bits replaced by its place; by full fp32
// values of exact functions (choose_exact); and in 64 bits (choose_wide).  Values
// of equal logit and bias need no more digits.  The weights themselves are of
// fp32 functions (the denominator's exponentials the SFU's), 6e-8 relative from
// the true ones as measured: a rounding or two of the result's.
#pragma once

#include <cuda_bf16.h>

#include <climits>
#include <cstdint>

#include "ops.cuh"

namespace os {
namespace route {

constexpr int kWarps = 4;      // warps per CTA
constexpr int kMaxExperts = 1024;

struct Shape {
    int experts, K, groups, topk_groups, group_top;
    int lanes, lanes_log2;  // lanes per group (a power of two)
    int per_lane;  // experts per lane
    int index_mask;  // experts up to a power of two, less one
    int slots;       // K up to a power of two: lanes per token after the choice
    int tokens;      // rows that a warp takes at a time, at most 32 / slots
    int sigmoid, renorm;
    float scale;
};

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }

// Order-preserving 32-bit key of a float (-0 must be +0); 0 is below every key.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kFullMask, v); }
__device__ __forceinline__ uint32_t warp_min(uint32_t v) { return __reduce_min_sync(kFullMask, v); }
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}

__device__ __forceinline__ float rcp_sfu(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float sigmoid(float x) {
    const float e = exp1(-fabsf(x));
    return __fdiv_rn(x < 0.f ? e : 1.f, 1.f + e);
}

// Sum of up to 1024 exponentials in [0, 1], of any order and split: each is a
// multiple of 2^-21 and a rest, the rest rounded to a multiple of 2^-42, and both
// are added as integers.  So the softmax's denominator has the same bits whichever
// kernel formed it (a token's weights do not depend on its batch), and its error
// is 2^-33 at most before the one rounding to fp32, where fp32 additions one after
// the other each lose up to 2^-24 of the sum.  The two parts come out of additions
// whose last bit is the unit wanted, two at a time, and carry the constants added
// along until the end of a run.
struct UnitSum {
    static constexpr float kHi = 4.f, kLo = 0x1.8p-19f;  // last bits 2^-21 and 2^-42
    uint32_t hi = 0, lo = 0;
    template <int N>
    __device__ __forceinline__ void add(const float (&e)[N]) {
        uint32_t h = 0, l = 0;
        constexpr int M = (N + 1) & ~1;
#pragma unroll
        for (int i = 0; i < M; i += 2) {
            // (a NaN counts for nothing)
            const float2 v = make_float2(fmaxf(e[i], 0.f), i + 1 < N ? fmaxf(e[i + 1], 0.f) : 0.f);
            const float2 t = add2(v, splat2(kHi));
            const float2 rest = fma2(add2(t, splat2(-kHi)), splat2(-1.f), v);  // exact
            const float2 r = add2(rest, splat2(kLo));
            h += __float_as_uint(t.x) + __float_as_uint(t.y);
            l += __float_as_uint(r.x) + __float_as_uint(r.y);
        }
        hi += h - uint32_t(M) * 0x40800000u;  // kHi
        lo += l - uint32_t(M) * 0x36400000u;  // kLo
    }
    // Over the warp's lanes.
    __device__ __forceinline__ void warp() {
        hi = __reduce_add_sync(kFullMask, hi);
        lo = __reduce_add_sync(kFullMask, lo);
    }
    // Over the four threads of a row (lanes that differ in their last two bits).
    __device__ __forceinline__ void four() {
#pragma unroll
        for (int o = 1; o <= 2; o *= 2) {
            hi += __shfl_xor_sync(kFullMask, hi, o);
            lo += __shfl_xor_sync(kFullMask, lo, o);
        }
    }
    __device__ __forceinline__ float value() const {
        return __ll2float_rn((static_cast<long long>(hi) << 21) + int(lo)) * 0x1p-42f;
    }
};

// This lane's run of a row: N consecutive values from p, `count` of them real
// (the rest -inf).  VEC: count is N or (a lane without experts) 0, and p
// aligned to min(16, N * sizeof(T)).
template <typename T, int N, bool VEC>
__device__ __forceinline__ void load_run(const T* p, int count, float (&v)[N]) {
    if constexpr (VEC) {
        if (count == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = -INFINITY;
            return;
        }
        constexpr int bytes = N * int(sizeof(T));
        uint32_t w[(bytes + 3) / 4];
        if constexpr (bytes >= 16) {
#pragma unroll
            for (int i = 0; i < bytes / 16; ++i)
                *reinterpret_cast<uint4*>(w + 4 * i) = __ldcs(reinterpret_cast<const uint4*>(p) + i);
        } else if constexpr (bytes == 8) {
            *reinterpret_cast<uint2*>(w) = __ldcs(reinterpret_cast<const uint2*>(p));
        } else if constexpr (bytes == 4) {
            w[0] = __ldcs(reinterpret_cast<const uint32_t*>(p));
        } else {
            w[0] = *reinterpret_cast<const uint16_t*>(p);
        }
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const float2 f = unpack_bf16x2(w[i / 2]);
                v[i] = f.x;
                if (i + 1 < N) v[i + 1] = f.y;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = i < count ? widen(p[i]) : -INFINITY;
    }
}

// A lane's place: its group, its experts base .. base + count - 1.
struct Place {
    int group, base, count;
    __device__ __forceinline__ explicit Place(const Shape& sh) {
        const int lane = threadIdx.x & 31, gsize = sh.experts / sh.groups;
        group = lane >> sh.lanes_log2;
        const int first = (lane & (sh.lanes - 1)) * sh.per_lane;  // within the group
        base = group * gsize + first;
        count = group < sh.groups ? max(0, min(sh.per_lane, gsize - first)) : 0;
    }
};

// Largest two values over the lanes of a group.
__device__ __forceinline__ void group_top2(const Shape& sh, float& a, float& b) {
    for (int o = sh.lanes / 2; o > 0; o >>= 1) {
        const float oa = __shfl_xor_sync(kFullMask, a, o), ob = __shfl_xor_sync(kFullMask, b, o);
        b = fmaxf(fminf(a, oa), fmaxf(b, ob));
        a = fmaxf(a, oa);
    }
}

// Twice what a score may be off by, so what the difference of two may be: with the
// SFU's functions, or in choose_exact with exp1 (`fine`).  In units of 2^-24:
//   softmax: e^z, z = x - m <= 0, is off by 2 |z| + 4 of itself (z rounded, its
//     product with log2 e rounded, ex2 to 2^-22), fine |z| + 2 (exp1 to one ulp).
//     The denominator's terms are off by that, weighted by their size: the mean of
//     |z| under the weights e^z is at most 4.5 (N equal terms beside one of z = 0
//     have z - 1 = N e^-z where it is largest: 4.45 for N = 1023), so 13, fine 6.5,
//     and its sum (UnitSum), its reciprocal and the product round once each.
//     Together e^-|z| (20 + 2 |z|), fine e^-|z| (11.5 + |z|), of s_max = 1 / d:
//     at most 20 and 11.5 (at z = 0), 21 and 12 are taken.
//   sigmoid: 1 / (1 + e^-x) is off by s (1 - s) (1.3 |x| + 4) + 3 s < 4, fine < 3
//     (a quotient exact to its rounding): 16 and 4 are taken.
__device__ __forceinline__ float score_bounds(const Shape& sh, float inv_d, bool fine) {
    if (sh.sigmoid) return fine ? 0x1p-21f : 0x1p-19f;
    return inv_d * (fine ? 0x1.8p-20f : 0x1.5p-19f);
}

// What a group's value may be off by, the sum a + b of two choice values (or a
// alone, b = 0): their scores' bounds, `err` for two, and the roundings of a, b
// and the sum, each |a| + |b| of 2^-24 however small the sum is (biases of
// opposite sign), and as much again for taking this bound off.
__device__ __forceinline__ float value_bound(float err, float a, float b) {
    return err + (fabsf(a) + fabsf(b)) * 0x1p-22f;
}

// The border between the groups that take part and the others: the least that
// one of the former can be worth and the most that one of the latter can.
struct Border {
    float low, high;
    bool near;  // they overlap
};

// Whether this lane's group takes part, of the given value, which is off by less
// than `bound` (`exact`: not at all).
__device__ __forceinline__ bool group_keep(const Shape& sh, int group, float value, float bound,
                                           bool exact, Border& border) {
    // round by round the best group that is left, ties to the lowest lane
    uint32_t left = group < sh.groups ? order_key(value + 0.f) : 0u;
    bool keep = false;
    for (int r = 0; r < sh.topk_groups; ++r) {
        const uint32_t top = warp_max(left);
        const int first = __ffs(__ballot_sync(kFullMask, left == top)) - 1;
        if (group == first >> sh.lanes_log2) {
            keep = true;
            left = 0u;
        }
    }
    border.near = false;
    if (!exact) {
        const bool out = left != 0u && value != -INFINITY;  // a group of nothing is last for certain
        const uint32_t low = warp_min(keep ? order_key(value - bound + 0.f) : 0xffffffffu);
        const uint32_t high = warp_max(out ? order_key(value + bound + 0.f) : 0u);
        border.low = key_value(low);
        border.high = key_value(high);
        border.near = high != 0u && !(border.low > border.high);
    }
    return keep;
}

// The same run written.
template <typename T, int N, bool VEC>
__device__ __forceinline__ void store_run(T* p, int count, const float (&v)[N]) {
    if constexpr (VEC) {
        if (count == 0) return;
        constexpr int bytes = N * int(sizeof(T));
        uint32_t w[(bytes + 3) / 4];
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = __float_as_uint(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < N; i += 2) w[i / 2] = pack_bf16x2(v[i], i + 1 < N ? v[i + 1] : 0.f);
        }
        if constexpr (bytes >= 16) {
#pragma unroll
            for (int i = 0; i < bytes / 16; ++i)
                reinterpret_cast<uint4*>(p)[i] =
                    make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else if constexpr (bytes == 8) {
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        } else if constexpr (bytes == 4) {
            *reinterpret_cast<uint32_t*>(p) = w[0];
        } else {
            *reinterpret_cast<uint16_t*>(p) = uint16_t(w[0]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < count) {
                if constexpr (sizeof(T) == 4) p[i] = v[i];
                else p[i] = __float2bfloat16_rn(v[i]);
            }
    }
}

// 64-bit order key of a double, and back.
__device__ __forceinline__ long long wide_key(double v) {
    const long long b = __double_as_longlong(v + 0.0);
    return b ^ ((b >> 63) & 0x7fffffffffffffffll);
}
__device__ __forceinline__ double wide_value(long long k) {
    return __longlong_as_double(k ^ ((k >> 63) & 0x7fffffffffffffffll));
}
constexpr long long kNoneWide = LLONG_MIN;
// Largest key over the warp: the high halves, then the low ones among equals.
__device__ __forceinline__ long long warp_max_wide(long long v) {
    const int hi = __reduce_max_sync(kFullMask, int(v >> 32));
    const uint32_t lo = __reduce_max_sync(kFullMask, int(v >> 32) == hi ? uint32_t(v) : 0u);
    return (static_cast<long long>(hi) << 32) | lo;
}

// The choice with c in 64 bits, one run per lane as in the kernel.  64-bit
// exponentials are slow (two lanes a clock per SM), so only the values that
// can matter are formed so: all of them where the choice of groups was too
// near (`all`), else those of at least `from`; the others are far from every
// border, and their fp32 values (c32) keep them in their places.
template <typename T, int N>
__device__ __noinline__ int choose_wide(const T* xrow, const float* bias, const Shape sh, float mf,
                                        const float* c32, float from, bool all) {
    const int lane = threadIdx.x & 31, E = sh.experts;
    const Place at_(sh);
    const int base = at_.base, count = at_.count;
    const bool by_score = bias != nullptr;
    const bool pair_sum = sh.groups > 1 && sh.group_top == 2;
    double d = 1.0;
    if (!sh.sigmoid && by_score) {  // without a bias it is a common factor
        d = 0.0;
        for (int i = 0; i < count; ++i) {
            const float x = widen(xrow[base + i]);
            if (x > -INFINITY) d += exp(double(x) - double(mf));
        }
        for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(kFullMask, d, o);
    }
    long long g[N];  // c, or for groups without a bias s
    for (int i = 0; i < N; ++i) {
        g[i] = kNoneWide;
        if (i >= count) continue;
        const float x = widen(xrow[base + i]);
        double v = -INFINITY;
        if (x > -INFINITY) {
            if (all || c32[i] >= from) {
                v = sh.sigmoid ? 1.0 / (1.0 + exp(-double(x))) : exp(double(x) - double(mf)) / d;
                if (by_score) v += double(bias[base + i]);
            } else {
                v = c32[i];
            }
        }
        g[i] = wide_key(v);
    }
    bool keep = true;
    if (sh.groups > 1) {
        long long a = kNoneWide, b = kNoneWide;
        for (int i = 0; i < N; ++i) {
            const long long lesser = min(a, g[i]);
            a = max(a, g[i]);
            b = max(b, lesser);
        }
        for (int o = sh.lanes / 2; o > 0; o >>= 1) {
            const long long oa = __shfl_xor_sync(kFullMask, a, o);
            const long long ob = __shfl_xor_sync(kFullMask, b, o);
            b = max(min(a, oa), max(b, ob));
            a = max(a, oa);
        }
        long long left = kNoneWide;
        if (at_.group < sh.groups) left = pair_sum ? wide_key(wide_value(a) + wide_value(b)) : a;
        keep = false;
        for (int r = 0; r < sh.topk_groups; ++r) {
            const long long top = warp_max_wide(left);
            const int first = __ffs(__ballot_sync(kFullMask, left == top)) - 1;
            if (at_.group == first >> sh.lanes_log2) {
                keep = true;
                left = kNoneWide;
            }
        }
    }
    for (int i = 0; i < N; ++i) {
        if (i < count && !by_score) g[i] = wide_key(widen(xrow[base + i]));  // s rises with x
        if (!keep) g[i] = kNoneWide;
    }
    int mine = 0;
    for (int k = 0; k < sh.K; ++k) {
        long long best = kNoneWide;
        int at = 0;
        for (int i = 0; i < N; ++i)
            if (g[i] > best) {
                best = g[i];
                at = i;
            }
        const long long top = warp_max_wide(best);
        const int src = __ffs(__ballot_sync(kFullMask, best == top)) - 1;
        const int e = min(__shfl_sync(kFullMask, base + at, src), E - 1);
        if (lane == k) mine = e;
        if (lane == src) g[at] = kNoneWide;
    }
    return mine;
}

// The choice with c in fp32 and experts beside it; every lane returns the
// expert of slot `lane` (lane < K).
template <typename T, int N>
__device__ __noinline__ int choose_exact(const T* xrow, const float* bias, const Shape sh) {
    const int lane = threadIdx.x & 31, E = sh.experts;
    const Place at_(sh);
    const int base = at_.base, count = at_.count;
    const bool by_score = bias != nullptr;
    const bool pair_sum = sh.groups > 1 && sh.group_top == 2;
    float v[N];
    load_run<T, N, false>(xrow + base, count, v);
    float m = 0.f, inv_d = 1.f;
    if (!sh.sigmoid) {
        m = v[0];
#pragma unroll
        for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
        m = key_value(warp_max(order_key(m + 0.f)));
        const float ref = m == -INFINITY ? 0.f : m;
        float e[N];
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = v[i] == -INFINITY ? 0.f : exp1(v[i] - ref);
        UnitSum sum;
        sum.add(e);
        sum.warp();
        const float d = sum.value();
        inv_d = d > 0.f ? __frcp_rn(d) : 0.f;
    }
    auto score = [&](float xv) {
        if (xv == -INFINITY) return 0.f;
        return sh.sigmoid ? sigmoid(xv) : exp1(xv - m) * inv_d;
    };
    const float err = score_bounds(sh, inv_d, true);

    // the value that is compared, as an order key; 0 = takes no part
    uint32_t key[N];
    float c32[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float c = v[i];
        if (by_score && v[i] != -INFINITY) c = score(v[i]) + bias[i < count ? base + i : 0];
        c32[i] = c;
        key[i] = i < count ? order_key(c + 0.f) : 0u;
    }
    bool groups_near = false, near = false;
    if (sh.groups > 1) {
        // the two best with their places, to tell equal sums from near ones
        float a = -INFINITY, b = -INFINITY, ax = 0.f, bx = 0.f, ab = 0.f, bb = 0.f;
        auto take = [&](float c, float x, float bi) {
            if (c > a) {
                b = a, bx = ax, bb = ab;
                a = c, ax = x, ab = bi;
            } else if (c > b) {
                b = c, bx = x, bb = bi;
            }
        };
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < count && v[i] != -INFINITY)
                take(pair_sum && !by_score ? score(v[i]) : c32[i], v[i],
                     by_score ? bias[base + i] : 0.f);
        for (int o = sh.lanes / 2; o > 0; o >>= 1) {
            const float oa = __shfl_xor_sync(kFullMask, a, o), ob = __shfl_xor_sync(kFullMask, b, o);
            const float oax = __shfl_xor_sync(kFullMask, ax, o), obx = __shfl_xor_sync(kFullMask, bx, o);
            const float oab = __shfl_xor_sync(kFullMask, ab, o), obb = __shfl_xor_sync(kFullMask, bb, o);
            take(oa, oax, oab);
            take(ob, obx, obb);
        }
        if (!pair_sum) b = 0.f, bx = 0.f, bb = 0.f;
        const float value = a + b, bound = value_bound(err, a, b);
        Border border;
        const bool keep = group_keep(sh, at_.group, value, bound, !(by_score || pair_sum), border);
        if (border.near) {
            // groups that may stand on either side of the border must all be
            // made of the same logits and biases: then the lower ones are right
            const bool in = at_.group < sh.groups &&
                            (keep ? !(value - bound > border.high)
                                  : value != -INFINITY && !(value + bound < border.low));
            const int src = max(__ffs(__ballot_sync(kFullMask, in)) - 1, 0);
            auto same = [&](float t) { return t == __shfl_sync(kFullMask, t, src); };
            const bool equal = same(a) & same(ax) & same(ab) & same(b) & same(bx) & same(bb);
            groups_near = __any_sync(kFullMask, in && !equal);
        }
        if (!keep) {
#pragma unroll
            for (int i = 0; i < N; ++i) key[i] = 0u;
        }
    }

    // K rounds: this lane's best, then the warp's
    uint32_t best = 0u;
    int at = 0;
    auto local_best = [&]() {
        best = 0u;
        at = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
    };
    local_best();
    int mine = 0;
    float prev_c = 0.f, prev_x = 0.f, prev_b = 0.f, slack = 0.f;
    for (int k = 0; k < sh.K; ++k) {
        const uint32_t top = warp_max(best);
        const int src = __ffs(__ballot_sync(kFullMask, best == top)) - 1;
        const int e = min(__shfl_sync(kFullMask, base + at, src), E - 1);
        if (lane == k) mine = e;
        if (by_score) {
            const float c = key_value(top), be = bias[e], xv = widen(xrow[e]);
            if (k > 0 && c != -INFINITY && !(prev_c - c > slack) && !(xv == prev_x && be == prev_b))
                near = true;
            prev_c = c;
            prev_x = xv;
            prev_b = be;
            slack = err + fabsf(c) * 0x1p-22f;
        }
        if (lane == src) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i == at) key[i] = 0u;
            local_best();
        }
    }
    if (by_score && prev_c != -INFINITY && best != 0u && !(key_value(best) < prev_c - slack)) {
        // experts left out that are too near the last one taken
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (key[i] != 0u && !(key_value(key[i]) < prev_c - slack) &&
                !(v[i] == prev_x && bias[base + i] == prev_b))
                near = true;
    }
    near = __any_sync(kFullMask, near);
    if (groups_near || near)
        mine = choose_wide<T, N>(xrow, bias, sh, m, c32, prev_c - 2.f * slack, groups_near);
    return mine;
}

// Descending order of N (a power of two, at most 8) values by a network.
template <int N>
__device__ __forceinline__ void sort_run(int (&k)[N]) {
#pragma unroll
    for (int width = 2; width <= N; width *= 2)
#pragma unroll
        for (int step = width / 2; step > 0; step /= 2)
#pragma unroll
            for (int i = 0; i < N; ++i)
                if ((i & step) == 0) {
                    const int a = k[i], b = k[i + step];
                    const bool down = (i & width) == 0;
                    k[i] = down ? max(a, b) : min(a, b);
                    k[i + step] = down ? min(a, b) : max(a, b);
                }
}

// Signed order key of a float, and back.
__device__ __forceinline__ int signed_key(float v) {
    const int b = __float_as_int(v);
    return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float signed_value(int k) {
    return __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
}
constexpr int kNone = INT_MIN;             // takes no part; below every key
constexpr int kMissing = int(0x80800000u);  // keys of -inf are below this

// Sum and maximum over the `width` lanes (a power of two) of this lane's slots.
__device__ __forceinline__ float slot_sum(float v, int width) {
    for (int o = width / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}
__device__ __forceinline__ float slot_max(float v, int width) {
    for (int o = width / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, o));
    return v;
}

// N: experts per lane, rounded up to a power of two.
//
// A warp chooses for `tokens` rows one after the other and then does what is
// left, slot by slot, for all of them at once: lane t * slots + k has slot k of
// token t (slots: K up to a power of two).
template <typename T, int N, bool VEC>
__global__ void __launch_bounds__(kWarps * 32, N <= 8 ? 6 : 3)
route_kernel(const T* __restrict__ x, const float* __restrict__ bias, float* __restrict__ weights,
             int* __restrict__ idx, int64_t rows, const Shape sh) {
    const int lane = threadIdx.x & 31;
    const int E = sh.experts, K = sh.K;
    const Place at(sh);
    const int base = at.base, count = at.count;
    const bool by_score = bias != nullptr;  // else logits give the order
    // the softmax's maximum and sum are needed for its scores themselves
    const bool pair_sum = sh.groups > 1 && sh.group_top == 2;
    const bool need_scores = by_score || pair_sum;
    const bool need_sum = !sh.sigmoid && (need_scores || !sh.renorm);
    constexpr int low_bits = N - 1;  // of a key: the place in the run, counted down
    __shared__ int chosen_at[kWarps][32];
    int* const chosen = chosen_at[threadIdx.x >> 5];  // experts, slot by slot
    const int my_token = lane / sh.slots, my_slot = lane % sh.slots;
    float be[N];
#pragma unroll
    for (int i = 0; i < N; ++i) be[i] = by_score && i < count ? bias[base + i] : 0.f;

    const int64_t step = int64_t(gridDim.x) * kWarps * sh.tokens;
    for (int64_t row0 = (int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * sh.tokens; row0 < rows;
         row0 += step) {
        const int tokens = int(min(int64_t(sh.tokens), rows - row0));
        int mine = kNone, after = kNone;     // this lane's slot and the next best
        float m_slot = 0.f, inv_slot = 1.f;  // its row's maximum and 1 / sum
        uint32_t unsure = 0;                 // one bit per token
        float v[N];
        load_run<T, N, VEC>(x + row0 * E + base, count, v);
        for (int t = 0; t < tokens; ++t) {
            float ahead[N];  // the next token's logits
            if (t + 1 < tokens) load_run<T, N, VEC>(x + (row0 + t + 1) * E + base, count, ahead);
            float m = 0.f, inv_d = 1.f;
            if (!sh.sigmoid) {
                m = v[0];
#pragma unroll
                for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
                m = key_value(warp_max(order_key(m + 0.f)));
            }
            float s[N];  // scores, where they are compared
            if (need_sum) {
                const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
                for (int i = 0; i < N; i += 2) {
                    const float2 e = exp_pair<false>(
                        make_float2(v[i] - ref, i + 1 < N ? v[i + 1] - ref : -INFINITY));
                    s[i] = e.x;
                    if (i + 1 < N) s[i + 1] = e.y;
                }
                UnitSum sum;
                sum.add(s);
                sum.warp();
                const float d = sum.value();
                inv_d = d > 0.f ? __frcp_rn(d) : 0.f;
#pragma unroll
                for (int i = 0; i < N; ++i) s[i] *= inv_d;
            } else if (need_scores) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    s[i] = rcp_sfu(1.f + ex2_sfu(-expc::kLog2e * v[i]));
            }
            if (my_token == t) {
                m_slot = m;
                inv_slot = inv_d;
            }
            float c[N];
#pragma unroll
            for (int i = 0; i < N; ++i)
                c[i] = by_score && v[i] != -INFINITY ? s[i] + be[i] : v[i];
            bool keep = true;
            if (sh.groups > 1) {
                float a = -INFINITY, b = -INFINITY;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    if (i < count) {
                        const float g = pair_sum && !by_score && v[i] != -INFINITY ? s[i] : c[i];
                        b = fmaxf(b, fminf(a, g));
                        a = fmaxf(a, g);
                    }
                }
                group_top2(sh, a, b);
                if (!pair_sum) b = 0.f;
                Border border;
                keep = group_keep(sh, at.group, a + b,
                                  value_bound(score_bounds(sh, inv_d, false), a, b),
                                  !need_scores, border);
                if (border.near) unsure |= 1u << t;
            }
            int key[N];
#pragma unroll
            for (int i = 0; i < N; ++i)
                key[i] = keep && i < count
                             ? ((signed_key(c[i] + 0.f) & ~low_bits) | (low_bits - i))
                             : kNone;

            // K rounds, and one for the best that is left out
            if constexpr (N <= 8) sort_run<N>(key);
            auto lane_best = [&]() {
                int best = key[0];
                if constexpr (N > 8) {
#pragma unroll
                    for (int i = 1; i < N; ++i) best = max(best, key[i]);
                }
                return best;
            };
            const int slot_here = my_token == t ? my_slot : -1;
            for (int k = 0; k < K; ++k) {
                const int best = lane_best();
                const int top = __reduce_max_sync(kFullMask, best & ~low_bits);
                if (slot_here == k) mine = top;
                // the lowest lane among equals has the lowest expert
                const int src = __ffs(__ballot_sync(kFullMask, (best & ~low_bits) == top)) - 1;
                const bool taken = lane == src;
                if (taken) chosen[t * sh.slots + k] = base + low_bits - (best & low_bits);
                if constexpr (N <= 8) {
#pragma unroll
                    for (int i = 0; i + 1 < N; ++i) key[i] = taken ? key[i + 1] : key[i];
                    key[N - 1] = taken ? kNone : key[N - 1];
                } else if (taken) {
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        if (key[i] == best) key[i] = kNone;
                }
            }
            const int next = __reduce_max_sync(kFullMask, lane_best() & ~low_bits);
            if (slot_here == K - 1) after = next;
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = ahead[i];
        }

        // ---- slot by slot: is the order certain?
        const bool real = my_token < tokens && my_slot < K;
        const T* xrow = x + (row0 + my_token) * E;
        __syncwarp();
        int e = real ? min(chosen[lane], E - 1) : 0;
        __syncwarp();
        float xm = real ? widen(xrow[e]) : -INFINITY;
        const float err = score_bounds(sh, inv_slot, false);
        if (by_score || sizeof(T) == 4) {
            const int below = __shfl_down_sync(kFullMask, mine, 1);
            if (my_slot != K - 1) after = below;
            bool near;
            if (by_score) {
                const float va = signed_value(mine), vb = signed_value(after);
                near = !(va - vb > err + (fabsf(va) + fabsf(vb)) * float(low_bits + 2) * 0x1p-23f);
            } else {
                near = mine == after;
            }
            near = near && real && after >= kMissing;
            if (__any_sync(kFullMask, near)) {
                // equal logits of equal bias stand in the order of their experts
                const float b = by_score ? bias[e] : 0.f;
                const float xa = __shfl_down_sync(kFullMask, xm, 1);
                const float ba = __shfl_down_sync(kFullMask, b, 1);
                if (near && (my_slot == K - 1 || xa != xm || ba != b)) unsure |= 1u << my_token;
            }
        }
        unsure = __reduce_or_sync(kFullMask, unsure);
        for (; unsure; unsure &= unsure - 1) {
            const int t = __ffs(unsure) - 1;
            const int chosen = choose_exact<T, N>(x + (row0 + t) * E, bias, sh);
            const int here = __shfl_sync(kFullMask, chosen, my_slot);
            if (my_token == t) {
                e = here;
                xm = real ? widen(xrow[e]) : -INFINITY;
            }
        }

        // ---- weights
        const bool live = real && xm != -INFINITY;
        float w;
        if (!sh.renorm) {
            w = sh.sigmoid ? sigmoid(xm) : exp1(xm - m_slot) * inv_slot;
            if (!live) w = 0.f;
        } else {
            // relative to the largest chosen logit, so that no sum underflows
            float top = slot_max(live ? xm : -INFINITY, sh.slots);
            if (sh.sigmoid) top = fminf(top, 0.f);
            if (sh.sigmoid && xm > 0.f) {
                w = sigmoid(xm);
            } else {
                w = exp1(xm - top);
                if (sh.sigmoid) w = __fdiv_rn(w, 1.f + exp1(xm));
            }
            if (!live) w = 0.f;
            const float sum = slot_sum(w, sh.slots);
            w = sum > 0.f ? __fdiv_rn(w, sum) : 0.f;
        }
        if (real) {
            weights[(row0 + my_token) * K + my_slot] = w * sh.scale;
            idx[(row0 + my_token) * K + my_slot] = e;
        }
    }
}

// ------------------------------------------------------------------ large batches
// Four threads per token.  What crosses lanes in the kernel above (redux, votes,
// shuffles, four fifths of its instructions) mostly happens in a thread's
// registers here, 8 tokens to an instruction, at the price of the rows' stay in
// shared memory and of latency, so it takes large batches only (rule and times: route_dispatch.cuh).
//
// A warp copies 8 rows in 16-byte chunks, placed so that the four threads of a
// row, reading one chunk each of neighbouring places or of different groups,
// and the next row's four hit different banks.  Every thread keeps the best P
// (K up to a power of two, at least 4) of its chunks as a sorted list of keys in
// registers, the value with its low bits replaced by the expert; four new ones
// are sorted and merged into it at once, and the best key that fell out is
// kept too.  The four lists are merged over shuffles.  Then the listed experts'
// full values settle the order that the cut-off bits hide; where a value is
// too near the next, or a key that fell out may hide a better one, the token
// goes to choose_exact (the whole warp).
constexpr int kListWarps = 4;
constexpr int kListRows = 8;       // rows per warp
constexpr int kListExperts = 1024;
// Bytes of shared memory before the rows: the bias, with groups their values and
// bounds too.
__host__ __device__ constexpr int list_head(int experts, int groups) {
    return (experts + 4 * groups + (groups > 1 ? 2 * kListWarps * kListRows * groups : 0)) * 4;
}

// a >= b after it.
__device__ __forceinline__ void order(int& a, int& b) {
    const int t = max(a, b);
    b = min(a, b);
    a = t;
}
// A bitonic list into falling order.
template <int P>
__device__ __forceinline__ void order_bitonic(int (&list)[P]) {
#pragma unroll
    for (int step = P / 2; step > 0; step /= 2)
#pragma unroll
        for (int i = 0; i < P; ++i)
            if ((i & step) == 0) order(list[i], list[i + step]);
}
// The best two keys that have fallen out of a list.
struct Fallen {
    int first = kNone, second = kNone;
    __device__ __forceinline__ void take(int k) {
        second = max(second, min(first, k));
        first = max(first, k);
    }
};
// Merges four keys into the sorted list.
template <int P>
__device__ __forceinline__ void merge4(int (&list)[P], int (&k)[4], Fallen& out) {
    order(k[0], k[1]);
    order(k[2], k[3]);
    order(k[0], k[2]);
    order(k[1], k[3]);
    order(k[1], k[2]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int& tail = list[P - 1 - i];
        out.take(min(tail, k[i]));
        tail = max(tail, k[i]);
    }
    order_bitonic<P>(list);  // P - 4 falling, then 4 rising
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem_addr(dst)), "l"(src)
                 : "memory");
}

// Sum, maximum, minimum over the four threads of a row.
__device__ __forceinline__ float row_sum(float v) {
    v += __shfl_xor_sync(kFullMask, v, 2);
    return v + __shfl_xor_sync(kFullMask, v, 1);
}
__device__ __forceinline__ float row_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(kFullMask, v, 1));
    return fmaxf(v, __shfl_xor_sync(kFullMask, v, 2));
}

// A sigmoid's choice value in 64 bits.
static __device__ __noinline__ double wide_choice(float x, float bias) {
    return 1.0 / (1.0 + exp(-double(x))) + double(bias);
}

// P: list length; N: experts per lane in choose_exact.
template <typename T, int P, int N>
__global__ void __launch_bounds__(kListWarps * 32, P <= 8 ? 5 : 4)
route_list_kernel(const T* __restrict__ x, const float* __restrict__ bias,
                  float* __restrict__ weights, int* __restrict__ idx, int64_t rows, const Shape sh) {
    constexpr int EPV = 16 / int(sizeof(T));
    extern __shared__ __align__(16) unsigned char list_smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane & 3, my = lane >> 2;  // thread of the row, row of the tile
    const int E = sh.experts, K = sh.K, G = sh.groups, gsize = E / G;
    const int chunks = E / EPV, group_chunks = gsize / EPV;
    const bool by_score = bias != nullptr;
    const bool pair_sum = G > 1 && sh.group_top == 2;
    const bool need_scores = by_score || pair_sum;
    const bool need_sum = !sh.sigmoid && (need_scores || !sh.renorm);
    const int mask = sh.index_mask;
    // bias, its groups 4 floats apart so that threads in different groups meet
    // different banks; the groups' values of every row and what they may be off
    // by; the warps' tiles
    float* const b_sm = reinterpret_cast<float*>(list_smem);
    float* const value = b_sm + E + 4 * G + (warp * kListRows + my) * G;  // where G > 1
    float* const bound = value + kListWarps * kListRows * G;
    unsigned char* const tile = list_smem + list_head(E, G) + warp * kListRows * E * int(sizeof(T));
    for (int e = threadIdx.x; e < E; e += kListWarps * 32)
        b_sm[e + 4 * (e / gsize)] = by_score ? bias[e] : 0.f;
    __syncthreads();
    auto place = [&](int r, int c) {
        return (r * chunks + (c ^ (((c >> 3) ^ ((r & 1) << 2)) & 7))) * 16;
    };

    const int64_t tiles = (rows + kListRows - 1) / kListRows;
    for (int64_t t = int64_t(blockIdx.x) * kListWarps + warp; t < tiles;
         t += int64_t(gridDim.x) * kListWarps) {
        const int64_t row0 = t * kListRows;
        const int here = int(min(int64_t(kListRows), rows - row0));
        __syncwarp();  // the last tile has been read
        for (int r = 0; r < here; ++r)
            for (int c = lane; c < chunks; c += 32)
                cp_async16(tile + place(r, c), x + (row0 + r) * E + c * EPV);
        // the next tile on its way into L2 while this one is worked on
        const int64_t ahead = t + int64_t(gridDim.x) * kListWarps;
        if (ahead < tiles) {
            const unsigned char* p = reinterpret_cast<const unsigned char*>(x + ahead * kListRows * E);
            const int bytes = int(min(int64_t(kListRows), rows - ahead * kListRows)) * E * int(sizeof(T));
            for (int i = lane * 128; i < bytes; i += 32 * 128)
                asm volatile("prefetch.global.L2 [%0];" :: "l"(p + i));
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        // threads past the last row work on row 0 and write nothing
        const int r = my < here ? my : 0;
        auto load = [&](int c, float (&v)[EPV]) {
            const uint4 w = *reinterpret_cast<const uint4*>(tile + place(r, c));
            const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 4) {
                    v[i] = __uint_as_float(a[i]);
                } else {
                    const float2 f = unpack_bf16x2(a[i]);
                    v[2 * i] = f.x;
                    v[2 * i + 1] = f.y;
                }
            }
        };
        auto logit = [&](int e) {
            return widen(reinterpret_cast<const T*>(tile + place(r, e / EPV))[e % EPV]);
        };

        float m = 0.f, inv_d = 1.f;
        if (!sh.sigmoid) {
            m = -INFINITY;
            for (int c = sub; c < chunks; c += 4) {
                float v[EPV];
                load(c, v);
#pragma unroll
                for (int i = 0; i < EPV; ++i) m = fmaxf(m, v[i]);
            }
            m = row_max(m);
            if (need_sum) {
                const float ref = m == -INFINITY ? 0.f : m;
                UnitSum sum;
                for (int c = sub; c < chunks; c += 4) {
                    float v[EPV];
                    load(c, v);
#pragma unroll
                    for (int i = 0; i < EPV; i += 2) {
                        const float2 e = exp_pair<false>(make_float2(v[i] - ref, v[i + 1] - ref));
                        v[i] = e.x;
                        v[i + 1] = e.y;
                    }
                    sum.add(v);
                }
                sum.four();
                const float d = sum.value();
                inv_d = d > 0.f ? __frcp_rn(d) : 0.f;
            }
        }
        const float err = score_bounds(sh, inv_d, false);
        auto score = [&](float v) {  // the SFU's; 0 for -inf
            return sh.sigmoid ? rcp_sfu(1.f + ex2_sfu(-expc::kLog2e * v))
                              : exp_pair<false>(make_float2(v - m, v - m)).x * inv_d;
        };

        // ---- groups that take part, one bit each; thread `sub` values every
        // fourth group and ranks it
        uint32_t kept = 0xffffffffu;
        bool unsure = false;
        if (G > 1) {
            for (int g = sub; g < G; g += 4) {
                float a = -INFINITY, b = -INFINITY;
                const float* gb = b_sm + g * (gsize + 4);
                for (int c = 0; c < group_chunks; ++c, gb += EPV) {
                    float v[EPV];
                    load(g * group_chunks + c, v);
#pragma unroll
                    for (int i = 0; i < EPV; ++i) {
                        float y = v[i];
                        if (need_scores) {
                            y = score(v[i]) + gb[i];
                            if (v[i] == -INFINITY) y = -INFINITY;
                        }
                        b = fmaxf(b, fminf(a, y));
                        a = fmaxf(a, y);
                    }
                }
                if (!pair_sum) b = 0.f;
                value[g] = a + b;
                bound[g] = value_bound(err, a, b);
            }
            __syncwarp();
            kept = 0;
            float low = INFINITY, high = -INFINITY;
            for (int g = sub; g < G; g += 4) {
                const float y = value[g];
                int rank = 0;
                for (int h = 0; h < G; ++h) {
                    const float o = value[h];
                    rank += o > y || (o == y && h < g);
                }
                if (rank < sh.topk_groups) {
                    kept |= 1u << g;
                    low = fminf(low, y - bound[g]);
                } else if (y != -INFINITY) {
                    high = fmaxf(high, y + bound[g]);
                }
            }
            kept |= __shfl_xor_sync(kFullMask, kept, 1);
            kept |= __shfl_xor_sync(kFullMask, kept, 2);
            low = -row_max(-low);
            high = row_max(high);
            // (fewer or more than topk_groups only where values are NaN)
            if (need_scores && high != -INFINITY && !(low > high)) unsure = true;
        }

        // ---- the P best of this thread's chunks: every fourth of those that
        // take part
        int list[P];
        Fallen out;
#pragma unroll
        for (int i = 0; i < P; ++i) list[i] = kNone;
        {
            uint32_t left = G > 1 ? kept : 1u;
            int c0 = sub;
            while (left) {
                while (left && c0 >= group_chunks) {
                    c0 -= group_chunks;
                    left &= left - 1;
                }
                if (!left) break;
                const int g = __ffs(left) - 1;
                float v[EPV];
                load(g * group_chunks + c0, v);
                const float* gb = b_sm + g * (gsize + 4) + c0 * EPV;
                const int first = mask - (g * gsize + c0 * EPV);
#pragma unroll
                for (int i = 0; i < EPV; i += 4) {
                    int k[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float y = v[i + j];
                        if (by_score) {
                            y = score(v[i + j]) + gb[i + j];
                            if (v[i + j] == -INFINITY) y = -INFINITY;
                        }
                        k[j] = (signed_key(y + 0.f) & ~mask) | (first - i - j);
                    }
                    merge4<P>(list, k, out);
                }
                c0 += 4;
            }
        }
        __syncwarp();
#pragma unroll
        for (int step = 1; step <= 2; step *= 2) {
            int other[P];
#pragma unroll
            for (int i = 0; i < P; ++i) other[i] = __shfl_xor_sync(kFullMask, list[i], step);
            const int first = __shfl_xor_sync(kFullMask, out.first, step);
            const int second = __shfl_xor_sync(kFullMask, out.second, step);
            out.take(first);
            out.take(second);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                out.take(min(list[i], other[P - 1 - i]));
                list[i] = max(list[i], other[P - 1 - i]);
            }
            order_bitonic<P>(list);
            // both threads of the pair saw the same keys fall, in another order
        }

        // ---- the listed experts' full values, and the best fallen one's, in
        // order
        constexpr int C = P + 1;
        float c[C];
        int e[C];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int k = i < P ? list[i < P ? i : 0] : out.first;
            e[i] = k == kNone ? E - 1 : mask - (k & mask);
            const float y = logit(e[i]);
            c[i] = k == kNone ? -INFINITY : y;
            if (by_score && c[i] != -INFINITY) c[i] = score(y) + b_sm[e[i] + 4 * (e[i] / gsize)];
        }
        auto swap_at = [&](int i) {
            const float tc = c[i];
            c[i] = c[i + 1];
            c[i + 1] = tc;
            const int te = e[i];
            e[i] = e[i + 1];
            e[i + 1] = te;
        };
        // neighbours whose cut-off bits hid their order change places
        const bool exact_keys = !by_score && sizeof(T) == 2;  // no bits were cut off
        bool wrong = false;
#pragma unroll
        for (int i = 0; i + 1 < C; ++i) wrong = wrong || c[i + 1] > c[i];
        if (__any_sync(kFullMask, wrong)) {
#pragma unroll
            for (int pass = 0; pass < 2; ++pass)
#pragma unroll
                for (int i = 0; i + 1 < C; ++i)
                    if (c[i + 1] > c[i]) swap_at(i);
            // (an expert more than two places down may have farther to go)
#pragma unroll
            for (int i = 0; i + 1 < C; ++i) unsure = unsure || c[i + 1] > c[i];
        }
        // values too near to their successors for this arithmetic
        bool near = false;
#pragma unroll
        for (int i = 0; i + 1 < C; ++i) {
            const float slack = by_score ? err + fabsf(c[i]) * 0x1p-22f : 0.f;
            near = near || (i < K && c[i + 1] != -INFINITY && !(c[i] - c[i + 1] > slack));
        }
        if (__any_sync(kFullMask, near && !exact_keys)) {
            // pairs in 64 bits: a sigmoid's needs nothing of the row (a
            // softmax's sum would); twice over for three in a row, and where
            // the second time still finds a pair to exchange there are more.
            // A run of near values that goes past slot K - 1 is ordered to its
            // end, for any of them may belong there
            auto wide = [&](int i) {
                return wide_choice(logit(e[i]), b_sm[e[i] + 4 * (e[i] / gsize)]);
            };
#pragma unroll 1
            for (int pass = 0; pass < 2; ++pass) {
                bool bad = false;
#pragma unroll
                for (int i = 0; i + 1 < C; ++i) {
                    const float slack = by_score ? err + fabsf(c[i]) * 0x1p-22f : 0.f;
                    bad = (i < K || bad) && c[i + 1] != -INFINITY && !exact_keys &&
                          !(c[i] - c[i + 1] > slack);
                    if (bad) {
                        // equal logits of equal bias stand in the order of
                        // their experts
                        const int p = e[i], n = e[i + 1];
                        const bool same = logit(p) == logit(n) &&
                                          b_sm[p + 4 * (p / gsize)] == b_sm[n + 4 * (n / gsize)];
                        bool change = same && n < p;
                        if (!same && by_score && sh.sigmoid) {
                            const double a = wide(i), b = wide(i + 1);
                            change = b > a || (b == a && n < p);
                        } else if (!same) {
                            unsure = true;
                        }
                        if (change) {
                            swap_at(i);
                            unsure = unsure || pass == 1;
                        }
                    }
                }
            }
        }
        // what the second fallen key, and those below it, can stand for
        if (!exact_keys && out.second >= kMissing) {
            const float rest = signed_value(out.second | mask);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float slack = by_score ? err + fabsf(c[i]) * 0x1p-22f : 0.f;
                if (i == K - 1 && !(c[i] - rest > slack)) unsure = true;
            }
        }
        for (uint32_t todo = __ballot_sync(kFullMask, unsure && my < here && sub == 0); todo;
             todo &= todo - 1) {
            const int src = __ffs(todo) - 1;
            const int chosen = choose_exact<T, N>(x + (row0 + (src >> 2)) * E, bias, sh);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int got = __shfl_sync(kFullMask, chosen, i);
                if (my == src >> 2 && i < K) e[i] = got;
            }
        }

        // ---- weights: thread `sub` has the slots sub, sub + 4, ...
        constexpr int Q = P / 4;
        float z[Q], w[Q], top = -INFINITY;
        int ez[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            ez[q] = sub == 0 ? e[4 * q] : sub == 1 ? e[4 * q + 1] : sub == 2 ? e[4 * q + 2] : e[4 * q + 3];
            z[q] = 4 * q + sub < K ? logit(ez[q]) : -INFINITY;
            top = fmaxf(top, z[q]);
        }
        top = row_max(top);
        if (sh.sigmoid) top = fminf(top, 0.f);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            if (!sh.renorm) {
                w[q] = sh.sigmoid ? sigmoid(z[q]) : exp1(z[q] - m) * inv_d;
            } else if (sh.sigmoid && z[q] > 0.f) {
                w[q] = sigmoid(z[q]);
            } else {
                w[q] = exp1(z[q] - top);
                if (sh.sigmoid) w[q] = __fdiv_rn(w[q], 1.f + exp1(z[q]));
            }
            if (z[q] == -INFINITY) w[q] = 0.f;
        }
        // added in the other kernel's order, so that renormalised weights do not
        // depend on the number of rows
        float part[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) part[q] = w[q];
#pragma unroll
        for (int step = Q / 2; step > 0; step /= 2)
#pragma unroll
            for (int q = 0; q < step; ++q) part[q] += part[q + step];
        const float sum = row_sum(part[0]);
        if (my < here) {
            const int64_t at = (row0 + my) * K;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                if (4 * q + sub < K) {
                    float y = w[q];
                    if (sh.renorm) y = sum > 0.f ? __fdiv_rn(y, sum) : 0.f;
                    weights[at + 4 * q + sub] = y * sh.scale;
                    idx[at + 4 * q + sub] = ez[q];
                }
            }
        }
    }
}

// Gradient of the weights with respect to the logits, for given experts.  With
// g_k = scale dw_k, s the scores, S = sum of the chosen scores, w = s / S:
//   sigmoid:              dx_e = sum over slots of e of g_k s (1 - s)
//   sigmoid, renormalised:       sum of w_k (g_k - D) (1 - s_k),  D = sum g w
//   softmax:              dx_e = s_e (sum over slots of e of g_k - D),  D = sum g_k s_k
//   softmax, renormalised: sum over slots of e of w_k (g_k - D),  D = sum g w
// Only the plain softmax gives every logit a gradient; the others are zero
// outside the chosen experts, whose logits alone are read.  One read of what
// is needed and one write of the dense row: memory bound.
//
// A warp takes `tokens` rows at a time, lane t * slots + k slot k of row t, as
// in the choice: what the slots add is worked out for all of them at once,
// the rows are written in whole vectors without it, and then each slot's lane
// writes its expert's value over the row's.  Slots that name one expert twice
// are summed in slot order by the first of them, which alone writes.
template <typename T, int N, bool VEC>
__global__ void __launch_bounds__(kWarps * 32)
route_bwd_kernel(const T* __restrict__ x, const int* __restrict__ idx,
                 const float* __restrict__ dweights, T* __restrict__ dx, int64_t rows,
                 const Shape sh) {
    const int lane = threadIdx.x & 31;
    const int E = sh.experts, K = sh.K;
    const int base = lane * sh.per_lane;
    const int count = max(0, min(sh.per_lane, E - base));
    const bool all = !sh.sigmoid && !sh.renorm;
    const int my_token = lane / sh.slots, my_slot = lane % sh.slots;
    const int64_t step = int64_t(gridDim.x) * kWarps * sh.tokens;
    for (int64_t row0 = (int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * sh.tokens; row0 < rows;
         row0 += step) {
        const int tokens = int(min(int64_t(sh.tokens), rows - row0));
        const int64_t my_row = row0 + my_token;
        // this slot's expert, logit and gradient; an expert outside the row
        // takes no part
        int e = -1;
        float xk = -INFINITY, g = 0.f;
        if (my_token < tokens && my_slot < K) {
            e = idx[my_row * K + my_slot];
            if (e < 0 || e >= E) e = -1;
            if (e >= 0) {
                xk = widen(x[my_row * E + e]);
                g = dweights[my_row * K + my_slot] * sh.scale;
            }
        }
        const bool live = xk != -INFINITY;
        // lanes of one token that name one expert
        const uint32_t same = __match_any_sync(kFullMask, e >= 0 ? my_token * kMaxExperts + e : -1 - lane);
        float slot = 0.f;  // what this slot adds to its expert's logit
        float m_row = 0.f, inv_row = 0.f;
        float v[N];
        if (all) {
            // every row's maximum and sum, kept by its slots' lanes
            for (int t = 0; t < tokens; ++t) {
                load_run<T, N, VEC>(x + (row0 + t) * E + base, count, v);
                float m = v[0];
#pragma unroll
                for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
                m = key_value(warp_max(order_key(m + 0.f)));
                if (m == -INFINITY) m = 0.f;
                float d = 0.f;
#pragma unroll
                for (int i = 0; i < N; i += 2) {
                    const float2 p = exp_pair<false>(
                        make_float2(v[i] - m, i + 1 < N ? v[i + 1] - m : -INFINITY));
                    d += p.x + p.y;
                    v[i] = p.x;
                    if (i + 1 < N) v[i + 1] = p.y;
                }
                d = warp_sum(d);
                const float inv_d = d > 0.f ? __frcp_rn(d) : 0.f;
                // D of this row from its slots
                float part = 0.f;
                if (my_token == t) {
                    m_row = m;
                    inv_row = inv_d;
                    if (live) part = g * (exp1(xk - m) * inv_d);
                }
                const float D = warp_sum(part);
                if (my_token == t) slot = D;
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] *= -inv_d * D;
                store_run<T, N, VEC>(dx + (row0 + t) * E + base, count, v);
            }
            // the slot's own value: s (g - D), with D taken off once below
            const float s = live ? exp1(xk - m_row) * inv_row : 0.f;
            const float D = slot;
            float sum = 0.f;
            if (__any_sync(kFullMask, __popc(same) > 1)) {
#pragma unroll 1
                for (int k = 0; k < 32; ++k) {
                    const float gk = __shfl_sync(kFullMask, g, k);
                    if ((same >> k) & 1) sum += gk;
                }
            } else {
                sum = g;
            }
            slot = s * (sum - D);
        } else {
            float top = 0.f, w;
            if (sh.renorm) {
                top = slot_max(live ? xk : -INFINITY, sh.slots);
                if (sh.sigmoid) top = fminf(top, 0.f);
            }
            const float s = sh.sigmoid ? sigmoid(xk) : 0.f;
            if (!sh.renorm || (sh.sigmoid && xk > 0.f)) {
                w = s;
            } else {
                w = exp1(xk - top);
                if (sh.sigmoid) w = __fdiv_rn(w, 1.f + exp1(xk));
            }
            if (!live) w = 0.f;
            float D = 0.f;
            if (sh.renorm) {
                const float sum = slot_sum(w, sh.slots);
                w = sum > 0.f ? __fdiv_rn(w, sum) : 0.f;
                D = slot_sum(g * w, sh.slots);
            }
            slot = w * (g - D);
            if (sh.sigmoid) slot *= sigmoid(-xk);
            if (!live) slot = 0.f;
            if (__any_sync(kFullMask, __popc(same) > 1)) {
                float sum = 0.f;
#pragma unroll 1
                for (int k = 0; k < 32; ++k) {
                    const float a = __shfl_sync(kFullMask, slot, k);
                    if ((same >> k) & 1) sum += a;
                }
                slot = sum;
            }
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = 0.f;
            for (int t = 0; t < tokens; ++t)
                store_run<T, N, VEC>(dx + (row0 + t) * E + base, count, v);
        }
        __syncwarp();  // orders the rows' stores before the slots'
        if (e >= 0 && (__ffs(same) - 1) == lane) {
            T* at = dx + my_row * E + e;
            if constexpr (sizeof(T) == 4) *at = slot;
            else *at = __float2bfloat16_rn(slot);
        }
        __syncwarp();
    }
}

}  // namespace route
}  // namespace os
