// sample_kernel.cuh -- one draw per row of logits: temperature, top-k, top-p and
// min-p from given uniform numbers.
//
// With m the row's maximum, weights w_c = e^((x_c - m) / T).  Sorted by (logit
// descending, column ascending) the filters each keep a prefix: top-k the
// first k; top-p the shortest prefix of those whose weight reaches p times
// theirs; min-p the columns with w >= min_p.  The draw is the lowest kept column
// whose running sum, in column order, exceeds u times the kept weight.
//
// Exact draws.  Where a cut or a draw falls depends on sums of up to 2^31
// weights compared with a border, so the sums are kept as integers: a weight
// is a multiple of 2^-B (B = 62 - log2 cols, at most 44), computed in two fp32
// parts to about 2^-38 relative, and a sum of them is a 64-bit integer.  Sums
// then do not depend on how the row was split or in which order atomics came,
// and a draw that differs from the one in real arithmetic needs u within about
// 2^-38 of a border.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "ops.cuh"

namespace os {
namespace sample {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
using u64 = unsigned long long;

// 2^(j/64) in two fp32 parts, j = 0..63
__device__ const float2 kPow2[64] = {
    {1.f, 0.f}, {0x1.02c9a4p+0f, -0x1.887fap-28f}, {0x1.059b0ep+0f, -0x1.9d4f52p-25f},
    {0x1.087452p+0f, -0x1.e2990ep-26f}, {0x1.0b5586p+0f, 0x1.9f3122p-25f}, {0x1.0e3ec4p+0f, -0x1.a585ccp-25f},
    {0x1.11301ep+0f, -0x1.fdb496p-25f}, {0x1.1429aap+0f, 0x1.d525bcp-25f}, {0x1.172b84p+0f, -0x1.c15742p-27f},
    {0x1.1a35bep+0f, 0x1.6df96ep-25f}, {0x1.1d4874p+0f, -0x1.d2e8cap-25f}, {0x1.2063b8p+0f, 0x1.0c519ap-25f},
    {0x1.2387a6p+0f, 0x1.ceac48p-25f}, {0x1.26b456p+0f, 0x1.789f38p-26f}, {0x1.29e9ep+0f, -0x1.5c0424p-25f},
    {0x1.2d285ap+0f, 0x1.b900c2p-26f}, {0x1.306fep+0f, 0x1.4636e2p-25f}, {0x1.33c08cp+0f, -0x1.b37d2p-25f},
    {0x1.371a74p+0f, -0x1.18aac6p-25f}, {0x1.3a7db4p+0f, -0x1.634c02p-25f}, {0x1.3dea64p+0f, 0x1.824684p-25f},
    {0x1.4160a2p+0f, 0x1.f72e2ap-28f}, {0x1.44e086p+0f, 0x1.8624b4p-30f}, {0x1.486a2cp+0f, -0x1.47d866p-25f},
    {0x1.4bfdaep+0f, -0x1.593abcp-25f}, {0x1.4f9b28p+0f, -0x1.2c5a6cp-25f}, {0x1.5342b6p+0f, -0x1.2c561p-25f},
    {0x1.56f474p+0f, -0x1.295b04p-25f}, {0x1.5ab07ep+0f, -0x1.5bd5ecp-27f}, {0x1.5e76f2p+0f, -0x1.4a5bd6p-25f},
    {0x1.6247ecp+0f, -0x1.f8b55p-25f}, {0x1.662388p+0f, 0x1.2a9112p-27f}, {0x1.6a09e6p+0f, 0x1.9fcef4p-26f},
    {0x1.6dfb24p+0f, -0x1.cd72e8p-27f}, {0x1.71f75ep+0f, 0x1.1d8beep-25f}, {0x1.75feb6p+0f, -0x1.37b306p-25f},
    {0x1.7a1148p+0f, -0x1.829fdp-25f}, {0x1.7e2f34p+0f, -0x1.261634p-25f}, {0x1.82589ap+0f, -0x1.accc7cp-26f},
    {0x1.868d9ap+0f, -0x1.2edb44p-26f}, {0x1.8ace54p+0f, 0x1.15506ep-27f}, {0x1.8f1aeap+0f, -0x1.baa232p-26f},
    {0x1.93737cp+0f, -0x1.e64744p-25f}, {0x1.97d82ap+0f, -0x1.0d8d84p-31f}, {0x1.9c4918p+0f, 0x1.51f848p-27f},
    {0x1.a0c668p+0f, -0x1.2886a6p-26f}, {0x1.a5503cp+0f, -0x1.b83b54p-25f}, {0x1.a9e6b6p+0f, -0x1.50c048p-25f},
    {0x1.ae89fap+0f, -0x1.a94b14p-26f}, {0x1.b33a2cp+0f, -0x1.ec3a82p-26f}, {0x1.b7f77p+0f, -0x1.a09438p-25f},
    {0x1.bcc1eap+0f, -0x1.f687c6p-25f}, {0x1.c199bep+0f, -0x1.3d56b2p-27f}, {0x1.c67f12p+0f, 0x1.cafa2ap-25f},
    {0x1.cb720ep+0f, -0x1.8837ccp-27f}, {0x1.d072d4p+0f, 0x1.40f13p-25f}, {0x1.d5818ep+0f, -0x1.822dbcp-27f},
    {0x1.da9e6p+0f, 0x1.ed9942p-27f}, {0x1.dfc974p+0f, -0x1.908c94p-25f}, {0x1.e502eep+0f, 0x1.e2cffep-26f},
    {0x1.ea4afap+0f, 0x1.52486cp-27f}, {0x1.efa1bep+0f, 0x1.cc2b44p-25f}, {0x1.f50766p+0f, -0x1.246ebp-26f},
    {0x1.fa7c18p+0f, 0x1.9e90d8p-28f},
};

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

// A row's weight function: w(x) = e^((x - m) / T) as a multiple of 2^-bits.
struct Weight {
    float m, c_hi, c_lo;  // maximum; log2 e / T in two parts
    int bits;             // 31..44
    const float2* table;  // kPow2 in shared memory

    // (x - m) log2 e / T = n + j/64 + g, |g| <= 1/128; 2^g - 1 = e^y - 1 with
    // y = g ln 2 = y_h + y_l; every product whose rounding would show at 2^-38
    // carries its residual.
    __device__ __forceinline__ u64 operator()(float x) const {
        if (x == m) return 1ull << bits;
        const float dh = x - m;
        const float bb = dh - x;
        const float dl = (x - (dh - bb)) + (-m - bb);  // x - m = dh + dl exactly
        const float th = dh * c_hi;
        if (!(th > -60.f)) return 0;  // below 2^-60, -inf
        const float tl = fmaf(dh, c_hi, -th) + fmaf(dh, c_lo, dl * c_hi);
        const float uf = fmaf(th, 64.f, expc::kRound);
        const float un = uf - expc::kRound;
        const float gh = fmaf(un, -0x1p-6f, th);
        const float g = gh + tl;
        const float gl = tl - (g - gh);
        const float yh = g * 0x1.62e43p-1f;
        const float yl = fmaf(g, 0x1.62e43p-1f, -yh) + fmaf(g, -0x1.05c61p-29f, gl * 0x1.62e43p-1f);
        const float poly = fmaf(yh, fmaf(yh, 0x1.555556p-5f, 0x1.555556p-3f), 0.5f);
        const float r = fmaf(yh * yh, poly, yl);
        const int i = __float_as_int(uf) - __float_as_int(expc::kRound);
        const float2 t = table[i & 63];
        const float wh = fmaf(t.x, yh, t.x);
        const float wl = fmaf(t.x, r, fmaf(t.x, yh, t.x - wh) + fmaf(t.y, yh, t.y));
        const float s = __int_as_float(((i >> 6) + 24 + 127) << 23);  // 2^(n + 24)
        const float i1 = rintf(wh * s);
        const float rest = fmaf(wh, s, -i1) + wl * s;
        const float i2 = rintf(rest * __int_as_float((bits - 24 + 127) << 23));
        const long long w = (static_cast<long long>(__float2int_rn(i1)) << (bits - 24)) + __float2int_rn(i2);
        return w > 0 ? static_cast<u64>(w) : 0ull;
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

struct Shared {
    float2 table[64];
    u64 mass[256];
    uint32_t count[256];
    u64 warp[kWarps];
    u64 result[2];
    uint32_t found[2];
};

// Sum of v over the CTA (all threads get it).
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

// Digit by digit from the top, the largest key T such that the elements with
// key >= T amount to at least `want`, an element amounting to amount(key) (its
// count or its weight).  On return `above` is what the keys > T amount to and
// `ties` the number of elements with key T.  each(f) calls f(key) for every
// element of the calling thread's share.
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
                atomicAdd(&sh.mass[b], amount(key) * times);
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

template <typename T>
__global__ void __launch_bounds__(kThreads)
sample_kernel(const T* __restrict__ x, const float* __restrict__ u, int* __restrict__ out,
              float* __restrict__ prob, int64_t rows, int cols, const Settings s, int bits) {
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < 64) sh.table[tid] = kPow2[tid];
    // columns of a warp: a run of whole 32-column pieces
    const int pieces = (cols + 31) / 32;
    const int64_t per_warp = int64_t(pieces + kWarps - 1) / kWarps * 32;
    const int64_t lo = min(int64_t(cols), warp * per_warp);
    const int64_t hi = min(int64_t(cols), (warp + 1) * per_warp);
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const T* p = x + row * cols;
        // ---- maximum and its lowest column
        u64 top = 0;
        for (int64_t c = tid; c < cols; c += kThreads) {
            const u64 k = (u64(order_key(widen(p[c]))) << 32) | (0xffffffffu - uint32_t(c));
            top = k > top ? k : top;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const u64 t = __shfl_xor_sync(kFullMask, top, o);
            top = t > top ? t : top;
        }
        __syncthreads();
        if (lane == 0) sh.warp[warp] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWarps; ++i) top = sh.warp[i] > top ? sh.warp[i] : top;
        const uint32_t top_key = uint32_t(top >> 32);
        const float T_ = s.temperature ? s.temperature[row] : s.temperature_all;
        if (top_key <= kKeyNegInf || !(T_ > 0.f)) {
            if (tid == 0) {
                out[row] = top_key <= kKeyNegInf ? -1 : int(0xffffffffu - uint32_t(top));
                if (prob) prob[row] = top_key <= kKeyNegInf ? 0.f : 1.f;
            }
            continue;
        }
        Weight w;
        w.m = key_value(top_key);
        const double c = fmin(1.4426950408889634074 / double(T_), 1e30);
        w.c_hi = float(c);
        w.c_lo = float(c - double(w.c_hi));
        w.bits = bits;
        w.table = sh.table;
        const int k = s.top_k ? s.top_k[row] : s.top_k_all;
        const float tp = s.top_p ? s.top_p[row] : s.top_p_all;
        const float mp = s.min_p ? s.min_p[row] : s.min_p_all;

        // ---- the kept prefix: keys > cut, and the first `room` columns with key == cut
        uint32_t cut = kKeyNegInf, room = 0;
        bool some = false;  // of the columns at the cut, only the first `room`
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
            } else if (!some) {
                room = ties;
            }
        }
        if (tp < 1.f) {
            const float pc = fmaxf(tp, 0.f);
            u64 total = 0;
            for (int64_t i = tid; i < cols; i += kThreads) {
                const float v = widen(p[i]);
                if (order_key(v) > cut) total += w(v);
            }
            const u64 w_cut = cut > kKeyNegInf ? w(key_value(cut)) : 0;
            total = cta_sum(sh, total) + w_cut * room;
            const u64 frac = __double2ull_rz(double(pc) * 18446744073709551616.0);
            u64 want = __umul64hi(frac, total) + (frac * total != 0);
            if (want == 0) want = 1;
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
        if (mp > 0.f) {
            const float q = fminf(mp, 1.f);
            const double thr = q < 1.f ? double(w.m) + double(T_) * log(double(q)) : double(w.m);
            uint32_t key = order_key(__double2float_ru(thr));
            if (key <= kKeyNegInf) key = kKeyNegInf + 1;
            if (key > top_key) key = top_key;
            if (key > cut) {  // everything from this key on
                cut = key - 1;
                some = false;
                room = 0;
            }
        }
        if (cut > kKeyNegInf && !some && room > 0) --cut;  // all columns at the cut stay: keys > cut - 1

        // ---- the last column that stays among those at the cut
        int last = -1;
        if (some) {
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
            last = int(sh.found[0]);
        }

        // ---- the draw, in column order
        const float uu = u[row] > 0.f ? fminf(u[row], 0x1.fffffep-1f) : 0.f;
        auto kept_weight = [&](int64_t i) -> u64 {
            const float v = widen(p[i]);
            const uint32_t key = order_key(v);
            if (!(key > cut || (key == cut && i <= last))) return 0;
            const u64 a = w(v);
            return uu == 0.f && a == 0 ? 1ull : a;  // u = 0: the first kept column, however small
        };
        u64 mine = 0;
        for (int64_t i = lo + lane; i < hi; i += 32) mine += kept_weight(i);
        mine = warp_sum64(mine);
        __syncthreads();
        if (lane == 0) sh.warp[warp] = mine;
        __syncthreads();
        u64 before = 0, total = 0;
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp) before += sh.warp[i];
            total += sh.warp[i];
        }
        const u64 target = __umul64hi(__double2ull_rz(double(uu) * 18446744073709551616.0), total);
        if (before <= target && target < before + mine) {
            u64 run = before;
            for (int64_t i0 = lo; i0 < hi; i0 += 32) {
                const u64 a = i0 + lane < hi ? kept_weight(i0 + lane) : 0;
                const u64 upto = run + warp_prefix64(a, lane);
                const uint32_t hit = __ballot_sync(kFullMask, upto > target);
                if (hit) {
                    if (lane == __ffs(hit) - 1) {
                        out[row] = int(i0 + lane);
                        // the weight itself, not its integer: a small one keeps its digits
                        if (prob) {
                            const float v = widen(p[i0 + lane]);
                            const double e = v == w.m ? 1.0 : exp((double(v) - double(w.m)) / double(T_));
                            prob[row] = float(ldexp(e, bits) / double(total));
                        }
                    }
                    break;
                }
                run = __shfl_sync(kFullMask, upto, 31);
            }
        }
    }
}

}  // namespace sample
}  // namespace os
