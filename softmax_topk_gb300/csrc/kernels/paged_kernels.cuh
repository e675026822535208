// paged_kernels.cuh -- what moves in and out of a paged key-value cache: new keys
// and values, rotated by their positions on the way, and the pages that follow a
// beam search's choice.
#pragma once

#include <cuda_bf16.h>

#include <climits>
#include <cstdint>

#include "paged_common.cuh"

namespace os {
namespace paged {

// ------------------------------------------------------------------ append
// Token i of sequence b's n new ones goes to position p = lengths[b] - n + i.  With
// angles a_f = p inv_freq_f the pairs (x, y) of the first rot dimensions of q and k
// become (x cos a_f - y sin a_f, y cos a_f + x sin a_f); v is copied.
//
// The angle is reduced in 64 bits: a / 2 pi less its nearest integer has an error of
// three roundings, 2^-51 of the number of turns at most.  For frequencies up to 1 that is
// 2^-22 turns at the last position and below fp32's own up to 2^26.  The rest is in fp32
// (sincospif of twice the fraction).
//
// What bounds it: memory.  36000 tokens of 16 + 8 heads of 128, 426 MB in and out: 69
// us, 6.2 TB/s (0.92 of the copy's rate); a batch of 256 tokens takes 2.7 us, the
// launch and two waits for memory.
struct AppendArgs {
    __nv_bfloat16* k_cache;  // [pages][kv_heads][page_size][D]
    __nv_bfloat16* v_cache;
    const int* table;        // [seqs][width]
    const int* lengths;      // [seqs]
    const __nv_bfloat16 *q, *k, *v;  // q may be NULL
    __nv_bfloat16* q_out;    // [tokens][q_heads][D]
    const int* starts;       // [seqs + 1] or NULL: one token per sequence
    const float* inv_freq;   // [rot / 2]
    int64_t q_stride, k_stride, v_stride, tokens;
    int seqs, width, pages, kv_heads, q_heads, rot;
    PageSplit split;
};

constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 4;  // at most, per CTA

// The last sequence that starts at or before token t (those without tokens end
// before it), or -1 where t is behind the last sequence or before the first.
__device__ __forceinline__ int sequence_of(const int* starts, int seqs, int64_t t, int lane) {
    if (t < *starts || t >= starts[seqs]) return -1;
    // (a lane may look up to 32 steps past lo: beyond 2^31 where there are nearly as many
    // sequences, so the places are unsigned)
    unsigned lo = 0, hi = seqs;  // starts[lo] <= t < starts[hi]
    while (hi - lo > 1) {
        const unsigned step = (hi - lo + 31) / 32;
        const unsigned at = lo + (lane + 1) * step;
        const unsigned ok = __ballot_sync(kFullMask, at < hi && starts[at] <= t);
        const unsigned nlo = lo + __popc(ok) * step;
        hi = min(hi, nlo + step);
        lo = nlo;
    }
    return static_cast<int>(lo);
}

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kAppendThreads)
    append_kernel(const __grid_constant__ AppendArgs a, int per_cta) {
    constexpr int kPairs = D / 16;  // pairs of 16-byte pieces of a head
    __shared__ float2 turn[kAppendTokens][D / 2];
    __shared__ int pos_sh[kAppendTokens], row_sh[kAppendTokens];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * per_cta;
    wait_before();
    let_next();
    if (warp < per_cta) {
        const int64_t t = t0 + warp;
        int pos = -1, row = -1;  // of the pool: page * kv_heads * page_size + slot
        if (t < a.tokens) {
            const int b = a.starts ? sequence_of(a.starts, a.seqs, t, lane) : static_cast<int>(t);
            if (b >= 0) {
                const int64_t p = a.starts ? t + a.lengths[b] - a.starts[b + 1]
                                           : static_cast<int64_t>(a.lengths[b]) - 1;
                pos = static_cast<int>(min(max(p, int64_t(-1)), int64_t(INT_MAX)));
                if (pos >= 0 && pos < a.width * a.split.size) {
                    const int at = a.split.page(pos);
                    const int page = a.table[static_cast<int64_t>(b) * a.width + at];
                    if (static_cast<unsigned>(page) < static_cast<unsigned>(a.pages))
                        row = page * a.kv_heads * a.split.size + pos - at * a.split.size;
                }
            }
        }
        if (lane == 0) pos_sh[warp] = pos, row_sh[warp] = row;
    }
    __syncthreads();
    const int half = a.rot / 2;
    for (int i = tid; i < per_cta * half; i += kAppendThreads) {
        const int w = i / half, f = i % half;
        const double turns = static_cast<double>(max(pos_sh[w], 0)) *
                             (static_cast<double>(a.inv_freq[f]) * 0.15915494309189535);
        const float part = static_cast<float>(turns - rint(turns));
        float s, c;
        sincospif(2.f * part, &s, &c);
        turn[w][f] = make_float2(c, s);
    }
    __syncthreads();
    const int heads = a.q_heads + 2 * a.kv_heads;
    const int items = heads * kPairs;
    for (int i = tid; i < per_cta * items; i += kAppendThreads) {
        const int w = i / items, h = i % items / kPairs, c = i % kPairs;
        const int64_t t = t0 + w;
        if (pos_sh[w] < 0) continue;
        const __nv_bfloat16* from;
        __nv_bfloat16* to;
        const bool is_q = h < a.q_heads, is_v = h >= a.q_heads + a.kv_heads;
        if (is_q) {
            from = a.q + t * a.q_stride + h * D;
            to = a.q_out + (t * a.q_heads + h) * D;
        } else {
            if (row_sh[w] < 0) continue;
            const int hk = h - a.q_heads - (is_v ? a.kv_heads : 0);
            from = (is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride) + hk * D;
            to = (is_v ? a.v_cache : a.k_cache) +
                 (static_cast<int64_t>(row_sh[w]) + static_cast<int64_t>(hk) * a.split.size) * D;
        }
        const bool turned = !is_v && c < a.rot / 16;
        // a pair's two sides: the halves' same places, or neighbours
        const bool apart = !INTERLEAVED && c < a.rot / 16;
        const int p0 = apart ? c : 2 * c, p1 = apart ? c + a.rot / 16 : 2 * c + 1;
        uint4 x = reinterpret_cast<const uint4*>(from)[p0];
        uint4 y = reinterpret_cast<const uint4*>(from)[p1];
        if (turned) {
            float u[16];
            auto* xb = reinterpret_cast<__nv_bfloat162*>(&x);
            auto* yb = reinterpret_cast<__nv_bfloat162*>(&y);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 fx = __bfloat1622float2(xb[e]), fy = __bfloat1622float2(yb[e]);
                u[2 * e] = fx.x, u[2 * e + 1] = fx.y, u[8 + 2 * e] = fy.x, u[9 + 2 * e] = fy.y;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 cs = turn[w][8 * c + e];
                const int i0 = INTERLEAVED ? 2 * e : e, i1 = INTERLEAVED ? 2 * e + 1 : e + 8;
                const float p = u[i0], r = u[i1];
                u[i0] = p * cs.x - r * cs.y;
                u[i1] = r * cs.x + p * cs.y;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                xb[e] = __floats2bfloat162_rn(u[2 * e], u[2 * e + 1]);
                yb[e] = __floats2bfloat162_rn(u[8 + 2 * e], u[9 + 2 * e]);
            }
        }
        reinterpret_cast<uint4*>(to)[p0] = x;
        reinterpret_cast<uint4*>(to)[p1] = y;
    }
}

// ------------------------------------------------------------------ reorder
// Sequence j = (group, beam) goes on as its parent p: the table's entries of p's full
// pages, and a copy of the rows of the page that p has filled in part, in the page
// that out_table names there.  A CTA copies one head of one layer, keys and values.
//
// What bounds it: memory.  256 sequences, 16 layers of 4 heads, half-filled pages of 64:
// 443 MB read and written in 74 us, 6.0 TB/s (95 us with one load of a thread on its way
// at a time).
struct ReorderArgs {
    __nv_bfloat16* k_cache;  // [layers][pages][kv_heads][page_size][D]
    __nv_bfloat16* v_cache;
    const int* table;
    const int* lengths;
    const int* parents;      // [seqs]: beam of the group
    int* out_table;
    int* out_lengths;        // or NULL
    int64_t page_bytes, head_bytes, row_bytes, layer_bytes;
    int seqs, beams, width, pages, kv_heads, layers;
    PageSplit split;
};

constexpr int kReorderThreads = 128;

__device__ __forceinline__ uint4 load_once(const char* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
    return r;
}

__global__ void __launch_bounds__(kReorderThreads)
    reorder_kernel(const __grid_constant__ ReorderArgs a) {
    const int tid = threadIdx.x;
    const int j = blockIdx.x % a.seqs;
    const int part = blockIdx.x / a.seqs;  // (layer, head)
    wait_before();
    let_next();
    const int parent = a.parents[j];
    const bool alive = static_cast<unsigned>(parent) < static_cast<unsigned>(a.beams);
    const int p = alive ? j / a.beams * a.beams + parent : j;
    const int len = alive ? max(0, min(a.lengths[p], a.width * a.split.size)) : 0;
    const int full = a.split.page(len), rest = len - full * a.split.size;
    const int* old_row = a.table + static_cast<int64_t>(p) * a.width;
    int* new_row = a.out_table + static_cast<int64_t>(j) * a.width;
    if (part == 0) {
        // (eight on their way at a time: the tables do not overlap)
        constexpr int kEntries = 8;
        for (int i0 = tid; i0 < full; i0 += kEntries * kReorderThreads) {
            int page[kEntries];
#pragma unroll
            for (int x = 0; x < kEntries; ++x)
                if (i0 + x * kReorderThreads < full) page[x] = old_row[i0 + x * kReorderThreads];
#pragma unroll
            for (int x = 0; x < kEntries; ++x)
                if (i0 + x * kReorderThreads < full) new_row[i0 + x * kReorderThreads] = page[x];
        }
        if (tid == 0 && a.out_lengths) a.out_lengths[j] = len;
    }
    if (rest == 0) return;
    const int from = old_row[full], to = new_row[full];
    if (static_cast<unsigned>(from) >= static_cast<unsigned>(a.pages) ||
        static_cast<unsigned>(to) >= static_cast<unsigned>(a.pages) || from == to)
        return;
    const int head = static_cast<int>(part % a.kv_heads);
    const int64_t base = part / a.kv_heads * a.layer_bytes + head * a.head_bytes;
    const int pieces = static_cast<int>(rest * a.row_bytes / 16);
    const char* k_from = reinterpret_cast<const char*>(a.k_cache) + base + from * a.page_bytes;
    const char* v_from = reinterpret_cast<const char*>(a.v_cache) + base + from * a.page_bytes;
    char* k_to = reinterpret_cast<char*>(a.k_cache) + base + to * a.page_bytes;
    char* v_to = reinterpret_cast<char*>(a.v_cache) + base + to * a.page_bytes;
    // eight loads on their way per thread before the first store
    constexpr int kAtOnce = 4;
    for (int i0 = tid; i0 < pieces; i0 += kAtOnce * kReorderThreads) {
        uint4 k[kAtOnce], v[kAtOnce];
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) {
            const int i = i0 + x * kReorderThreads;
            if (i < pieces) {
                k[x] = load_once(k_from + 16 * static_cast<int64_t>(i));
                v[x] = load_once(v_from + 16 * static_cast<int64_t>(i));
            }
        }
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) {
            const int i = i0 + x * kReorderThreads;
            if (i < pieces) {
                reinterpret_cast<uint4*>(k_to)[i] = k[x];
                reinterpret_cast<uint4*>(v_to)[i] = v[x];
            }
        }
    }
}

}  // namespace paged
}  // namespace os
