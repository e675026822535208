// paged_attention_kernel.cuh -- attention of one new token per sequence over a
// paged key-value cache, split over the cache's length and joined.
//
// Per sequence b, key head h and query head of its group:
//   s_j = scale q . k_j,  O = sum_j e^(s_j - m) v_j / l,  l = sum_j e^(s_j - m),
//   L = m + ln l,  over the keys j < lengths[b] whose page is in the pool.
//
// A (b, h, up to 8 NT query heads) is a unit, 16 keys of it a block.  The blocks
// of all units, laid end to end, are shared out evenly: every CTA gets a run of
// them and every warp a run of the CTA's, whatever the sequences' lengths, so a
// long sequence is split as far as the GPU is wide.  A unit that lies in one
// warp's run is written by it; the pieces of one that does not are joined by
// the CTA after its last block, and those of one that spans CTAs by the second
// kernel, from the workspace, in the order of the keys: the same bits from call
// to call.
//
// The products run on the tensor cores as S^T = K Q^T (16 keys x 8 heads) and
// O^T = V^T P^T (D x 8 heads): eight query heads fill the narrow side, where
// one query per sequence would leave 15 of 16 rows of the usual form empty.
//
// Every warp has a ring of its own in shared memory, filled by asynchronous copies
// of 16 bytes, K and V of two blocks ahead of the one it works on: the rows of a
// block may lie in 16 different pages, and no warp waits for another.  (Keys and
// values loaded straight into the fragments' registers, where a warp's loads are in
// flight only half of the time, took 430 us where the ring takes 319.)
//
// What bounds it: memory, once there is enough to read.  64 sequences of 4096
// keys, 16 heads of 128: 2.15 GB in 316 to 321 us, 6.7 TB/s, the measured copy's rate (four
// schedulers issue in a quarter of their cycles).  128 sequences of up to 2000, 16
// heads of 64: 96 us, 5.9 TB/s; one of 131072, 2 key heads: 29 us, 4.6 TB/s; one of
// 1000: 6.6 us.  What is left is a constant of 6 to 10 us: three waits in a row for
// memory (lengths, table, first keys, 2.5 us), the last block, its pieces and the
// second kernel (4 us), and two launches.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "paged_common.cuh"

namespace os {
namespace paged {

constexpr int kBlock = 16;  // keys per block
// The running maximum is raised only when a score passes it by this much (in
// bits), so weights stay below 2^8 and nearly every block skips the rescaling.
constexpr float kSlack = 8.f;
constexpr float kLn2f = 0.693147182f;

struct AttnArgs {
    const __nv_bfloat16* q;  // [seqs][q_stride], heads of D
    const __nv_bfloat16* k;  // [pages][kv_heads][page_size][D]
    const __nv_bfloat16* v;
    const int* table;        // [seqs][width]
    const int* lengths;      // [seqs]
    __nv_bfloat16* out;      // [seqs][heads][D]
    float* lse;              // [seqs][heads] or NULL
    float* parts;            // workspace: two pieces per CTA
    int4* tails;             // per CTA: of the unit that goes on behind it, row of out (or -1), CTAs, heads
    int64_t q_stride;
    PageSplit split;
    int seqs, width, pages, kv_heads;
    int group, chunks, units;  // query heads per key head; their chunks; kv_heads * chunks
    int ctas;                  // of the first kernel
    float scale_log2;          // scale * log2 e
};

template <int D, int NT>
struct AttnShape {
    static constexpr int kHeads = 8 * NT;  // query heads of a unit
    // 96 to 128 KB on their way; ten warps of D = 128 and sixteen of D = 64 were slower
    // (61 ragged sequences 54.0 -> 55.0 us, 128 x 2000 98.9 -> 105)
    static constexpr int kWarps = D == 128 ? 8 : 12;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kRow = D * 2;               // bytes of a key
    static constexpr int kSide = kBlock * kRow;      // K or V of a block
    static constexpr int kAhead = 2;                 // blocks asked for ahead
    static constexpr int kHeadStride = D + 4;        // of a piece: spreads the heads over the banks
    static constexpr int kPiece = kHeads * kHeadStride + 2 * kHeads;  // floats: O, m, l
    static constexpr int kM = kHeads * kHeadStride, kL = kM + kHeads;
};

template <int D, int NT>
struct AttnShared {
    using S = AttnShape<D, NT>;
    unsigned char ring[S::kWarps][S::kAhead][2][S::kSide];  // K, V of a block
    float head[S::kWarps][S::kPiece];  // the piece of a unit begun before the warp
    // The warps' pieces: [0] of a unit begun before the warp, [1] of one begun in it; where
    // the unit begins in the line (or -1), and of [1] where it ends and its first row of out
    int unit[2][S::kWarps];
    int end[S::kWarps], row[S::kWarps], head_row;  // head_row: of [0] of the first warp
    // The piece that the warp began lies in its ring, which is empty when it is written.
    __device__ __forceinline__ float* piece(int warp, int which) {
        static_assert(S::kPiece * sizeof(float) <= sizeof(ring[0]), "a piece fits the ring");
        return which ? reinterpret_cast<float*>(ring[warp]) : head[warp];
    }
};

// 16 bytes to shared memory; zeros where `there` is false (nothing is read then).
__device__ __forceinline__ void copy_async(uint32_t to, const void* from, bool there) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;"
                 :: "r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}

template <bool TRANS>
__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t at) {
    if constexpr (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ float ex2f(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ int used_length(const AttnArgs& a, int b) {
    const int len = a.lengths[b];
    return max(0, min(len, a.width * a.split.size));
}

// (a length may be near 2^31)
__device__ __forceinline__ int blocks_in(int len) {
    return static_cast<int>((static_cast<unsigned>(len) + kBlock - 1) / kBlock);
}

// A place in the line of blocks: block j of query heads' chunk c of key head h of
// sequence b.
struct Cursor {
    int b, h, c, j, blocks, len;
    __device__ __forceinline__ void sequence(const AttnArgs& a) {
        len = used_length(a, b);
        blocks = blocks_in(len);
    }
    __device__ __forceinline__ void next(const AttnArgs& a) {
        if (++j < blocks) return;
        j = 0;
        if (++c < a.chunks) return;
        c = 0;
        if (++h < a.kv_heads) return;
        h = 0;
        do {
            if (++b >= a.seqs) return;
            sequence(a);
        } while (blocks == 0);
    }
};

// Where key 16 j + (lane mod 16) lies: its page (asked for; -1 behind the length), and its
// row in the page.
struct Key {
    int page, in;
    __device__ __forceinline__ void ask(const AttnArgs& a, const Cursor& c, int lane) {
        const int key = c.j * kBlock + (lane & 15);
        const int at = a.split.page(key);
        page = -1;
        if (key < c.len) page = a.table[static_cast<int64_t>(c.b) * a.width + at];
        in = c.h * a.split.size + key - at * a.split.size;
    }
    // the pool's row, or -1: no such page
    __device__ __forceinline__ int row(const AttnArgs& a) const {
        return static_cast<unsigned>(page) < static_cast<unsigned>(a.pages)
                   ? page * a.kv_heads * a.split.size + in : -1;
    }
};

// One head's L from m and l; without keys -inf, and NaN where a score was one.
__device__ __forceinline__ void store_lse(const AttnArgs& a, int row, float m, float l) {
    if (a.lse) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2f;
}

// What O's sums are multiplied by.
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }

// A piece's weight beside the joined maximum; a piece without keys has none.
__device__ __forceinline__ float piece_weight(float m, float joined) {
    return m == -INFINITY ? 0.f : ex2f(m - joined);
}

template <int D, int NT>
__global__ void __launch_bounds__(AttnShape<D, NT>::kThreads, 1)
    paged_attention_kernel(const __grid_constant__ AttnArgs a) {
    using S = AttnShape<D, NT>;
    constexpr int kTiles = D / 16;    // contraction steps of K Q^T, 16-row tiles of O^T
    constexpr int kChunks = D / 8;    // 16-byte pieces of a row
    constexpr int kLanesRow = kChunks;             // lanes that copy one row
    constexpr int kRowsAtOnce = 32 / kLanesRow;
    extern __shared__ __align__(16) unsigned char raw[];
    auto& sh = *reinterpret_cast<AttnShared<D, NT>*>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    wait_before();

    // ---- this warp's run of blocks: every warp adds up the lengths itself, which for
    // the usual numbers of sequences takes less time than waiting for others
    if (lane < 2) sh.unit[lane][warp] = -1;
    auto blocks_of = [&](int b) {
        return b < a.seqs ? blocks_in(used_length(a, b)) : 0;
    };
    auto scanned = [&](int v) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int before = __shfl_up_sync(kFullMask, v, o);
            if (lane >= o) v += before;
        }
        return v;
    };
    const int per_lane = (a.seqs + 31) / 32;
    int mine = 0;
#pragma unroll 4
    for (int i = 0; i < per_lane; ++i) mine += blocks_of(lane * per_lane + i);
    const int upto = scanned(mine) * a.units;
    const int total = __shfl_sync(kFullMask, upto, 31);
    // CTAs, then warps, take equal runs; the last ones may have none
    const int per_cta = (total + gridDim.x - 1) / gridDim.x;
    const int cta_begin = static_cast<int>(
        min(static_cast<int64_t>(total), static_cast<int64_t>(per_cta) * blockIdx.x));
    const int cta_end = cta_begin + min(total - cta_begin, per_cta);
    const int per_warp = (cta_end - cta_begin + S::kWarps - 1) / S::kWarps;
    const int begin = min(cta_end, cta_begin + per_warp * warp);
    const int n = min(cta_end - begin, per_warp);
    const int heads = a.kv_heads * a.group;

    // ---- sequences without keys
    for (int b = blockIdx.x; b < a.seqs; b += gridDim.x) {
        if (used_length(a, b) > 0) continue;
        for (int i = tid; i < heads * (D / 8); i += S::kThreads)
            reinterpret_cast<uint4*>(a.out)[static_cast<int64_t>(b) * heads * (D / 8) + i] =
                make_uint4(0, 0, 0, 0);
        for (int i = tid; a.lse && i < heads; i += S::kThreads)
            a.lse[static_cast<int64_t>(b) * heads + i] = -INFINITY;
    }

    if (n > 0) {
        Cursor cur;
        int unit_end;  // of the current unit, in the line
        {
            // the lane whose sequences hold `begin`, then the sequence
            const int holder = __ffs(__ballot_sync(kFullMask, upto > begin)) - 1;
            int before = __shfl_sync(kFullMask, upto - mine * a.units, holder);
            cur.b = holder * per_lane;
            while (per_lane > 1) {
                const int here = scanned(blocks_of(cur.b + lane)) * a.units;
                const unsigned past = __ballot_sync(kFullMask, before + here > begin);
                const int skip = past ? __ffs(past) - 1 : 32;
                if (skip > 0) before += __shfl_sync(kFullMask, here, skip - 1);
                cur.b += skip;
                if (past) break;
            }
            cur.sequence(a);
            const int unit = (begin - before) / cur.blocks;
            cur.j = begin - before - unit * cur.blocks;
            cur.h = a.chunks == 1 ? unit : unit / a.chunks;
            cur.c = a.chunks == 1 ? 0 : unit % a.chunks;
            unit_end = begin - cur.j + cur.blocks;
        }
        uint32_t q[NT][kTiles][2];
        float o[NT][kTiles][4], m[NT][2], l[NT][2];
        const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(sh.ring[warp]));
        uint32_t place = ring;  // of the current block
        // K or V of 16 rows; a row's 16-byte pieces change places with its low bits, so that
        // the same piece of eight rows lies in different banks.  Rows that are not there are
        // zeros: their weights are 0, and what memory holds there may be no number.
        auto fetch = [&](const __nv_bfloat16* pool, uint32_t to, int rows) {
            const int chunk = lane % kLanesRow, r0 = lane / kLanesRow;
#pragma unroll
            for (int i = 0; i < kBlock / kRowsAtOnce; ++i) {
                const int r = r0 + i * kRowsAtOnce;
                const int row = __shfl_sync(kFullMask, rows, r);
                copy_async(to + r * S::kRow + ((chunk ^ (r & 7)) * 16),
                           pool + static_cast<int64_t>(max(row, 0)) * D + chunk * 8, row >= 0);
            }
        };

        auto load_q = [&]() {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int head = cur.c * S::kHeads + nt * 8 + g;
                const __nv_bfloat16* p =
                    a.q + cur.b * a.q_stride + (cur.h * a.group + head) * D + 2 * t;
#pragma unroll
                for (int j = 0; j < kTiles; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        q[nt][j][e] = head < a.group
                                          ? *reinterpret_cast<const uint32_t*>(p + 16 * j + 8 * e)
                                          : 0u;
            }
        };
        load_q();

        // rows of the current block and of kAhead behind it; the one after those is asked
        // for a block before it is used
        int rows[S::kAhead + 1];
        Cursor ahead = cur;
        Key key[S::kAhead + 1];
#pragma unroll
        for (int i = 0; i <= S::kAhead; ++i) {
            key[i].page = -1;
            if (i < n) {
                if (i > 0) ahead.next(a);
                key[i].ask(a, ahead, lane);
            }
        }
#pragma unroll
        for (int i = 0; i <= S::kAhead; ++i) rows[i] = key[i].row(a);
#pragma unroll
        for (int i = 0; i < S::kAhead; ++i) {
            if (i < n) fetch(a.k, ring + 2 * i * S::kSide, rows[i]);
            copy_commit();
            if (i < n) fetch(a.v, ring + (2 * i + 1) * S::kSide, rows[i]);
            copy_commit();
        }
        bool fresh = true;       // the block begins a unit, or the run
        bool begun_here = cur.j == 0;
        for (int i = 0; i < n; ++i) {
            Key after;
            after.page = -1;
            if (i + S::kAhead + 1 < n) {
                ahead.next(a);
                after.ask(a, ahead, lane);
            }
            if (fresh) {
                if (i > 0) load_q();
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int j = 0; j < kTiles; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[nt][j][e] = 0.f;
                    m[nt][0] = m[nt][1] = -INFINITY;
                    l[nt][0] = l[nt][1] = 0.f;
                }
            }
            // ---- scores (two sums that take turns: half the wait for each other)
            copy_wait<2 * S::kAhead - 1>();
            __syncwarp();
            float s[NT][4], s_odd[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[nt][e] = s_odd[nt][e] = 0.f;
            {
                const int r = lane & 15;
                const uint32_t at = place + r * S::kRow;
#pragma unroll
                for (int j = 0; j < kTiles; ++j) {
                    uint32_t kf[4];
                    load_matrices<false>(kf, at + (((2 * j + (lane >> 4)) ^ (r & 7)) * 16));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16816(j & 1 ? s_odd[nt] : s[nt], kf, q[nt][j][0], q[nt][j][1]);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[nt][e] += s_odd[nt][e];
            // K of a later block into this one's place
            __syncwarp();
            if (i + S::kAhead < n) fetch(a.k, place, rows[S::kAhead]);
            copy_commit();
            const bool seen0 = __shfl_sync(kFullMask, rows[0], g) >= 0;
            const bool seen1 = __shfl_sync(kFullMask, rows[0], g + 8) >= 0;
            // ---- weights: s[nt] holds (key g, heads 2t, 2t+1), (key g + 8, the same)
            bool raise = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[nt][e] = (e < 2 ? seen0 : seen1) ? s[nt][e] * a.scale_log2 : -INFINITY;
                    raise |= s[nt][e] > m[nt][e & 1] + kSlack;
                }
            }
            if (__any_sync(kFullMask, raise)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = fmaxf(s[nt][e], s[nt][e + 2]);
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1)
                            top = fmaxf(top, __shfl_xor_sync(kFullMask, top, x));
                        top = fmaxf(top, m[nt][e]);
                        const float f = piece_weight(m[nt][e], top);
                        m[nt][e] = top;
                        l[nt][e] *= f;
#pragma unroll
                        for (int j = 0; j < kTiles; ++j) {
                            o[nt][j][e] *= f;
                            o[nt][j][e + 2] *= f;
                        }
                    }
                }
            }
            // Weights as the sum of two bf16 numbers, one product each: 2^-17 of a
            // weight, where one number would leave 2^-9 in every sum.
            uint32_t p[NT][2], p_lo[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // (nothing seen so far: the scores are -inf, the weights 0)
                const float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0];
                const float m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
                for (int i2 = 0; i2 < 2; ++i2) {
                    const float w0 = ex2f(s[nt][2 * i2] - m0), w1 = ex2f(s[nt][2 * i2 + 1] - m1);
                    l[nt][0] += w0;
                    l[nt][1] += w1;
                    const uint32_t w = pack_bf16(w0, w1);
                    p[nt][i2] = transpose8x8(w);
                    p_lo[nt][i2] = transpose8x8(pack_bf16(w0 - __uint_as_float(w << 16),
                                                          w1 - __uint_as_float(w & 0xffff0000u)));
                }
            }
            // ---- O^T += V^T P^T, and V of a later block
            copy_wait<2 * S::kAhead - 1>();
            __syncwarp();
            {
                const int r = (lane & 7) + 8 * (lane >> 4);
                const uint32_t at = place + S::kSide + r * S::kRow;
#pragma unroll
                for (int j = 0; j < kTiles; ++j) {
                    uint32_t vf[4];
                    load_matrices<true>(vf, at + (((2 * j + ((lane >> 3) & 1)) ^ (r & 7)) * 16));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma16816(o[nt][j], vf, p[nt][0], p[nt][1]);
                        mma16816(o[nt][j], vf, p_lo[nt][0], p_lo[nt][1]);
                    }
                }
            }
            __syncwarp();
            if (i + S::kAhead < n) fetch(a.v, place + S::kSide, rows[S::kAhead]);
            copy_commit();
            place += 2 * S::kSide;
            if (place == ring + 2 * S::kAhead * S::kSide) place = ring;
#pragma unroll
            for (int x = 0; x < S::kAhead; ++x) rows[x] = rows[x + 1];
            rows[S::kAhead] = after.row(a);
            fresh = cur.j + 1 == cur.blocks;
            if (fresh || i + 1 == n) {
                // ---- the unit's last block, or the run's
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1)
                            l[nt][e] += __shfl_xor_sync(kFullMask, l[nt][e], x);
                const int head0 = cur.c * S::kHeads;
                const int row0 = cur.b * heads + cur.h * a.group + head0;
                if (fresh && begun_here) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int head = nt * 8 + 2 * t + e;
                            if (head0 + head >= a.group) continue;
                            const float f = inverse(l[nt][e]);
                            if (g == 0) store_lse(a, row0 + head, m[nt][e], l[nt][e]);
                            __nv_bfloat16* to =
                                a.out + static_cast<int64_t>(row0 + head) * D + g;
#pragma unroll
                            for (int j = 0; j < kTiles; ++j) {
                                to[16 * j] = __float2bfloat16(f * o[nt][j][e]);
                                to[16 * j + 8] = __float2bfloat16(f * o[nt][j][2 + e]);
                            }
                        }
                    }
                } else {
                    const int which = begun_here ? 1 : 0;
                    float* piece = sh.piece(warp, which);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int head = nt * 8 + 2 * t + e;
                            if (g == 0) {
                                piece[S::kM + head] = m[nt][e];
                                piece[S::kL + head] = l[nt][e];
                            }
                            float* to = piece + head * S::kHeadStride + g;
#pragma unroll
                            for (int j = 0; j < kTiles; ++j) {
                                to[16 * j] = o[nt][j][e];
                                to[16 * j + 8] = o[nt][j][2 + e];
                            }
                        }
                    }
                    if (lane == 0) {
                        sh.unit[which][warp] = unit_end - cur.blocks;  // (where it begins)
                        if (which) sh.end[warp] = unit_end, sh.row[warp] = row0;
                        else if (warp == 0) sh.head_row = row0;
                    }
                }
                begun_here = true;
            }
            if (i + 1 < n) {
                cur.next(a);
                if (fresh) unit_end += cur.blocks;
            }
        }
    }
    __syncthreads();

    // The join's CTAs, which wait for this grid's end themselves: not before the keys are
    // read (at the start 1 x 1000 took 7.2 us, 1 x 131072 31.7, the 61 ragged ones 51.2; here
    // 7.0, 31.0, 50.8).
    let_next();
    // ---- pieces of units that warps share: unit j begins before the CTA (0) or in warp
    // j - 1; the warps share its heads out
    const int first_of = lane < S::kWarps ? sh.unit[0][lane] : -1;
    const int begun_by = lane < S::kWarps ? sh.unit[1][lane] : -1;
    const bool goes_on = begun_by >= 0 && sh.end[min(lane, S::kWarps - 1)] > cta_end;
    const unsigned open_ones = __ballot_sync(kFullMask, goes_on);
#pragma unroll 1
    for (int j = 0; j <= S::kWarps; ++j) {
        const int w0 = max(j - 1, 0), slot = j > 0;
        const int unit = __shfl_sync(kFullMask, slot ? begun_by : first_of, w0);
        if (unit < 0) continue;
        // this piece, and the first ones of the warps behind it that go on with the unit
        const unsigned same = __ballot_sync(kFullMask, first_of == unit);
        const int parts = __ffs(~(same >> (w0 + 1)));
        const bool open = slot == 0 || (open_ones >> w0 & 1);  // other CTAs have pieces too
        float* to = a.parts + (2 * static_cast<int64_t>(blockIdx.x) + slot) * S::kPiece;
        const int row0 = slot ? sh.row[w0] : sh.head_row;
        const int left = a.group - row0 % a.group;  // heads of the unit's chunk
#pragma unroll 1
        for (int head = warp; head < min(S::kHeads, left); head += S::kWarps) {
            float top = -INFINITY;
#pragma unroll 4
            for (int i = 0; i < parts; ++i)
                top = fmaxf(top, sh.piece(w0 + i, i ? 0 : slot)[S::kM + head]);
            float sum = 0.f, acc[D / 32] = {};
#pragma unroll 4
            for (int i = 0; i < parts; ++i) {
                const float* from = sh.piece(w0 + i, i ? 0 : slot);
                const float f = piece_weight(from[S::kM + head], top);
                sum += f * from[S::kL + head];
#pragma unroll
                for (int x = 0; x < D / 32; ++x)
                    acc[x] += f * from[head * S::kHeadStride + lane * (D / 32) + x];
            }
            if (open) {
#pragma unroll
                for (int x = 0; x < D / 32; ++x)
                    to[head * S::kHeadStride + lane * (D / 32) + x] = acc[x];
                if (lane == 0) {
                    to[S::kM + head] = top;
                    to[S::kL + head] = sum;
                }
            } else {
                const float f = inverse(sum);
#pragma unroll
                for (int x = 0; x < D / 32; x += 2)
                    *reinterpret_cast<uint32_t*>(a.out + static_cast<int64_t>(row0 + head) * D +
                                                 lane * (D / 32) + x) =
                        pack_bf16(f * acc[x], f * acc[x + 1]);
                if (lane == 0) store_lse(a, row0 + head, top, sum);
            }
        }
    }
    if (warp == 0) {
        // the unit that goes on behind the CTA, if one does: its first row of out, in how
        // many CTAs it has pieces, and its heads
        if (goes_on) {
            const int row0 = sh.row[lane];
            a.tails[blockIdx.x] = make_int4(
                row0, (sh.end[lane] - 1) / per_cta - static_cast<int>(blockIdx.x) + 1,
                min(S::kHeads, a.group - row0 % a.group), 0);
        } else if (lane == 0 && open_ones == 0) {
            a.tails[blockIdx.x] = make_int4(-1, 0, 0, 0);
        }
    }
}

// The units that span CTAs, a CTA per query head: the pieces' sum weighted by their maxima,
// dealt out to the warps in turn.  BY_UNIT, where there are fewer units than CTAs of the
// first kernel: blockIdx.x is a unit, whose CTAs are found from the lengths while the first
// kernel's last CTAs still run.  Otherwise it is a CTA of the first kernel, which has left a
// note of the unit that it began and did not end.  (1 x 131072, two units of 76 CTAs: 31.0
// us with the notes, 28.6 by unit.)
constexpr int kJoinWarps = 16, kFewJoinWarps = 4;

template <int D, int NT, bool BY_UNIT, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, WARPS == kJoinWarps ? 1 : 8)
    paged_join_kernel(const __grid_constant__ AttnArgs a) {
    using S = AttnShape<D, NT>;
    static_assert(32 * WARPS >= D, "a thread per dimension");
    __shared__ float acc_sh[WARPS][D], top_sh[WARPS], sum_sh[WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, head = blockIdx.y;
    int first = blockIdx.x;  // CTA that began the unit
    int row0 = -1, parts = 0, heads = 0;  // the unit's first row of out, its CTAs, its heads
    if constexpr (BY_UNIT) {
        // (no newer than this kernel: the first one had waited for what was before it when it
        // let this one come)
        auto blocks_of = [&](int i) {
            return blocks_in(max(0, min(__ldcg(a.lengths + i), a.width * a.split.size)));
        };
        const int b = blockIdx.x / a.units, unit = blockIdx.x % a.units;
        int total = 0, before = 0;
        for (int i = lane; i < a.seqs; i += 32) {
            const int blocks = blocks_of(i);
            total += blocks;
            before += i < b ? blocks : 0;
        }
        const int mine = blocks_of(b);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            total += __shfl_xor_sync(kFullMask, total, o);
            before += __shfl_xor_sync(kFullMask, before, o);
        }
        const int per_cta = (total * a.units + a.ctas - 1) / a.ctas;
        const int begin = before * a.units + unit * mine;
        if (mine > 0) {
            first = begin / per_cta;
            parts = (begin + mine - 1) / per_cta - first + 1;
        }
        const int chunk = unit % a.chunks * S::kHeads;
        heads = min(S::kHeads, a.group - chunk);
        if (parts > 1) row0 = (b * a.kv_heads + unit / a.chunks) * a.group + chunk;
    }
    wait_before();
    let_next();
    // the first piece is the second one of the CTA that began the unit
    auto piece = [&](int i) {
        return a.parts + (2 * (static_cast<int64_t>(first) + i) + (i == 0)) * S::kPiece;
    };
    // A lane has the maximum and the sum of one piece, asked for before it is known how many
    // there are (what is no piece is not used).
    const int most = BY_UNIT ? parts : min(32 * WARPS, static_cast<int>(gridDim.x) - first);
    int mine = warp + lane * WARPS;
    float m = -INFINITY, l = 0.f;
    if (mine < most) m = piece(mine)[S::kM + head], l = piece(mine)[S::kL + head];
    if constexpr (!BY_UNIT) {
        const int4 tail = a.tails[blockIdx.x];  // (row of out, CTAs, heads)
        row0 = tail.x, parts = tail.y, heads = tail.z;
    }
    if (row0 < 0 || head >= heads) return;
    float top = -INFINITY, sum = 0.f, acc[D / 32] = {};
    for (int i0 = warp; i0 < parts; i0 += 32 * WARPS, mine += 32 * WARPS) {
        if (i0 > warp && mine < parts) m = piece(mine)[S::kM + head], l = piece(mine)[S::kL + head];
        if (mine >= parts) m = -INFINITY, l = 0.f;
        float to = fmaxf(top, m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) to = fmaxf(to, __shfl_xor_sync(kFullMask, to, o));
        const float f0 = piece_weight(top, to), f = piece_weight(m, to);
        top = to;
        sum *= f0;
#pragma unroll
        for (int x = 0; x < D / 32; ++x) acc[x] *= f0;
        const int here = min(32, (parts - i0 + WARPS - 1) / WARPS);
#pragma unroll 4
        for (int i = 0; i < here; ++i) {
            const float w = __shfl_sync(kFullMask, f, i);
            sum += w * __shfl_sync(kFullMask, l, i);
            const float* from = piece(i0 + i * WARPS) + head * S::kHeadStride + lane * (D / 32);
#pragma unroll
            for (int x = 0; x < D / 32; ++x) acc[x] += w * from[x];
        }
    }
#pragma unroll
    for (int x = 0; x < D / 32; ++x) acc_sh[warp][lane * (D / 32) + x] = acc[x];
    if (lane == 0) top_sh[warp] = top, sum_sh[warp] = sum;
    __syncthreads();
    const int d = threadIdx.x;
    if (d >= D) return;
    top = -INFINITY;
    for (int w = 0; w < WARPS; ++w) top = fmaxf(top, top_sh[w]);
    float all = 0.f, value = 0.f;
    for (int w = 0; w < WARPS; ++w) {
        const float f = piece_weight(top_sh[w], top);
        all += f * sum_sh[w];
        value += f * acc_sh[w][d];
    }
    const int row = row0 + head;
    a.out[static_cast<int64_t>(row) * D + d] = __float2bfloat16(all == 0.f ? 0.f : value / all);
    if (d == 0) store_lse(a, row, top, all);
}

}  // namespace paged
}  // namespace os
