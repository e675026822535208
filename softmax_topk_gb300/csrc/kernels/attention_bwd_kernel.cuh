// attention_bwd_kernel.cuh -- gradient of the attention forward on the
// fifth-generation tensor cores.
//
// With S = scale Q K^T, P = e^(S - L) (L the forward's logsumexp, so P is the
// softmax itself, recomputed instead of stored), and the row constants
// delta_i = dO_i . O_i - dL_i:
//   dV = P^T dO,   dP = dO V^T,   dS = P o (dP - delta),
//   dQ = scale dS K,   dK = scale dS^T Q.
// Two walks, one per side that a sum runs over, so that every output row is
// summed by one CTA in a fixed order (no atomics, results do not depend on
// scheduling):
//   KV = true:  one item is a tile of 128 keys; it keeps K and V of those rows
//               and streams the tiles of (Q, dO), accumulating dK and dV;
//   KV = false: one item is a tile of 128 queries; it keeps Q and dO and
//               streams the tiles of (K, V), accumulating dQ.
// Both are the same program on swapped operands: with (X, Y) the resident pair
// and (U, W) the streamed one, per tile
//   A1 = X U^T  (S or its transpose),  A2 = Y W^T  (dP or its transpose),
//   P and dS from A1 and A2 element by element,
//   acc1 += dS U  (dK or dQ),  acc2 += P W  (dV, KV only).
// The price of the split is that S and dP are formed twice: seven products
// instead of five.
//
// GB300 mapping (persistent CTAs, one per SM, warp-specialised):
//   * load warp: TMA tiled loads of the resident pair once per item and of the
//     streamed pairs through a ring of stages;
//   * issuing warps (one lane each): the products, accumulators in tensor
//     memory.  One warp issues A1 and A2, another the sums (without KV A1, A2
//     and the sum have a warp each): an issuer needs some 300 cycles between
//     two products for its waits and commits, which one alone left the tensor
//     pipe idle for (57 % busy), and the other's product fills.  A product that
//     overwrites what an earlier one reads is issued after that one's
//     completion was seen;
//   * stat warp (KV only): the streamed rows' -L log2e and -delta into shared
//     memory, L = +inf for rows past the end so that their P is 0;
//   * eight compute warps: thread (r, h) owns tile row r (one tensor-memory
//     lane) and half h of its columns: P = 2^(A1 scale log2e - L log2e) to
//     bf16 for the dV product, dS = P (A2 - delta) to bf16 for the dK / dQ
//     product (both read from tensor memory as the A operand), fp32 in between.
//     The two roundings to bf16 are the price of the bf16 tensor cores, as P's
//     is in the forward; sums are fp32.
//
// Tensor memory (512 columns).  With KV and D = 128 the two sums take 256
// columns, so A1 and A2 take turns in one buffer of 128, and P and dS share
// another.  A1 and A2 are read into registers as soon as they are complete, and
// the sums run between them: A1(g), dS(g-1) U, A2(g), P(g) W, A1(g+1), ...
// Otherwise A1 and A2 have buffers of their own (d = 64, 16 x 16384 causal: 1851
// us with a shared one), and without KV dS has two.
//
// What bounds it (64 x 4096, 1.37 TFLOP of the five products): d = 128 1177 us,
// 1168 TFLOP/s, or 1632 with the two products that are formed twice, 0.84 of the
// measured bf16 rate: the tensor pipe, which is busy 2048 of ~2700 cycles of a key
// tile and 1536 of ~1740 of a query tile.  d = 64 (0.69 TFLOP) 899 us: the compute
// warps' chain per tile, for a product takes half as long for as many scores.
// Under the mask 700 us at d = 128, and 16 x 16384 at d = 64 1768 us.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include <cstdint>

#include "../ctl.h"
#include "attention_kernel.cuh"
#include "ops.cuh"
#include "umma.cuh"

namespace os {
namespace attn_bwd {

constexpr int kRows = 128;          // rows of a tile, resident or streamed
constexpr int kComputeWarps = 8;
constexpr int kCompute = kComputeWarps * 32;
constexpr int kLoadWarp = 8;
constexpr int kMmaWarp = 9;    // A1; with KV A2 too
constexpr int kSumWarp = 10;   // the sums
constexpr int kStatWarp = 11;  // KV: the statistics; else A2
constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;
// Tensor memory columns.  bf16 operands (P, dS) take 32 columns for tile
// columns 0-63 and 32 for 64-127, 64 apart.
template <int D, bool KV>
struct Tmem {
    static constexpr bool kShared = KV && D == 128;   // A1 and A2 in one buffer
    static constexpr uint32_t kA1 = 0;                // fp32, 128 columns
    static constexpr uint32_t kA2 = kShared ? 0 : 128;
    static constexpr uint32_t kP = kShared ? 128 : 256;   // KV
    static constexpr uint32_t kDs = KV ? kP + 32 : 384;   // tile g at kDs + 32 (g % kDsBuffers)
    static constexpr int kDsBuffers = KV ? 1 : 2;
    static constexpr uint32_t kAcc1 = kShared || !KV ? 256 : 384;  // dK or dQ, D columns
    static constexpr uint32_t kAcc2 = kShared ? 384 : 448;         // dV, D columns (KV)
};
constexpr float kLog2e = 1.442695041f;

// One stage more for U than for W: U of a tile is read twice, by its first and
// its last product, W is done with earlier.  At D = 128 that fills the SM's
// shared memory to the last kilobyte, so the barriers live in it too.
template <int D>
struct Layout {
    static constexpr int kUStages = D == 128 ? 3 : 4;
    static constexpr int kWStages = D == 128 ? 2 : 4;
    static constexpr int kBlock = kRows * 64 * 2;  // 16 KB: 128 rows of 64 bf16
    static constexpr int kTile = kRows * D * 2;
    static constexpr int kX = 0;
    static constexpr int kY = kX + kTile;
    static constexpr int kU = kY + kTile;               // kUStages buffers
    static constexpr int kW = kU + kUStages * kTile;    // kWStages buffers
    static constexpr int kStat = kW + kWStages * kTile;  // 2 x (128 -L log2e, 128 -delta)
    static constexpr int kBars = kStat + 2 * 2 * kRows * 4;
    static constexpr int kBytes = kBars + 512;
};

template <int D>
struct Barriers {
    using L = Layout<D>;
    uint64_t x_full, x_empty;                      // resident pair landed / its products done
    uint64_t u_full[L::kUStages], u_empty[L::kUStages];  // streamed tile landed / read
    uint64_t w_full[L::kWStages], w_empty[L::kWStages];
    uint64_t a1_full, a2_full;                     // A1 / A2 of a tile in tensor memory
    uint64_t a1_free, a2_free;                     // they are in registers (all compute threads)
    uint64_t p_full;                               // P in tensor memory (all compute threads)
    uint64_t ds_full[2];                           // dS likewise, one per buffer: a buffer is
                                                   // filled again only once its sum was issued
    uint64_t pw_done;                              // acc2 += P W completed
    uint64_t acc_done[2];                          // both sums of tile g (at g & 1) completed
    uint64_t acc_empty;                            // an item's sums are in registers
    uint64_t stat_full[2], stat_empty[2];          // the streamed rows' statistics there / read
    uint64_t drain;
    uint32_t tmem;
};

// Bounded waits of one role: once one gave up, the rest return at once, so a
// kernel whose data never comes ends after one timeout per role.
struct Waiter {
    const KernelCtl& ctl;
    bool ok;
    __device__ __forceinline__ explicit Waiter(const KernelCtl& c) : ctl(c), ok(true) {}
    __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
        if (ok) ok = umma::mbar_wait(bar, parity, ctl);
    }
};

// Tiles that item `tile` walks: all of them, or under the mask the queries at
// or after a key tile (KV) and the keys at or before a query tile.
template <bool KV>
__device__ __forceinline__ void tile_range(int tile, int nt, bool causal, int& first, int& count) {
    first = KV && causal ? tile : 0;
    count = !causal ? nt : (KV ? nt - tile : tile + 1);
}

// delta[i] = dO_i . O_i - dL_i, one group of D / 8 lanes per row, 16 bytes a lane.
template <int D>
__global__ void __launch_bounds__(256)
delta_kernel(const __nv_bfloat16* __restrict__ o, const __nv_bfloat16* __restrict__ dout,
             const float* __restrict__ dlse, float* __restrict__ delta, int64_t rows) {
    constexpr int G = D / 8;
    const int64_t row = (int64_t(blockIdx.x) * 256 + threadIdx.x) / G;
    const int part = threadIdx.x % G;
    float s = 0.f;
    if (row < rows) {
        const uint4 a = *reinterpret_cast<const uint4*>(o + row * D + part * 8);
        const uint4 b = *reinterpret_cast<const uint4*>(dout + row * D + part * 8);
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = unpack_bf16x2(aw[i]), y = unpack_bf16x2(bw[i]);
            s = fmaf(x.x, y.x, s);
            s = fmaf(x.y, y.y, s);
        }
    }
#pragma unroll
    for (int k = G / 2; k > 0; k >>= 1) s += __shfl_xor_sync(kFullMask, s, k);
    if (row < rows && part == 0) delta[row] = s - (dlse ? dlse[row] : 0.f);
}

// One side's arguments.
struct Side {
    CUtensorMap x, y, u, w;
    __nv_bfloat16 *out1, *out2;
};

// The program of one CTA: number `cta` of `ctas` that walk the side's units.
template <int D, bool KV>
__device__ __forceinline__ void bwd_cta(const CUtensorMap& map_x, const CUtensorMap& map_y,
                                        const CUtensorMap& map_u, const CUtensorMap& map_w,
                                        const float* __restrict__ lse,
                                        const float* __restrict__ delta,
                                        __nv_bfloat16* __restrict__ out1,
                                        __nv_bfloat16* __restrict__ out2, int n, int nt, int units,
                                        float scale, int causal_flag, const KernelCtl& ctl, int cta,
                                        int ctas) {
    using L = Layout<D>;
    using TM = Tmem<D, KV>;
    constexpr int US = L::kUStages, WS = L::kWStages;
    static_assert(sizeof(Barriers<D>) <= L::kBytes - L::kBars, "barriers");
    // no static shared memory: the dynamic part starts on a 1024-byte boundary
    extern __shared__ __align__(1024) unsigned char smem[];
    Barriers<D>& bars = *reinterpret_cast<Barriers<D>*>(smem + L::kBars);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool causal = causal_flag != 0;

    if (tid == 0) {
        mbar_init(&bars.x_full, 1);
        mbar_init(&bars.x_empty, KV ? 1 : 2);  // the issuers of A1 and A2
        for (int s = 0; s < US; ++s) {
            mbar_init(&bars.u_full[s], 1);
            mbar_init(&bars.u_empty[s], 1);
        }
        for (int s = 0; s < WS; ++s) {
            mbar_init(&bars.w_full[s], 1);
            mbar_init(&bars.w_empty[s], KV ? 2 : 1);  // A2, and with KV P W
        }
        mbar_init(&bars.a1_full, 1);
        mbar_init(&bars.a2_full, 1);
        mbar_init(&bars.p_full, kCompute);
        mbar_init(&bars.ds_full[0], kCompute);
        mbar_init(&bars.ds_full[1], kCompute);
        mbar_init(&bars.a1_free, kCompute);
        mbar_init(&bars.a2_free, kCompute);
        mbar_init(&bars.pw_done, 1);
        mbar_init(&bars.acc_done[0], 1);
        mbar_init(&bars.acc_done[1], 1);
        mbar_init(&bars.acc_empty, kCompute);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars.stat_full[s], 32);
            mbar_init(&bars.stat_empty[s], kComputeWarps);
        }
        mbar_init(&bars.drain, KV ? 2 : 3);  // every issuer
        mbar_init_fence();
    }
    if (warp == 0) umma::tmem_alloc(&bars.tmem, kTmemCols);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = bars.tmem;

    // Every role walks the same items in the same order (work units as in the
    // forward: single tiles, or balanced pairs under the mask); g counts the
    // streamed tiles and it the items across the whole walk, and give the
    // barriers' phases.
    if (warp == kLoadWarp) {
        if (lane == 0) {
            umma::prefetch_tensormap(&map_x);
            umma::prefetch_tensormap(&map_y);
            umma::prefetch_tensormap(&map_u);
            umma::prefetch_tensormap(&map_w);
            Waiter wait(ctl);
            int g = 0, nu = 0, it = 0;  // tiles of W and of U, items so far
            for (int u = cta; u < units && wait.ok; u += ctas) {
                int bh, ta, tb;
                const int cnt = attn::work_unit(u, nt, causal, bh, ta, tb);
                for (int e = 0; e < cnt && wait.ok; ++e) {
                    const int tile = e == 0 ? ta : tb;
                    int first, count;
                    tile_range<KV>(tile, nt, causal, first, count);
                    if (it > 0) wait(&bars.x_empty, (it - 1) & 1);
                    if (!wait.ok) break;
                    mbar_arrive_expect_tx(&bars.x_full, 2 * L::kTile);
                    ++it;
#pragma unroll
                    for (int blk = 0; blk < D / 64; ++blk) {
                        umma::tma_load_3d(smem + L::kX + blk * L::kBlock, &map_x, 64 * blk,
                                          tile * kRows, bh, &bars.x_full);
                        umma::tma_load_3d(smem + L::kY + blk * L::kBlock, &map_y, 64 * blk,
                                          tile * kRows, bh, &bars.x_full);
                    }
                    for (int j = 0; j < count; ++j) {
                        const int us = g % US, ws = g % WS;
                        if (g >= US) wait(&bars.u_empty[us], (g / US - 1) & 1);
                        if (!wait.ok) break;
                        mbar_arrive_expect_tx(&bars.u_full[us], L::kTile);
#pragma unroll
                        for (int blk = 0; blk < D / 64; ++blk)
                            umma::tma_load_3d(smem + L::kU + us * L::kTile + blk * L::kBlock,
                                              &map_u, 64 * blk, (first + j) * kRows, bh,
                                              &bars.u_full[us]);
                        ++nu;
                        if (g >= WS) wait(&bars.w_empty[ws], (g / WS - 1) & 1);
                        if (!wait.ok) break;
                        mbar_arrive_expect_tx(&bars.w_full[ws], L::kTile);
#pragma unroll
                        for (int blk = 0; blk < D / 64; ++blk)
                            umma::tma_load_3d(smem + L::kW + ws * L::kTile + blk * L::kBlock,
                                              &map_w, 64 * blk, (first + j) * kRows, bh,
                                              &bars.w_full[ws]);
                        ++g;
                    }
                }
            }
            // no copy may land after this CTA has gone
            if (it > 0)
                mbar_wait_bounded_ns(&bars.x_full, (it - 1) & 1, kDrainTimeoutNs, ctl.err);
            for (int k = nu > US ? nu - US : 0; k < nu; ++k)
                mbar_wait_bounded_ns(&bars.u_full[k % US], (k / US) & 1, kDrainTimeoutNs, ctl.err);
            for (int k = g > WS ? g - WS : 0; k < g; ++k)
                mbar_wait_bounded_ns(&bars.w_full[k % WS], (k / WS) & 1, kDrainTimeoutNs, ctl.err);
        }
    } else if (warp == kMmaWarp || warp == kSumWarp || (!KV && warp == kStatWarp)) {
        if (lane == 0) {
            constexpr uint32_t id_a = umma::idesc_bf16(kRows, kRows, false);
            constexpr uint32_t id_acc = umma::idesc_bf16(kRows, D, true);
            // descriptors of the buffers' starts; an offset adds to the address field
            const uint64_t x_desc = umma::desc_sw128(smem_addr(smem + L::kX), 16, 1024);
            const uint64_t y_desc = umma::desc_sw128(smem_addr(smem + L::kY), 16, 1024);
            const uint64_t u_desc = umma::desc_sw128(smem_addr(smem + L::kU), 16, 1024);
            const uint64_t w_desc = umma::desc_sw128(smem_addr(smem + L::kW), 16, 1024);
            const uint64_t u_sum = umma::desc_sw128(smem_addr(smem + L::kU), L::kBlock, 1024);
            const uint64_t w_sum = umma::desc_sw128(smem_addr(smem + L::kW), L::kBlock, 1024);
            Waiter wait(ctl);
            // A (128 x 128 fp32) = resident tile times streamed tile transposed
            auto product = [&](uint32_t dst, uint64_t a, uint64_t b) {
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint32_t off = ((s >> 2) * L::kBlock + (s & 3) * 32) >> 4;
                    umma::mma_bf16(tmem + dst, a + off, b + off, id_a, s > 0);
                }
            };
            // acc (128 x D) += P or dS (tensor memory, tile columns 0-63 at
            // `src`, 64-127 at src + 64) times a streamed tile
            auto accumulate = [&](uint32_t dst, uint32_t src, uint64_t b, bool keep) {
#pragma unroll
                for (int s = 0; s < kRows / 16; ++s)
                    umma::mma_bf16_tmem_a(tmem + dst, tmem + src + (s < 4 ? 8 * s : 32 + 8 * s),
                                          b + ((s * 2048) >> 4), id_acc, keep || s > 0);
            };
            auto tile_at = [](uint64_t desc, int stage) {
                return desc + uint64_t(stage) * (L::kTile >> 4);
            };
            auto issue_a1 = [&](int g, bool last) {
                const int us = g % US;
                wait(&bars.u_full[us], (g / US) & 1);
                if (g > 0) wait(TM::kShared ? &bars.a2_free : &bars.a1_free, (g - 1) & 1);
                if (!wait.ok) return;
                umma::fence_after_sync();
                product(TM::kA1, x_desc, tile_at(u_desc, us));
                umma::commit(&bars.a1_full);
                if (!KV && last) umma::commit(&bars.x_empty);
            };
            auto issue_a2 = [&](int g, bool last) {
                const int ws = g % WS;
                wait(&bars.w_full[ws], (g / WS) & 1);
                if (TM::kShared) wait(&bars.a1_free, g & 1);
                else if (g > 0) wait(&bars.a2_free, (g - 1) & 1);
                if (!wait.ok) return;
                umma::fence_after_sync();
                product(TM::kA2, y_desc, tile_at(w_desc, ws));
                umma::commit(&bars.a2_full);
                umma::commit(&bars.w_empty[ws]);
                if (last) umma::commit(&bars.x_empty);  // the last reader of X and Y
            };
            // the item's first products (j == 0) overwrite the sums, which the
            // compute warps must have read
            auto issue_sums = [&](int g, int j, int it) {
                const int us = g % US, ws = g % WS;
                if (j == 0 && it > 0) wait(&bars.acc_empty, (it - 1) & 1);
                if (KV) {
                    wait(&bars.w_full[ws], (g / WS) & 1);  // P does not depend on W
                    wait(&bars.p_full, g & 1);
                    if (!wait.ok) return;
                    umma::fence_after_sync();
                    accumulate(TM::kAcc2, TM::kP, tile_at(w_sum, ws), j > 0);
                    if (D == 128) umma::commit(&bars.pw_done);
                    umma::commit(&bars.w_empty[ws]);
                }
                constexpr int B = TM::kDsBuffers;
                wait(&bars.ds_full[g % B], (g / B) & 1);  // U(g): dS was made from its product
                if (!wait.ok) return;
                umma::fence_after_sync();
                accumulate(TM::kAcc1, TM::kDs + 32 * (g % B), tile_at(u_sum, us), j > 0);
                umma::commit(&bars.acc_done[g & 1]);
                umma::commit(&bars.u_empty[us]);
            };
            int g = 0, it = 0;
            for (int u = cta; u < units && wait.ok; u += ctas) {
                int bh, ta, tb;
                const int cnt = attn::work_unit(u, nt, causal, bh, ta, tb);
                for (int e = 0; e < cnt && wait.ok; ++e, ++it) {
                    int first, count;
                    tile_range<KV>(e == 0 ? ta : tb, nt, causal, first, count);
                    if (warp != kSumWarp) wait(&bars.x_full, it & 1);
                    for (int j = 0; j < count && wait.ok; ++j, ++g) {
                        const bool last = j + 1 == count;
                        if (warp == kSumWarp) issue_sums(g, j, it);
                        else if (warp == kMmaWarp) issue_a1(g, last);
                        if (KV ? warp == kMmaWarp : warp == kStatWarp) issue_a2(g, last);
                    }
                }
            }
            // no product may be in flight when tensor memory is given back
            umma::commit(&bars.drain);
            mbar_wait_bounded_ns(&bars.drain, 0, kDrainTimeoutNs, ctl.err);
        }
    } else if (warp == kStatWarp) {
        if (KV) {
            Waiter wait(ctl);
            int g = 0;
            for (int u = cta; u < units; u += ctas) {
                int bh, ta, tb;
                const int cnt = attn::work_unit(u, nt, causal, bh, ta, tb);
                for (int e = 0; e < cnt; ++e) {
                    int first, count;
                    tile_range<KV>(e == 0 ? ta : tb, nt, causal, first, count);
                    const float* lrow = lse + int64_t(bh) * n;
                    const float* drow = delta + int64_t(bh) * n;
                    for (int j = 0; j < count; ++j, ++g) {
                        const int base = (first + j) * kRows;
                        float lv[4], dv[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int q = base + lane + 32 * i;
                            lv[i] = q < n ? -lrow[q] * kLog2e : -INFINITY;
                            dv[i] = q < n ? -drow[q] : 0.f;
                            // L = -inf, a row without keys: P is 0, and so is
                            // delta, which may be NaN or infinite there
                            if (lv[i] == INFINITY) lv[i] = -INFINITY, dv[i] = 0.f;
                        }
                        // buffer g & 1 was last read for tile g - 2
                        if (g >= 2) wait(&bars.stat_empty[g & 1], ((g - 2) >> 1) & 1);
                        float* stat = reinterpret_cast<float*>(smem + L::kStat) + (g & 1) * 2 * kRows;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            stat[lane + 32 * i] = lv[i];
                            stat[kRows + lane + 32 * i] = dv[i];
                        }
                        umma::mbar_arrive(&bars.stat_full[g & 1]);
                    }
                }
            }
        }
    } else {
        // ---------------------------------------------------------------- compute
        const int r = tid & 127, half = tid >> 7;  // tile row, column half
        const uint32_t lane_addr = tmem + (uint32_t((warp & 3) * 32) << 16);
        const uint32_t a1 = lane_addr + TM::kA1 + 64 * half, a2 = lane_addr + TM::kA2 + 64 * half;
        const float scale_log2 = scale * kLog2e;
        Waiter wait(ctl);
        int g = 0;
        for (int u = cta; u < units; u += ctas) {
            int bh, ta, tb;
            const int cnt = attn::work_unit(u, nt, causal, bh, ta, tb);
            for (int e = 0; e < cnt; ++e) {
                const int tile = e == 0 ? ta : tb;
                int first, count;
                tile_range<KV>(tile, nt, causal, first, count);
                const int row = tile * kRows + r;
                float row_l = -INFINITY, row_delta = 0.f;  // negated
                if (!KV && row < n) {
                    row_l = -lse[int64_t(bh) * n + row] * kLog2e;
                    row_delta = -delta[int64_t(bh) * n + row];
                    if (row_l == INFINITY) row_l = -INFINITY, row_delta = 0.f;
                }
                for (int j = 0; j < count; ++j, ++g) {
                    const int col0 = (first + j) * kRows + 64 * half;
                    const float* stat =
                        reinterpret_cast<const float*>(smem + L::kStat) + (g & 1) * 2 * kRows + 64 * half;
                    float p[64];
                    wait(&bars.a1_full, g & 1);
                    umma::fence_after_sync();
                    umma::tmem_ld32(a1, p);
                    umma::tmem_ld32(a1 + 32, p + 32);
                    if (KV) wait(&bars.stat_full[g & 1], (g >> 1) & 1);
                    umma::tmem_wait_ld();
                    umma::fence_before_sync();
                    umma::mbar_arrive(&bars.a1_free);
                    float dp[64];
                    constexpr bool kEarly = !KV && D == 64;
                    if (kEarly) {
                        // A2 is there by now, and its load passes under the
                        // exponentials
                        wait(&bars.a2_full, g & 1);
                        umma::fence_after_sync();
                        umma::tmem_ld32(a2, dp);
                        umma::tmem_ld32(a2 + 32, dp + 32);
                    }
                    // columns [lo, hi) of this half take part: keys up to the
                    // end and the query (KV = false), queries from the key on
                    // (KV = true; queries past the end have L = +inf)
                    int lo = 0, hi = 64;
                    if (KV) {
                        if (causal) lo = row - col0;
                    } else {
                        hi = n - col0;
                        if (causal) hi = min(hi, row - col0 + 1);
                    }
#pragma unroll
                    for (int c = 0; c < 64; c += 4) {
                        float4 l4;
                        if (KV) l4 = *reinterpret_cast<const float4*>(stat + c);
                        else l4 = make_float4(row_l, row_l, row_l, row_l);
                        const float2 za = fma2(make_float2(p[c], p[c + 1]), splat2(scale_log2),
                                               make_float2(l4.x, l4.y));
                        const float2 zb = fma2(make_float2(p[c + 2], p[c + 3]), splat2(scale_log2),
                                               make_float2(l4.z, l4.w));
                        p[c] = ex2_sfu(za.x);
                        p[c + 1] = ex2_sfu(za.y);
                        p[c + 2] = ex2_sfu(zb.x);
                        p[c + 3] = ex2_sfu(zb.y);
                    }
                    if (lo > 0 || hi < 64) {
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            if (c < lo || c >= hi) p[c] = 0.f;
                    }

                    if (KV) {
                        uint32_t pk[32];
#pragma unroll
                        for (int c = 0; c < 32; ++c) pk[c] = pack_bf16x2(p[2 * c], p[2 * c + 1]);
                        // P's last reader: P W of tile g - 1.  At d = 64 dS U of
                        // that tile is done by now too and its barrier serves
                        // both; at d = 128 it would hold P up (1195 -> 1303 us)
                        if (g > 0) {
                            if (D == 128) wait(&bars.pw_done, (g - 1) & 1);
                            else wait(&bars.acc_done[(g - 1) & 1], ((g - 1) >> 1) & 1);
                        }
                        umma::fence_after_sync();
                        umma::tmem_st32(lane_addr + TM::kP + 64 * half,
                                        reinterpret_cast<const float*>(pk));
                        umma::tmem_wait_st();
                        umma::fence_before_sync();
                        umma::mbar_arrive(&bars.p_full);
                    }

                    if (!kEarly) {
                        wait(&bars.a2_full, g & 1);
                        umma::fence_after_sync();
                        umma::tmem_ld32(a2, dp);
                        umma::tmem_ld32(a2 + 32, dp + 32);
                    }
                    umma::tmem_wait_ld();
                    // (nothing that uses dp moves above the wait)
#pragma unroll
                    for (int c = 0; c < 64; ++c) asm volatile("" : "+f"(dp[c]));
                    umma::fence_before_sync();
                    umma::mbar_arrive(&bars.a2_free);
                    uint32_t ds[32];
#pragma unroll
                    for (int c0 = 0; c0 < 64; c0 += 16) {
                        float4 d4[4];  // four loads ahead of their use
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            d4[i] = KV ? *reinterpret_cast<const float4*>(stat + kRows + c0 + 4 * i)
                                       : make_float4(row_delta, row_delta, row_delta, row_delta);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int c = c0 + 4 * i;
                            const float2 a = mul2(make_float2(p[c], p[c + 1]),
                                                  add2(make_float2(dp[c], dp[c + 1]),
                                                       make_float2(d4[i].x, d4[i].y)));
                            const float2 b = mul2(make_float2(p[c + 2], p[c + 3]),
                                                  add2(make_float2(dp[c + 2], dp[c + 3]),
                                                       make_float2(d4[i].z, d4[i].w)));
                            ds[c / 2] = pack_bf16x2(a.x, a.y);
                            ds[c / 2 + 1] = pack_bf16x2(b.x, b.y);
                        }
                    }
                    // the buffer's last reader: the sum of tile g - kDsBuffers
                    constexpr int lag = TM::kDsBuffers;
                    if ((!KV || D == 128) && g >= lag) {
                        wait(&bars.acc_done[(g - lag) & 1], ((g - lag) >> 1) & 1);
                        umma::fence_after_sync();
                    }
                    umma::tmem_st32(lane_addr + TM::kDs + 32 * (g % lag) + 64 * half,
                                    reinterpret_cast<const float*>(ds));
                    umma::tmem_wait_st();
                    umma::fence_before_sync();
                    umma::mbar_arrive(&bars.ds_full[g % lag]);
                    if (KV) {
                        __syncwarp();
                        if (lane == 0) umma::mbar_arrive(&bars.stat_empty[g & 1]);
                    }
                }
                // the item's sums: complete with the last tile's
                wait(&bars.acc_done[(g - 1) & 1], ((g - 1) >> 1) & 1);
                umma::fence_after_sync();
                constexpr int H = D / 2;  // columns per thread
                float o1[H], o2[KV ? H : 1];
#pragma unroll
                for (int c = 0; c < H / 32; ++c) {
                    umma::tmem_ld32(lane_addr + TM::kAcc1 + half * H + 32 * c, o1 + 32 * c);
                    if constexpr (KV)
                        umma::tmem_ld32(lane_addr + TM::kAcc2 + half * H + 32 * c, o2 + 32 * c);
                }
                umma::tmem_wait_ld();
                umma::fence_before_sync();
                umma::mbar_arrive(&bars.acc_empty);
                if (row < n && wait.ok) {
                    const int64_t at = (int64_t(bh) * n + row) * D + half * H;
#pragma unroll
                    for (int v = 0; v < H / 8; ++v) {
                        uint4 w;
                        w.x = pack_bf16x2(o1[8 * v + 0] * scale, o1[8 * v + 1] * scale);
                        w.y = pack_bf16x2(o1[8 * v + 2] * scale, o1[8 * v + 3] * scale);
                        w.z = pack_bf16x2(o1[8 * v + 4] * scale, o1[8 * v + 5] * scale);
                        w.w = pack_bf16x2(o1[8 * v + 6] * scale, o1[8 * v + 7] * scale);
                        *reinterpret_cast<uint4*>(out1 + at + 8 * v) = w;
                        if constexpr (KV) {
                            w.x = pack_bf16x2(o2[8 * v + 0], o2[8 * v + 1]);
                            w.y = pack_bf16x2(o2[8 * v + 2], o2[8 * v + 3]);
                            w.z = pack_bf16x2(o2[8 * v + 4], o2[8 * v + 5]);
                            w.w = pack_bf16x2(o2[8 * v + 6], o2[8 * v + 7]);
                            *reinterpret_cast<uint4*>(out2 + at + 8 * v) = w;
                        }
                    }
                }
            }
        }
    }

    umma::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        umma::fence_after_sync();
        umma::tmem_dealloc(tmem, kTmemCols);
    }
}

// Both sides in one launch: the first half of the CTAs takes keys, the second
// queries.  They need nothing of each other, and no more than one CTA fits an SM, so
// a CTA of the second half starts where one of the first has ended, or at once on
// an SM that the first half leaves free (64 x 4096, d = 128: 1196 us with a launch
// per side, d = 64 938; one launch less counts at 2 x 300 too, 28 -> 24 us a call).
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attention_bwd_kernel(const __grid_constant__ Side kv, const __grid_constant__ Side q,
                     const float* __restrict__ lse, const float* __restrict__ delta, int n, int nt,
                     int units, float scale, int causal, KernelCtl ctl) {
    const int ctas = gridDim.x / 2, cta = blockIdx.x;
    if (cta < ctas)
        bwd_cta<D, true>(kv.x, kv.y, kv.u, kv.w, lse, delta, kv.out1, kv.out2, n, nt, units, scale,
                         causal, ctl, cta, ctas);
    else
        bwd_cta<D, false>(q.x, q.y, q.u, q.w, lse, delta, q.out1, q.out2, n, nt, units, scale,
                          causal, ctl, cta - ctas, ctas);
}

}  // namespace attn_bwd
}  // namespace os
