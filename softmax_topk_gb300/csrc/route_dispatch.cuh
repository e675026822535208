// route_dispatch.cuh -- router over experts: the choice of kernel variant and the
// launches, per dtype (route_f32.cu, route_bf16.cu).
#pragma once

#include "host_common.h"
#include "internal.h"
#include "kernels/route_kernel.cuh"

namespace os {
namespace {

using route::Shape;

constexpr int64_t kListRowsPerSm = 16;

// Lanes per group: the largest power of two that still gives every group its
// own lanes; experts per lane follow.
inline Shape make_shape(const RouteArgs& a, int groups) {
    Shape s = {};
    s.experts = a.experts;
    s.K = a.K;
    s.groups = groups;
    s.topk_groups = a.topk_groups;
    s.group_top = a.group_top;
    s.lanes = 1;
    while (s.lanes * 2 * groups <= 32) {
        s.lanes *= 2;
        ++s.lanes_log2;
    }
    s.per_lane = (a.experts / groups + s.lanes - 1) / s.lanes;
    s.index_mask = pow2_at_least(a.experts) - 1;
    s.slots = pow2_at_least(a.K);
    s.tokens = 1;
    s.sigmoid = a.score == OS_SCORE_SIGMOID;
    s.renorm = a.renorm;
    s.scale = a.scale;
    return s;
}

// Whole vectors: every lane that has experts has a full run, which starts on a
// boundary of its own size (at most 16 bytes).
inline bool whole_runs(const Shape& s, int N, int size, const void* p, const void* q) {
    const int bytes = N * size < 16 ? N * size : 16;
    return s.per_lane == N && s.experts == s.groups * s.lanes * N &&
           reinterpret_cast<uintptr_t>(p) % bytes == 0 && reinterpret_cast<uintptr_t>(q) % bytes == 0;
}

inline int64_t grid_for(int64_t rows, int tokens) {
    return min64(ceil_div(rows, int64_t(route::kWarps) * tokens), int64_t(1) << 22);
}

// Rows per warp: one while the GPU has warps to spare (the latency of one
// row), else several, which share the work after the choice (65536 rows, us with
// one / by this rule: 64 experts 43 / 23, 128 experts 47 / 29, their gradients
// 25 / 9 and 24 / 11).
inline bool share_rows(const RouteArgs& a, Shape& s) {
    const DeviceInfo* dev = device_info();
    if (!dev) return false;
    while (s.tokens * 2 * s.slots <= 32 && a.rows >= int64_t(dev->sms) * 32 * s.tokens * 2)
        s.tokens *= 2;
    return true;
}

template <typename T, int N>
cudaError_t launch_fwd(const RouteArgs& a, Shape s, float* weights, int32_t* idx,
                       cudaStream_t stream) {
    if (!share_rows(a, s)) return cudaErrorInvalidDevice;
    auto k = route::route_kernel<T, N, false>;
    if constexpr (N <= 32)  // groups of 33 to 64 experts to a lane never fill it
        if (whole_runs(s, N, sizeof(T), a.x, a.x)) k = route::route_kernel<T, N, true>;
    return launch_kernel(k, grid_for(a.rows, s.tokens), route::kWarps * 32, 1, 0, stream,
                         static_cast<const T*>(a.x), a.bias, weights, reinterpret_cast<int*>(idx),
                         a.rows, s);
}

template <typename T, int N>
cudaError_t launch_bwd(const RouteArgs& a, Shape s, const int32_t* idx,
                       const float* dweights, void* dx, cudaStream_t stream) {
    if (!share_rows(a, s)) return cudaErrorInvalidDevice;
    auto k = whole_runs(s, N, sizeof(T), a.x, dx) ? route::route_bwd_kernel<T, N, true>
                                                  : route::route_bwd_kernel<T, N, false>;
    return launch_kernel(k, grid_for(a.rows, s.tokens), route::kWarps * 32, 1, 0, stream,
                         static_cast<const T*>(a.x), reinterpret_cast<const int*>(idx), dweights,
                         static_cast<T*>(dx), a.rows, s);
}

// The kernel of four threads per row: rows and groups of whole 16-byte chunks
// (rows of eight of them, for the copy's placement), lists and choose_exact's
// runs that fit, enough rows, and enough experts for the lists to pay (65536
// rows, us, one warp / four threads per row: 64 experts 15.5 / 19.2, 128 with
// a bias 27 / 29, 256 with a bias and groups 76 / 52, 512 with a bias 160 / 127).
template <typename T>
bool list_fits(const RouteArgs& a, const Shape& s, int sms) {
    const int bytes = a.experts * int(sizeof(T));
    return a.K <= 16 && a.experts >= 256 && a.experts <= route::kListExperts && bytes % 128 == 0 &&
           a.experts / a.groups * int(sizeof(T)) % 16 == 0 && s.per_lane <= 32 &&
           reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.rows >= int64_t(sms) * kListRowsPerSm;
}

template <typename T, int P>
cudaError_t launch_list(const RouteArgs& a, const Shape& s, float* w, int32_t* idx, int sms,
                        cudaStream_t stream) {
    auto k = s.per_lane <= 8 ? route::route_list_kernel<T, P, 8> : route::route_list_kernel<T, P, 32>;
    constexpr int kRows = route::kListWarps * route::kListRows;
    const int smem = route::list_head(a.experts, a.groups) + kRows * a.experts * int(sizeof(T));
    const int per_sm = blocks_per_sm(k, route::kListWarps * 32, smem);
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    const int64_t grid = min64(ceil_div(a.rows, kRows), int64_t(sms) * per_sm);
    return launch_kernel(k, grid, route::kListWarps * 32, 1, smem, stream,
                         static_cast<const T*>(a.x), a.bias, w, reinterpret_cast<int*>(idx), a.rows, s);
}

template <typename T>
cudaError_t fwd(const RouteArgs& a, float* w, int32_t* idx, cudaStream_t stream) {
    const Shape s = make_shape(a, a.groups);
    const DeviceInfo* dev = device_info();
    if (!dev) return cudaErrorInvalidDevice;
    if (list_fits<T>(a, s, dev->sms)) {
        if (a.K <= 4) return launch_list<T, 4>(a, s, w, idx, dev->sms, stream);
        if (a.K <= 8) return launch_list<T, 8>(a, s, w, idx, dev->sms, stream);
        return launch_list<T, 16>(a, s, w, idx, dev->sms, stream);
    }
    if (s.per_lane <= 1) return launch_fwd<T, 1>(a, s, w, idx, stream);
    if (s.per_lane <= 2) return launch_fwd<T, 2>(a, s, w, idx, stream);
    if (s.per_lane <= 4) return launch_fwd<T, 4>(a, s, w, idx, stream);
    if (s.per_lane <= 8) return launch_fwd<T, 8>(a, s, w, idx, stream);
    if (s.per_lane <= 16) return launch_fwd<T, 16>(a, s, w, idx, stream);
    if (s.per_lane <= 32) return launch_fwd<T, 32>(a, s, w, idx, stream);
    return launch_fwd<T, 64>(a, s, w, idx, stream);  // 3, 5-7, 9-15 or 17-31 groups
}

template <typename T>
cudaError_t bwd(const RouteArgs& a, const int32_t* idx, const float* dw, void* dx,
                cudaStream_t stream) {
    const Shape s = make_shape(a, 1);
    if (s.per_lane <= 1) return launch_bwd<T, 1>(a, s, idx, dw, dx, stream);
    if (s.per_lane <= 2) return launch_bwd<T, 2>(a, s, idx, dw, dx, stream);
    if (s.per_lane <= 4) return launch_bwd<T, 4>(a, s, idx, dw, dx, stream);
    if (s.per_lane <= 8) return launch_bwd<T, 8>(a, s, idx, dw, dx, stream);
    if (s.per_lane <= 16) return launch_bwd<T, 16>(a, s, idx, dw, dx, stream);
    return launch_bwd<T, 32>(a, s, idx, dw, dx, stream);
}

}  // namespace
}  // namespace os
