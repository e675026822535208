// route_dispatch.cuh -- router over experts: the choice of kernel variant and the
// launches, per dtype (route_f32.cu, route_bf16.cu).
#pragma once

#include "host_common.h"
#include "internal.h"
#include "kernels/route_kernel.cuh"

namespace os {
namespace {

using route::Shape;

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
// row), else several, which share the work after the choice.  fp32, softmax, us
// with one / by this rule, choice and gradient (inputs past L2 at 65536 rows; at
// most 4864 rows have one either way):
//   rows          9728               19456              65536
//   64, K 6       7.7/6.4  6.0/3.9   14.1/9.2  9.3/4.1  45.6/24.1 27.3/10.0
//   128, K 8      8.4/7.6  6.5/4.9   14.7/11.7 10.1/7.4 46.6/31.2 27.1/17.5
//   512, K 16     32.1/29.7 9.4/8.3  59/52.2   15.7/14.2  185/159   48/40
// (From a quarter as many rows on, 64 experts take 5.3 us instead of 6.4 at 9728
// rows, and 60 of bf16 7.5 instead of 5.9.)
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

// Rows per SM from which the kernel of four threads per row is faster than the
// warps' (INT64_MAX: never).  Sigmoid scores take the most instructions and near
// ones are settled in the thread, the orders of logits least; a softmax's near
// scores go to choose_exact, a row of the tile after the other, and rows of 4 KB
// leave room for one CTA per SM.  Us, one warp / four threads per row, K = 8:
//   rows                           2432       4864       9728       19456      65536
//   sigmoid, bias       256 fp32   12.1/13.5  15.9/14.5  22.1/15.6  27.3/22.3  55.7/50.2
//                       512 fp32   20.3/17.6  27.2/17.8  34.7/21.6  48.2/35.8  115/86
//                      1024 fp32   41.1/26.0  59.7/29.5  75.7/53.9  105/97     281/257
//   and 8 groups        256 fp32   13.9/12.8  19.5/16.8  25.3/15.7  33.0/28.2  73.8/68.6
//   logits (softmax)    256 fp32    4.9/7.7    7.2/7.8   10.6/9.1   15.7/14.3  41.8/41.7
//                       512 fp32    8.9/10.8  12.0/10.9  19.5/17.3  31.4/31.4  91.8/69.6
//                       768 bf16   10.8/12.2  17.7/12.4  30.8/17.2  54.3/28.7  169/86
//                      1024 fp32   14.8/16.5  24.2/21.1  37.2/33.9  62.6/69.7  173/211
//   softmax, bias       256 fp32    9.0/13.5  12.3/14.6  19.7/22.9  32.0/41.0  62.8/75.1
//                       512 fp32   15.7/19.2  22.7/26.4  34.2/47.3  44.7/65.8  123/153
//                       640 fp32   24.4/23.2  35.5/27.9  64.2/59.4  85/87      217/188
//                       768 bf16   20.3/16.6  35.5/29.8  50.7/41.2  83/73      220/177
//                      1024 fp32   46.0/44.2  64.2/55.8  86/108     124/161    276/377
//   sigmoid, bias       128 fp32   10.2/12.5  11.6/12.6  14.0/13.8  17.7/16.6  36.8/37.1
//                       192 fp32   12.0/12.7  16.5/14.3  20.4/14.8  26.4/19.3  55.2/44.9
//   logits (softmax)    128 fp32    3.3/6.4    5.3/6.6    7.0/7.1   11.4/9.8   29.4/28.6
//                       192 fp32    4.9/7.4    7.2/7.5   10.2/8.4   15.9/12.3  43.3/35.8
// so up to 128 experts the warps' kernel stays.
inline int64_t list_rows_per_sm(const RouteArgs& a, int row_bytes) {
    if (a.score == OS_SCORE_SIGMOID && (a.bias || (a.groups > 1 && a.group_top == 2))) return 16;
    if (row_bytes >= 4096 || (a.bias && a.score == OS_SCORE_SOFTMAX && a.experts <= 512))
        return INT64_MAX;
    return 32;
}

// That kernel fits: rows and groups of whole 16-byte chunks (rows of eight of
// them, for the copy's placement), lists and choose_exact's runs that fit, and
// enough rows and experts.
template <typename T>
bool list_fits(const RouteArgs& a, const Shape& s, int sms) {
    const int bytes = a.experts * int(sizeof(T));
    return a.K <= 16 && a.experts > 128 && a.experts <= route::kListExperts && bytes % 128 == 0 &&
           a.experts / a.groups * int(sizeof(T)) % 16 == 0 && s.per_lane <= 32 &&
           reinterpret_cast<uintptr_t>(a.x) % 16 == 0 &&
           a.rows / sms >= list_rows_per_sm(a, bytes);
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
