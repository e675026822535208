// Beam search's selection: the rows' runs, then the groups.
#include <algorithm>

#include "beam_error.h"
#include "host_common.h"
#include "internal.h"
#include "kernels/beam_kernel.cuh"

namespace os {

namespace {

constexpr int kMaxRuns = 32;

// Runs per row: as many as the GPU holds at once (three to an SM), for each run pays for a
// selection of its own.  us with 1, 2, 3 runs, where no beam has ended, one in eight, seven
// in eight:
//   128 rows of 128256 bf16   25.9 21.6 23.3   26.3 21.8 23.8   24.5 19.5 18.7   (3 are taken)
//   160                       28.3 24.5 26.3   28.7 24.6 23.2   24.7 20.0 20.6   (2)
//   256                       29.1 32.9 30.5   29.0 27.5 30.0   26.1 20.8 21.5   (1)
//   512                       49.2 46.5 46.7   38.3 41.5 42.8   27.7 24.9 26.1   (1)
//   256 rows of 32000 fp32    17.7 21.3 20.7   17.8 18.4 20.7   15.3 16.4 16.7   (1)
// The host does not know which beams have ended.  The rule loses 2 to 3 us at 128 rows, and at
// 512 where none has; 5 at 256 where most have.
constexpr int kRunsPerSm = 3;

struct Split {
    int runs;
    int64_t run_tiles;
};

Split split_rows(int64_t rows, int64_t cols, os_dtype in, int sms) {
    const int64_t tiles = in == OS_F32 ? ceil_div(cols + 3, beam::Tile<float>::kTile)
                                       : ceil_div(cols + 7, beam::Tile<__nv_bfloat16>::kTile);
    const int64_t want = min64(min64(tiles, kMaxRuns),
                               std::max<int64_t>(1, int64_t(sms) * kRunsPerSm / rows));
    Split s;
    s.run_tiles = ceil_div(tiles, want);
    s.runs = static_cast<int>(ceil_div(tiles, s.run_tiles));
    return s;
}

template <typename T, int KP>
cudaError_t launch(const beam::BeamArgs& a, int64_t groups, cudaStream_t stream) {
    auto runs = beam::beam_runs_kernel<T, KP>;
    constexpr int smem = sizeof(beam::RunShared<T>);
    if (!prepare_kernel(runs, 1, smem)) return cudaErrorInvalidConfiguration;
    const cudaError_t e =
        launch_behind(runs, dim3(static_cast<unsigned>(groups * a.beams * a.runs)), beam::kThreads,
                      smem, stream, a);
    if (e != cudaSuccess) return e;
    return launch_kernel(beam::beam_merge_kernel<T, KP>, groups * a.helpers, beam::kMergeThreads,
                         a.helpers, 0, stream, a);
}

template <typename T>
cudaError_t launch_k(const beam::BeamArgs& a, int64_t groups, cudaStream_t stream) {
    if (a.K <= 8) return launch<T, 8>(a, groups, stream);
    if (a.K <= 16) return launch<T, 16>(a, groups, stream);
    if (a.K <= 32) return launch<T, 32>(a, groups, stream);
    return launch<T, 64>(a, groups, stream);
}

}  // namespace

int64_t beam_select_workspace(int64_t groups, int beams, int64_t cols, int K, os_dtype in, int sms) {
    const Split s = split_rows(groups * beams, cols, in, sms);
    return groups * beams * s.runs * (K + 1) * 8;
}

cudaError_t launch_beam_select(const BeamSelectArgs& p, cudaStream_t stream) {
    const DeviceInfo* dev = device_info();
    if (!dev) return cudaErrorInvalidDevice;
    const Split s = split_rows(p.groups * p.beams, p.cols, p.in, dev->sms);
    beam::BeamArgs a = {};
    a.x = p.x;
    a.scores = p.scores;
    a.ended = p.ended;
    a.out = p.out;
    a.parents = p.parents;
    a.tokens = p.tokens;
    a.states = static_cast<float2*>(p.workspace);
    a.lists = reinterpret_cast<beam::u64*>(a.states + p.groups * p.beams * s.runs);
    a.cols = p.cols;
    a.beams = p.beams;
    a.K = p.K;
    a.runs = s.runs;
    a.run_tiles = static_cast<int>(s.run_tiles);
    a.pad = p.pad;
    // the CTAs of a group share the exact sums, where there are SMs for them
    a.helpers = beam::kHelpers;
    while (a.helpers > 1 && p.groups * a.helpers > 2 * dev->sms) a.helpers /= 2;
    // (31 units of 2^-23 for 1000 columns, 33 for 50257 in runs of one tile, 38 for 128256 in one)
    const int per_tile = p.in == OS_F32 ? beam::Tile<float>::kPer : beam::Tile<__nv_bfloat16>::kPer;
    a.eps = static_cast<float>(beam_lse_error(p.cols, s.run_tiles * per_tile));
    return p.in == OS_F32 ? launch_k<float>(a, p.groups, stream)
                          : launch_k<__nv_bfloat16>(a, p.groups, stream);
}

}  // namespace os
