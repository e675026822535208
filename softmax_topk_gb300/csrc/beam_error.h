// beam_error.h -- how far the selection's fp32 sums can be off.
#pragma once

#include <cmath>
#include <cstdint>

namespace os {

// A bound of the error of a row's ln d as beam_runs_kernel and beam_merge_kernel form it,
// for rows of `cols` columns of which a thread sums `share` of one run.  In units u of
// 2^-23 of the value (a rounding loses u / 2 at most, exp1 0.75, ex2.approx 2):
//
//   exponents and differences of maxima  A rounded difference loses u / 2 times its size.
//       From a value by its thread's reference, the references behind it, the warp's, the
//       run's and the row's maximum they add up to y, the value's distance from the row's
//       maximum, and 2 (a value is up to 1 above its reference).  Weights e^-y of n
//       columns, one of which has y = 0, have a mean y of at most 1 + ln n.  With log2 e in
//       one part (0.112 y): 0.612 (3 + ln cols).
//   a reference whose product with log2 e is rounded  the factor between the two
//       (ex2.approx, a product): 2.5.  The two are 1 apart for references of 2^24 and up to
//       16 for 2^28, the largest that go this way, and exponents are as much longer: 5.5
//       more for rows whose maximum is beyond 2^24 (kFarError).
//   weights  ex2.approx: 2.
//   sums  a tile's 32 values 4.5; tiles, compensated, at the end 0.5, and what the sum
//       of the lost parts loses itself: an addition 2^-24 of them, which are at most 2^-24
//       of the sum for each addition before: share^2 2^-26.
//   changes of the reference  exp1 and a product, 1.25 each on what was summed before.  A
//       change comes for a value more than 1 above the reference, so what has been through
//       j of them is at most share e^-j beside that value's own weight: ln share + 0.6
//       changes in the mean.
//   merges  exp1, a product and a tree of sums: threads to a warp 3.75, warps to a run 2.75,
//       runs to a row 3.75; the logarithm 0.5.
//
// The sums that are formed one by one (careful_sum) have fewer of each.
constexpr float kFarError = 5.5f * 0x1p-23f;
inline double beam_lse_error(int64_t cols, int64_t share) {
    const double n = static_cast<double>(share);
    const double units = 0.612 * (3 + std::log(static_cast<double>(cols))) + 2.5 + 2 + 5 +
                         1.25 * (std::log(n) + 0.6) + 10.75 + n * n * 0x1p-26;
    return units * 0x1p-23;
}

}  // namespace os
