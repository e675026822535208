// paged_common.cuh -- where a position of a sequence lies in a paged cache.
#pragma once

#include "ops.cuh"

namespace os {

// The kernels of a decode step follow one another on a stream.  Each is launched so that
// it may be put in place while the one before it still runs (launch_behind): wait_before
// holds it until that one has ended and its writes are seen, let_next lets the one behind
// it come as soon as every CTA has called it.  What the one before may have written is read
// by plain loads: for those of the read-only path the compiler may take it that nothing
// writes there while the kernel runs, its wait included, and move them before the wait.
__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;"); }

namespace paged {

// Position -> page of a sequence, slot in it.  Pages of 2^shift slots by a shift,
// others (shift < 0) by the high half of a product with floor(2^64 / size) + 1,
// exact for positions of 32 bits.
struct PageSplit {
    int size, shift;
    unsigned long long magic;
    __device__ __forceinline__ int page(int pos) const {
        return shift >= 0 ? pos >> shift
                          : static_cast<int>(
                                __umul64hi(magic, static_cast<unsigned long long>(pos)));
    }
};

inline PageSplit page_split(int size) {
    PageSplit s = {size, -1, 0};
    for (int i = 0; i < 31; ++i)
        if (size == (1 << i)) s.shift = i;
    if (s.shift < 0) s.magic = ~0ull / static_cast<unsigned>(size) + 1;
    return s;
}

}  // namespace paged
}  // namespace os
