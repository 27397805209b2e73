// Bounded waits for copies and matrix steps that complete on an mbarrier, of the projection and
// attention kernels.  A wait that runs out is given up; the kernel then waits once more, with the
// default limit, for what it has under way: nothing may land in shared memory that another use
// or another CTA has by then.
#pragma once
#include "internal.cuh"

namespace edge0 {

// limit of the launches from now on (edge0_block_set_wait_limit)
unsigned long long block_wait_limit();

// Waits for a copy's phase, at most `limit` ns; by a whole warp, which agrees on the answer.
// (Where the limit is 0 the kernels have given up from the start: a test of it here cost the
// projection of 20,000 x 2048 at 256 tokens 4 %.)
__device__ __forceinline__ bool wait_copy(uint64_t* bar, uint32_t parity, unsigned long long limit) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
        unsigned long long t0, now;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
        do {
            ok = mbar_try_wait(bar, parity);
            asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
        } while (!ok && now - t0 < limit);
    }
    return __all_sync(0xffffffffu, ok);
}

// After giving up: waits for the copies first .. last - 1 of a ring of `stages`.
__device__ __forceinline__ void drain_copies(uint64_t* bar, int first, int last, int stages) {
    for (int s = first; s < last; ++s) wait_copy(&bar[s % stages], (uint32_t)(s / stages) & 1, kDefaultWaitNs);
}
// ... out of line, where that leaves the registers to the way that is taken
static __device__ __noinline__ void drain_copies_call(uint64_t* bar, int first, int last, int stages) {
    drain_copies(bar, first, last, stages);
}

}  // namespace edge0
