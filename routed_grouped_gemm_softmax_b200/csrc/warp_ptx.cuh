// warp_ptx.cuh -- roles that a whole converged warp plays, one elected lane of it issuing
// the TMA loads, barrier arrivals and tcgen05 MMAs.
//
// Those instructions take addresses, descriptors and coordinates from uniform registers.
// In a branch that lane 0 takes by its index nothing can be computed there, and each operand
// of each instruction is moved over on its own: issuing one 128 x N x 16 MMA took 80
// cycles in the dense products' loop.  A warp that stays converged, its index read by a shuffle,
// computes them in place (32 cycles there), and elect.sync marks a branch as one lane's.
// Back to back, without a loop's waits, an MMA of N <= 64 takes 64 cycles from lane 0 and 49 so;
// from N = 128 on, 64 cycles (128 at N = 256), the tensor core is the bound either way.
#pragma once
#include "sm100_ptx.cuh"

namespace moe {

// This thread's warp, in a form that is known to be the same for the whole warp.
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(0xffffffffu, threadIdx.x / 32, 0); }

// mbar_wait by a whole converged warp.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, uint64_t limit_ns = kWaitLimitNs)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 256; ++i)
            if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > limit_ns)) return false;
    }
}

// True in one lane of a converged warp, always the same one.
__device__ __forceinline__ bool elect_one()
{
    uint32_t on;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
    return on != 0;
}

}  // namespace moe
