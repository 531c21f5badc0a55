// ring.cuh -- the bookkeeping of a ring of shared-memory stages that one warp fills by
// asynchronous copies, a full barrier per stage, and how such a warp winds down.
//
// Copies that land after their block has left write into the next block's shared memory, so
// a filling warp leaves only once the last fill of every stage has landed (or that wait,
// bounded like all others, has run out too).  On the way of a call without faults the
// readers wait for the same fills, and this costs nothing.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define MOE_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MOE_HOST_DEVICE inline
#endif

namespace moe {

// Parity of the last fill of stage i, seen from the filler's position: the next stage it will
// fill and that lap's parity.  Stages before it were filled in this lap, the others in the
// lap before; of a stage that was never filled this is the parity before the first phase,
// for which no wait blocks.
MOE_HOST_DEVICE uint32_t last_fill_parity(int i, int stage, uint32_t phase) { return i < stage ? phase : phase ^ 1u; }

}  // namespace moe

#ifdef __CUDACC__
#include "sm100_ptx.cuh"

namespace moe {

// Bounds-checked builds can make these waits give up at once (moe_checked_give_up_waits): the
// winding down is tested so.
#if MOE_CHECKED
__device__ int g_give_up_waits;
#endif

__device__ __forceinline__ bool ring_wait(uint64_t &bar, uint32_t parity) {
#if MOE_CHECKED
    if (*static_cast<volatile int *>(&g_give_up_waits)) {
        raise_device_error(MOE_DEVERR_TIMEOUT);
        return false;
    }
#endif
    return ptx::mbar_wait(ptx::smem_u32(&bar), parity);
}

// Wait of a block that shares the flag `failed`: false once a wait gave up (and raised the
// device error), at once after that unless the phase is over.  A reader whose wait failed
// runs out over what the buffers hold.  Its arrival on `empty` would let a stage be filled
// over a copy that is still under way, so either it arrives no more (the matvec), or the
// filler tests `failed`, which is set before such an arrival, between its wait and its copy
// (the row kernels, whose registers are scarcer: a predicate kept across the reader's loop
// took up to a third longer on narrow rows.  The test hides behind the making of addresses
// there; on the matvec's shorter way it cost 3% of long rows).
__device__ __forceinline__ bool wait_or_fail(int &failed, uint64_t &bar, uint32_t parity) {
    volatile int *flag = &failed;
    if (ptx::mbar_test_wait(ptx::smem_u32(&bar), parity)) return true;
    if (!*flag && ring_wait(bar, parity)) return true;
    *flag = 1;
    return false;
}

// The filling warp's last step: a lane per stage waits until its last fill has landed.
__device__ __forceinline__ void wait_for_fills(uint64_t *full, int stages, int stage, uint32_t phase) {
    const int i = threadIdx.x & 31;
    if (i < stages) ptx::mbar_wait(ptx::smem_u32(&full[i]), last_fill_parity(i, stage, phase));
    __syncwarp();
}

}  // namespace moe
#endif
