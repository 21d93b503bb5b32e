// watchdog.cuh -- bounded mbarrier waits and the status record of a launch.
// P is a kernel's parameter block; it holds `status` (4 ints in global memory:
// code, role, block, iteration) and `watchdog_ns` (the limit of every wait).
#pragma once

#include <cstdint>

#include "layout.h"
#include "ptx.cuh"

namespace tg {

template <class P>
__device__ __forceinline__ void report(const P &p, int code, int role, int iter)
{
    if (atomicCAS(p.status, 0, code) == 0) {
        p.status[1] = role;
        p.status[2] = int(blockIdx.x);
        p.status[3] = iter;
    }
}

// Debug-check builds (TGEMM_DEBUG_CHECKS=1) test every shared-memory, tensor-
// memory and TMA address the kernel forms against the plan's layout before the
// access.  A failed check records TGEMM_ERR_CHECK with the role and the
// iteration, raises the CTA's abort flag and skips the access, so a bug shows
// up as a status code, never as a fault.  Release builds compile the checks
// away.
#ifndef TGEMM_DEBUG_CHECKS
#define TGEMM_DEBUG_CHECKS 0
#endif

template <class P>
__device__ __forceinline__ bool check(bool ok, const P &p, volatile int *abort, int role, int iter)
{
    if (TGEMM_DEBUG_CHECKS && !ok) {
        report(p, kErrCheck, role, iter);
        *abort = 1;
        return false;
    }
    return true;
}

// Bounded wait for the phase of parity `parity` of `bar`.  Returns false when
// the CTA has aborted (if honour_abort) or when the watchdog expires; the
// latter is recorded and raises the CTA's abort flag.
template <class P>
__device__ __noinline__ bool wait_bar(uint32_t bar, uint32_t parity, const P &p, volatile int *abort, int role,
                                      int iter, bool honour_abort = true)
{
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer();
    uint32_t spins = 0;
    for (;;) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((++spins & 15u) == 0) {
            if (honour_abort && *abort) return false;
            if (globaltimer() - t0 > p.watchdog_ns) {
                *abort = 1;
                report(p, kErrTimeout, role, iter);
                return false;
            }
        }
    }
}

// Warp-collective form of wait_bar: every lane polls once (the common case
// is a phase that has already completed); otherwise lane 0 waits with the
// watchdog and the outcome is broadcast, so the warp stays converged and its
// control flow uniform.
template <class P>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const P &p, volatile int *abort, int role,
                                          int iter, bool honour_abort = true)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    int ok = 1;
    if ((threadIdx.x & 31u) == 0) ok = wait_bar(bar, parity, p, abort, role, iter, honour_abort) ? 1 : 0;
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

}  // namespace tg
