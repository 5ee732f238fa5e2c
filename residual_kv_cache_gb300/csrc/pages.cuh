// pages.cuh - waits of the full-attention layers' tensor-core kernels.
#pragma once
#include "pages.h"
#include "tc_common.cuh"

namespace rkv {

// One thread's bounded wait.  The plain test comes first: of a phase that is complete it
// takes 48 cycles, where the wait with a suspend-time hint takes 83, and these kernels' roles
// mostly find their barriers ready.
template <long long kCycles = kWaitCycles>
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  return mbar_test(bar, parity) || mbar_wait<kCycles>(bar, parity, abort, status);
}

// A warp's: every lane waits, the verdict is common (a wait of lane 0 handed on by a shuffle
// takes 258 cycles).
template <long long kCycles = kWaitCycles>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  return __all_sync(0xffffffffu, wait_one<kCycles>(bar, parity, abort, status));
}

// Limit of a wait for a place that whole pieces of work leave, whatever their length: the roles at
// work wait for each other with the usual limit, and give up for this one too.
constexpr long long kWaitForWork = 64 * kWaitCycles;

}  // namespace rkv
