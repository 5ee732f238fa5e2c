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

// A warp's wait for something that takes as long as the work in between: it gives up only when
// `moved`, which that work changes, has stood still for as long as any other wait lasts.
template <long long kCycles = kWaitCycles>
__device__ __forceinline__ bool wait_warp_while_moving(uint64_t* bar, uint32_t parity, volatile int* moved,
                                                       volatile int* abort, int* status) {
  bool ok = mbar_test(bar, parity);
  if (!ok) {
    long long t0 = clock64();
    int last = *moved;
    while (!(ok = mbar_try_wait(bar, parity)) && !*abort) {
      const int now = *moved;
      if (now != last) {
        last = now, t0 = clock64();
      } else if (clock64() - t0 > kCycles) {
        *abort = 1;
        atomicOr(status, RKV_FLAG_TIMEOUT);
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

}  // namespace rkv
