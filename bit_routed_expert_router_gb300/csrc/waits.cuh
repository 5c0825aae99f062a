// Bounded waits on barriers, and what a CTA does in which one ran out.
#pragma once

#include "common.cuh"
#include "grouped.h"

namespace moe {

// A CTA's bounded waits.
struct Waits {
  volatile int abort;   // 1: one ran out; 2: the launch had given up before this CTA started
  int limit;            // of each, in 1024 cycles
};

__device__ __forceinline__ unsigned long long this_grid() {
  unsigned long long g;
  asm volatile("mov.u64 %0, %%gridid;" : "=l"(g));
  return g + 1;
}

constexpr long long kSettleCycles = 20000000;

// Bounded wait that also ends when another role of the CTA gave up.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, Waits* w) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (w->abort) return false;
    if (clock64() - t0 > 1024LL * w->limit) {
      w->abort = 1;
      return false;
    }
  }
}

// The same by a whole warp, which then agrees on the outcome.
__device__ __forceinline__ bool wait_bar_warp(uint64_t* bar, uint32_t parity, Waits* w) {
  return __all_sync(0xFFFFFFFFu, wait_bar(bar, parity, w));
}

// The end of a CTA that gave up, by all of its threads.  Copies, products and
// arrivals may be on their way, and no barrier tells which: those of a pair's odd
// CTA count on the even one's barriers, of which the phases that miss a share
// stay open.  All of them take microseconds; the CTA keeps its memories for
// another 10 ms.
__device__ __forceinline__ void report_and_settle(GaveUp* gave_up) {
  if (threadIdx.x == 0) {
    *static_cast<volatile unsigned long long*>(&gave_up->grid) = this_grid();
    atomicAdd(&gave_up->count, 1u);
  }
  const long long t0 = clock64();
  while (clock64() - t0 < kSettleCycles) __nanosleep(1000);
}

}  // namespace moe
