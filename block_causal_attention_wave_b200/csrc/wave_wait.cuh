// Bounded waits of the single-token kernels.
#pragma once
#include <cstdint>

#include "wave_sync.cuh"

namespace wavei {

// wait_bar with the first test in line, for threads whose time between waits is
// what a loop is bound by. A try_wait may suspend for longer than a short bound
// and then succeed, so with bounds under a millisecond (which a test sets to
// make a wait run out) the clock decides after a success too.
__device__ __forceinline__ bool wait_within(uint32_t bar, uint32_t parity, const Ctl& ctl, int code) {
  if (ctl.timeout_ns >= kLongWaitNs) {
    if (wptx::mbar_try_wait(bar, parity)) return true;
    return wait_bar(bar, parity, ctl, code);
  }
  const uint64_t t0 = wptx::globaltimer_ns();
  if (!wait_bar(bar, parity, ctl, code)) return false;
  if (wptx::globaltimer_ns() - t0 <= ctl.timeout_ns) return true;
  *ctl.abort_flag = 1;
  atomicCAS(ctl.status, 0, code);
  return false;
}

}  // namespace wavei
