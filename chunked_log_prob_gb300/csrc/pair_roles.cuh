// What the warps of a CTA pair's GEMM share: bounded waits of a whole warp, the drain
// of copies in flight before a CTA leaves, and the lane that issues.
#pragma once

#include "ptx.cuh"

namespace grpo {

// Waits, with a limit, for a phase that no role depends on any more.
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > kWaitLimitCycles) return;
}

// A warp's wait: one answer for all lanes, before steps of the whole warp. Each
// polls for itself, and one may give up (or see the abort flag) as another finds
// the phase done.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                          int* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status)) != 0;
}

// True in one lane of the (whole) warp. The compiler then knows that one thread
// runs what follows and feeds tcgen05 and TMA their uniform operands directly;
// behind `lane == 0` it cannot, and a stage took its issuing thread twice as
// long as the tensor core (weight gradient from a checkpoint, 16384 x 4096 x 4096: 518
// us against 407).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "elect.sync _|P, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, P;\n\t}"
      : "=r"(p));
  return p != 0;
}

}  // namespace grpo
