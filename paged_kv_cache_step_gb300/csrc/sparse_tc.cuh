// What the tensor-core kernels over listed blocks share: the blocks of a piece of
// rows, and bounded waits.
#pragma once

#include <cstdint>

#include "step.cuh"
#include "tc_ptx.cuh"

namespace gp {

// Bounded wait for a phase of an mbarrier; gives up when the limit passes or *abort
// is set.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, const volatile int* abort) {
  if (tc::mbar_try(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (*abort || clock64() - t0 > kDefaultWaitLimit) return false;
    if (tc::mbar_try(bar, parity)) return true;
  }
}
// The same for what a role has in flight before it ends: whatever *abort says.
__device__ __forceinline__ void drain_phase(uint32_t bar, uint32_t parity) {
  const int zero = 0;
  wait_phase(bar, parity, &zero);
}

// Sets the bits of a row's listed blocks in `seen` (cleared before): up to the first
// entry that is negative, not above the one before it or past `own`.  A whole warp.
__device__ __forceinline__ void mark_blocks(const int32_t* list, int top, int own, unsigned* seen) {
  const int lane = threadIdx.x & 31;
  int before = -1;
  for (int k0 = 0; k0 < top; k0 += 32) {
    const int b = k0 + lane < top ? list[k0 + lane] : -1;
    int last = __shfl_up_sync(0xffffffffu, b, 1);
    if (lane == 0) last = before;
    const unsigned ends = __ballot_sync(0xffffffffu, b < 0 || b <= last || b > own);
    if (!(ends & ((2u << lane) - 1))) atomicOr(&seen[b >> 5], 1u << (b & 31));
    if (ends) break;
    before = __shfl_sync(0xffffffffu, b, 31);
  }
}

}  // namespace gp
