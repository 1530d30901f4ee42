// What the tensor-core kernels over listed blocks share: the blocks of a piece of
// rows, and bounded waits.
#pragma once

#include <cstdint>

#include "step.cuh"
#include "tc_ptx.cuh"

namespace gp {

// Bounded wait for a phase of an mbarrier; gives up when the limit passes or *abort
// is set.  (A try may itself wait for a while; a limit of 0 is looked at by the warp that
// loads, before it tries for a free buffer.)
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, const volatile int* abort, long long limit) {
  if (tc::mbar_try(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (*abort || clock64() - t0 > limit) return false;
    if (tc::mbar_try(bar, parity)) return true;
  }
}
// The same for what a role has in flight before it ends: whatever *abort says.
__device__ __forceinline__ void drain_phase(uint32_t bar, uint32_t parity) {
  const int zero = 0;
  wait_phase(bar, parity, &zero, kDefaultWaitLimit);
}

// The lists of a piece's rows: every warp of the CTA takes each WARPS-th row, its loads
// in flight together.  The first 32 entries are loaded ahead, as the rows are known
// before their places are.
template <int WARPS, int T>
struct BlockLists {
  static constexpr int N = (T + WARPS - 1) / WARPS;
  int b[N];

  __device__ __forceinline__ void load(const SparseArgs& a, size_t row0, int h, unsigned live, int k0) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i)
      b[i] = (live >> i & 1u) && k0 + lane < a.top ? a.blocks[((row0 + warp + i * WARPS) * a.Hkv + h) * a.top + k0 + lane] : -1;
  }
  static __device__ __forceinline__ unsigned rows_of(int m) {  // of this warp, of m in the piece
    unsigned live = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((int)(threadIdx.x >> 5) + i * WARPS < m) live |= 1u << i;
    return live;
  }
  // Sets the bits of the blocks that this warp's `live` rows list, a row's in seen[x * words]
  // and all of them in any (both cleared before).  A list counts up to its first entry that is negative,
  // not above the one before it or past the row's own block.
  __device__ __forceinline__ void mark(const SparseArgs& a, size_t row0, int h, unsigned live, int first_at, int lb, int words,
                                       unsigned* seen, unsigned* any) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int before[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      before[i] = -1;
      if (!(live >> i & 1u)) b[i] = -1;
    }
    for (int k0 = 0; live; load(a, row0, h, live, k0)) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int x = warp + i * WARPS;
        int last = __shfl_up_sync(0xffffffffu, b[i], 1);
        if (lane == 0) last = before[i];
        const unsigned ends = __ballot_sync(0xffffffffu, b[i] < 0 || b[i] <= last || b[i] > (first_at + x) >> lb);
        if (!(ends & ((2u << lane) - 1))) {
          atomicOr(&seen[x * words + (b[i] >> 5)], 1u << (b[i] & 31));
          atomicOr(&any[b[i] >> 5], 1u << (b[i] & 31));
        }
        if (ends) live &= ~(1u << i);
        before[i] = __shfl_sync(0xffffffffu, b[i], 31);
      }
      k0 += 32;
      if (k0 >= a.top) break;
    }
  }
};

// Puts the marked blocks in order: put(place, block).  Every warp of the CTA calls it,
// takes each WARPS-th word (a lane a bit) and gets the count.
template <int WARPS, typename Put>
__device__ __forceinline__ int list_blocks(const unsigned* any, int words, Put&& put) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int total = 0;
  for (int w0 = 0; w0 < words; w0 += 32) {
    const unsigned mine = w0 + lane < words ? any[w0 + lane] : 0u;
    int upto = __popc(mine);
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += v;
    }
    const int before = total + upto - __popc(mine);
    total += __shfl_sync(0xffffffffu, upto, 31);
    for (int w = warp; w < 32 && w0 + w < words; w += WARPS) {
      const unsigned bits = __shfl_sync(0xffffffffu, mine, w);
      const int at = __shfl_sync(0xffffffffu, before, w);
      if (bits >> lane & 1u) put(at + __popc(bits & ((1u << lane) - 1)), (w0 + w) * 32 + lane);
    }
  }
  return total;
}

}  // namespace gp
