// Reading a step's device arrays inside a kernel.  The host has not seen them:
// every index is held to the sizes of the launch before it is used, and one that
// is outside sets an error bit and leaves its row out.
#pragma once

#include <cstdint>
#include <utility>

#include "chained.cuh"
#include "sparse_kernels.h"

namespace gp {

constexpr int kStepPage = 256;
constexpr int kStepPageLog = 8;

// log2 of a block's tokens: places and pages of blocks are shifts (a division by a
// size that the compiler does not know is some thirty instructions).
__host__ __device__ constexpr int log2_const(int n) { return n > 1 ? 1 + log2_const(n / 2) : 0; }
__device__ __forceinline__ int log2_of(int block) { return 31 - __clz(block); }

// A call's launch.  The calls of a step follow one another on the engine stream with
// little to do each: the next one's blocks are placed while the last ones of this one
// still run, and wait on the device for its end before they touch anything (every kernel
// calls begin_step first; all it reads after that, by ordinary loads or TMA).
template <typename... P, typename... A>
cudaError_t launch_step_kernel(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t s, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}
__device__ __forceinline__ void begin_step() {
  let_next_in();
  wait_for_previous();
}

// One rule for the rows of every kernel: row i is request r's if row_req[i] names r and row0
// has it there, row0[r] <= i < row0[r + 1].  It takes part if r's slot is the engine's and
// its own place, cached + i - row0[r], is in the tables; if not, it alone is left out and
// an error bit set.  Rows that row_req gives to none, or behind row0[n], are left out as they are.
__device__ __forceinline__ bool row_named(const StepArgs& s, int named, int r) {
  if (named != r && named != -1) atomicOr(s.err, ERR_BAD_SLOT);
  return named == r;
}
// How many of the request's rows [row0, end) take part: the first ones.
__device__ __forceinline__ int rows_placed(const StepArgs& s, int row0, int end, int slot, int cached, bool report) {
  int bad = 0, rows = 0;
  if (row0 < 0 || end < row0 || end > s.max_rows) {
    bad = ERR_BAD_SLOT;
  } else if (end > row0) {
    const int room = cached < 0 ? 0 : max(s.maxp * kStepPage - cached, 0);
    rows = slot < 0 || slot >= s.M ? 0 : min(end - row0, room);
    bad = slot < 0 || slot >= s.M ? ERR_BAD_SLOT : rows < end - row0 ? ERR_BAD_PAGE : 0;
  }
  if (bad && report) atomicOr(s.err, bad);
  return rows;
}

// A single row: its request's slot and its logical slot there (it sees the slots [0, at]).
struct StepRow {
  bool live;
  int slot;
  int at;
};
__device__ __forceinline__ StepRow find_row(const StepArgs& s, int row, bool report) {
  const int r = s.row_req[row], rows = s.row0[s.n];
  if (r == -1 || row >= rows) return {false, 0, 0};
  if (r < 0 || r >= s.n) {
    if (report) atomicOr(s.err, ERR_BAD_SLOT);
    return {false, 0, 0};
  }
  const int row0 = s.row0[r], end = s.row0[r + 1], slot = s.slots[r], cached = s.cached[r];
  if (row < row0 || row >= end) {
    if (report) atomicOr(s.err, ERR_BAD_SLOT);
    return {false, 0, 0};
  }
  return {row - row0 < rows_placed(s, row0, end, slot, cached, report), slot, cached + (row - row0)};
}

// The page of a logical page of `slot`; -1 (and the error bit) if it is none.
__device__ __forceinline__ int step_page(const StepArgs& s, int slot, int logical) {
  const int page = s.tables[(size_t)slot * s.maxp + logical];
  if (page >= 0 && page < s.num_pages_total) return page;
  atomicOr(s.err, ERR_BAD_PAGE);
  return -1;
}

// Pieces of 2^log rows of each request, numbered over all of them: request r's
// are base(r), base(r) + 1, ... with base(r) = (row0[r] >> log) + extra r, so that
// the launch can be sized without the lengths (at most (max_rows >> log) + extra n
// pieces; those that no row falls into are left at once).  A whole warp calls it;
// `report`: this thread tells of rows that cannot take part.
struct StepPiece {
  int r;     // -1: none
  int at;    // number within the request
  int rows;  // of the request, that take part
  int row0;
  int slot, cached;
};
__device__ __forceinline__ StepPiece find_piece(const StepArgs& s, int j, int log, int extra, bool report) {
  const int lane = threadIdx.x & 31;
  StepPiece p;
  int end;
  if (s.n <= 64) {  // everything of every request at once: one trip to memory instead of two
    int v[2][4];
    unsigned below = 0u;  // requests whose first piece is j or before
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = lane + 32 * i;
      v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0;
      if (r < s.n) {
        v[i][0] = s.row0[r];
        v[i][1] = s.row0[r + 1];
        v[i][2] = s.slots[r];
        v[i][3] = s.cached[r];
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      below += __popc(__ballot_sync(0xffffffffu, lane + 32 * i < s.n && (v[i][0] >> log) + extra * (lane + 32 * i) <= j));
    p.r = (int)below - 1;
    const bool upper = p.r >= 32;
    p.row0 = __shfl_sync(0xffffffffu, upper ? v[1][0] : v[0][0], p.r & 31);
    end = __shfl_sync(0xffffffffu, upper ? v[1][1] : v[0][1], p.r & 31);
    p.slot = __shfl_sync(0xffffffffu, upper ? v[1][2] : v[0][2], p.r & 31);
    p.cached = __shfl_sync(0xffffffffu, upper ? v[1][3] : v[0][3], p.r & 31);
    if (p.r < 0) return {-1, 0, 0, 0, 0, 0};
  } else {
    int below = 0;
    for (int r = lane; r < s.n; r += 32) below += (s.row0[r] >> log) + extra * r <= j;
    below = __reduce_add_sync(0xffffffffu, below);
    if (below == 0) return {-1, 0, 0, 0, 0, 0};
    p.r = below - 1;
    p.row0 = s.row0[p.r];
    end = s.row0[below];
    p.slot = s.slots[p.r];
    p.cached = s.cached[p.r];
  }
  p.at = j - ((p.row0 >> log) + extra * p.r);
  p.rows = rows_placed(s, p.row0, end, p.slot, p.cached, report);
  if (p.rows == 0 || p.at < 0) return {-1, 0, 0, 0, 0, 0};
  return p;
}

// The exponent of a scale: the least whole e >= -100 with top <= 127 * 2^e, at
// most 100 (top >= 0, finite or not).
__device__ __forceinline__ int scale_exponent(float top) {
  if (!(top > 0.f)) return -100;
  const unsigned u = __float_as_uint(top);
  const int e = (int)(u >> 23) - 133 + ((u & 0x7fffffu) > 0x7e0000u);  // 127 = 0x1.fcp6
  return min(max(e, -100), 100);
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((unsigned)(e + 127) << 23); }

}  // namespace gp
