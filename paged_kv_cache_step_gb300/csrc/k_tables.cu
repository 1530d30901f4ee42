// Block tables, slot map and positions of a step, from lengths that only the
// GPU knows.
//
//   need_r  = ceil((cached_r + new_r) / 256) pages, take_r = max(0, need_r - held_r)
//   a request is given its rows and pages if it is valid, its rows fit the
//   buffers behind those that the valid requests before it ask for (given or not: a
//   plain running sum), and the free list holds its pages behind theirs; else it has no row in this step and keeps its table
//   row0  = running sum of the given rows
//   row i of request r: logical slot t = cached_r + i, page table[t / 256] or, for
//   t / 256 >= held_r, free[taken + (pages given before) + t / 256 - held_r]
//
// Bounded by latency: a step of 64 requests reads and writes 5 KB and takes 4 us in a
// graph.  One launch:
// every block of a cluster scans all requests for itself (4 bytes x 5 a request),
// the cluster meets once, so that no output is written before every input is
// read (num_pages may be held, taken taken_in), and then shares the rows.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "shared_limit.cuh"
#include "step.cuh"

namespace gp {
namespace {

constexpr int PAGE = 256;
constexpr int AT_ONCE = 2;
enum { GIVEN = 0, NO_PAGES = 1, NO_ROWS = 2, INVALID = 3 };  // gp_step_state

// Inclusive sum over the block's threads; every thread also gets the total.
__device__ __forceinline__ int block_sum(int v, int* part, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int x = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += x;
  }
  if (lane == 31) part[warp] = v;
  __syncthreads();
  int w = lane < warps ? part[lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int x = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += x;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  v += warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
  __syncthreads();
  return v;
}

__global__ void __launch_bounds__(1024, 1) k_tables(const __grid_constant__ TablesArgs a) {
  extern __shared__ int sm[];
  int* row0 = sm;               // [n + 1]
  int* first = row0 + a.n + 1;  // [n] pages given before
  int* held = first + a.n;      // [n]
  int* cached = held + a.n;     // [n]
  int* slots = cached + a.n;    // [n]
  unsigned* seen = reinterpret_cast<unsigned*>(slots + a.n);  // a bit a slot
  const int words = (a.M + 31) / 32;
  unsigned* twice = seen + words;
  __shared__ int part[32];
  const int tid = threadIdx.x, nt = blockDim.x;
  const unsigned rank = blockIdx.x, ranks = gridDim.x;  // (of one cluster, unless the buffers are apart)
  const bool leader = rank == 0;

  for (int i = tid; i < 2 * words; i += nt) seen[i] = 0;
  begin_step();
  __syncthreads();
  for (int r = tid; r < a.n; r += nt) {  // a slot that is listed twice is no one's
    const int s = a.slots[r];
    if (s >= 0 && s < a.M && (atomicOr(&seen[s >> 5], 1u << (s & 31)) >> (s & 31) & 1)) atomicOr(&twice[s >> 5], 1u << (s & 31));
  }
  const int before = a.taken_in ? *a.taken_in : 0;
  const int room = before >= 0 && before <= a.num_free ? a.num_free - before : 0;
  __syncthreads();

  int rows_wanted = 0, pages_wanted = 0, rows = 0, pages = 0;  // of the requests before this round's
  for (int r0 = 0; r0 < a.n; r0 += nt) {
    const int r = r0 + tid;
    int have = 0, fresh = 0, need = 0, state = INVALID, s = 0, c = 0;
    if (r < a.n) {
      s = a.slots[r];
      c = a.cached[r];
      const int m = a.fresh[r];
      if (s >= 0 && s < a.M) {
        have = a.held[s];
        if (!(twice[s >> 5] >> (s & 31) & 1) && c >= 0 && m >= 0 && (int64_t)c + m <= (int64_t)a.maxp * PAGE && have <= a.maxp && have >= (c + PAGE - 1) / PAGE) {
          state = GIVEN;
          fresh = m;
          need = (c + m + PAGE - 1) / PAGE;
        }
      }
    }
    int total;
    const int upto = rows_wanted + block_sum(fresh, part, total);
    rows_wanted += total;
    if (state == GIVEN && fresh > 0 && upto > a.max_rows) state = NO_ROWS;
    int take = state == GIVEN ? max(0, need - have) : 0;
    const int pages_upto = pages_wanted + block_sum(take, part, total);
    pages_wanted += total;
    if (take > 0 && pages_upto > room) state = NO_PAGES;
    if (state != GIVEN) fresh = take = 0;
    const int row_end = rows + block_sum(fresh, part, total);
    rows += total;
    const int page_end = pages + block_sum(take, part, total);
    pages += total;
    if (r < a.n) {
      row0[r] = row_end - fresh;
      first[r] = page_end - take;
      held[r] = have;
      cached[r] = c;
      slots[r] = s;
      if (r == a.n - 1) row0[a.n] = row_end;
    }
    // kept for the writes below: the state of this round's request
    if (r < a.n && leader) a.state[r] = state;
  }
  if (a.n == 0 && tid == 0) row0[0] = 0;
  // every block has read what another may write
  if (ranks > 1 && !a.apart) {
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
  const int stride = nt * (int)ranks, me = (int)rank * nt + tid;
  for (int r = me; r < a.n; r += stride) {
    a.row0[r] = row0[r];
    const int taken = (r + 1 < a.n ? first[r + 1] : pages) - first[r];
    const int s = slots[r];
    if (s >= 0 && s < a.M) {  // (one that is listed twice keeps its pages: the same number twice)
      a.num_pages[s] = held[r] + taken;
      for (int j = 0; j < taken; ++j) a.tables[(size_t)s * a.maxp + held[r] + j] = a.free_pages[before + first[r] + j];
    }
  }
  if (me == 0) {
    a.row0[a.n] = row0[a.n];
    *a.taken = before + pages;
  }
  // A warp takes 32 AT_ONCE rows that follow each other, of few requests as a rule: it
  // looks up the first row's request, and a row of another its own.
  // (The entries of the tables that are read here are not those written above.)
  const int live = row0[a.n];
  auto request_of = [&](int row, int lo) {  // row0[lo] <= row
    int hi = a.n;                           // row0[request] <= row < row0[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (row0[mid] <= row) lo = mid;
      else hi = mid;
    }
    return lo;
  };
  for (int w0 = me / 32 * (32 * AT_ONCE); w0 < a.max_rows; w0 += stride * AT_ONCE) {
    const int base = w0 < live ? request_of(w0, 0) : 0, r0 = w0 + (tid & 31);
    int req[AT_ONCE], at[AT_ONCE], page[AT_ONCE];
    int64_t pos[AT_ONCE];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int row = r0 + 32 * i;
      req[i] = -1;
      at[i] = page[i] = 0;
      pos[i] = 0;
      if (row < live) {
        const int lo = row < row0[base + 1] ? base : request_of(row, base + 1);
        req[i] = lo;
        at[i] = cached[lo] + row - row0[lo];
        const int j = at[i] / PAGE;
        page[i] = j < held[lo] ? a.tables[(size_t)slots[lo] * a.maxp + j] : a.free_pages[before + first[lo] + j - held[lo]];
        pos[i] = a.pos[lo] + (row - row0[lo]);
      }
    }
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int row = r0 + 32 * i;
      if (row >= a.max_rows) break;
      const bool ok = page[i] >= 0 && page[i] < a.num_pages_total;
      if (!ok) atomicOr(a.err, ERR_BAD_PAGE);
      a.row_req[row] = req[i];
      a.slot_map[row] = req[i] >= 0 && ok ? (int64_t)page[i] * PAGE + at[i] % PAGE : -1;
      a.positions[row] = pos[i];
    }
  }
}

}  // namespace

cudaError_t launch_tables(const TablesArgs& a, cudaStream_t s) {
  // Buffers of their own for what is read and written need no meeting: blocks of 512
  // threads, one for 1024 rows.  Else a cluster, which 16 blocks are the most of.
  // 43 943 rows of 300 requests: 45, 26, 15, 10.3 and 7.5 us with 1, 2, 4, 8 and 16 blocks
  // of 1024 threads in a cluster, 5.1 us with 43 blocks apart.
  const bool small = a.n <= 256 && a.max_rows <= 512, large = !small && !a.apart && a.max_rows > 16384;
  const size_t smem = sizeof(int) * ((size_t)5 * a.n + 1 + 2 * ((size_t)(a.M + 31) / 32));
  cudaError_t e = allow_shared<&k_tables>(sizeof(int) * (5 * kStepMaxRequests + 1 + 2 * kStepMaxSlots / 32));
  if (e != cudaSuccess) return e;
  if (large && (e = allow_large_clusters<&k_tables>()) != cudaSuccess) return e;
  const int blocks = small ? 1 : a.apart ? std::min((a.max_rows + 1023) / 1024 + 1, 128) : large ? 16 : 8;
  return launch_step_kernel(k_tables, dim3((unsigned)blocks), small ? 256 : a.apart ? 512 : 1024, smem, a.apart ? 1 : blocks, s, a);
}

}  // namespace gp
