// Bounds of the keys of a block, per dimension, in 8 bits:
//
//   e  = the least whole number >= -100 with max |k| <= 127 * 2^e (at most 100)
//   lo = floor(min k / 2^e),  hi = ceil(max k / 2^e),  held to [-127, 127]
// over the block's tokens of one KV head, for every block that a new token of the
// step falls into (all of its tokens, the older ones among them).  The scale is a
// power of two, so both bounds are exact whole numbers and really bounds, and
// forming them again from the same keys gives the same bits.  NaN elements are
// left out; a dimension with no other counts as 0.
//
// Bounded by HBM for prompts (each key is read once) and by latency for a decode
// step: the whole block is read again rather than the old bounds moved, 16 KB a
// block of 64 tokens and head, which keeps the call free of a read-modify-write
// and makes it the one that rebuilds after an eviction too.
//
// A power of two of threads a (block, head), 16 bytes of a token each, eight loads in
// flight where the block has that many.  Measured: 64 blocks of 64 tokens with 8 heads 8.1 us
// (four dependent reads, from row0 to the keys; 5.2 us with the keys in L2), 13 734 tokens in
// blocks of 32 11 us (7.2 us), where reading the keys takes 4.3 at the copy rate: every CTA goes
// through that chain for one block, with nothing else in flight.
#include <cuda_bf16.h>

#include <cstdint>

#include "step.cuh"

namespace gp {
namespace {

constexpr int NT = 256;

template <int D, bool F32>
__global__ void __launch_bounds__(NT) k_bounds(const __grid_constant__ BoundsArgs a, int threads, int heads) {
  constexpr int N = F32 ? 4 : 8;   // elements of a piece
  constexpr int PIECES = D / N;    // of a row
  __shared__ float lo_s[NT * N], hi_s[NT * N];
  const int tid = threadIdx.x, unit = tid / threads, t = tid % threads;
  const int h = blockIdx.y * heads + unit, lb = log2_of(a.block);
  begin_step();
  const StepPiece p = find_piece(a.s, blockIdx.x, lb, 2, tid == 0);
  if (p.r < 0) return;
  const int last = p.cached + p.rows - 1;  // the request's last slot
  const int b = (p.cached >> lb) + p.at;
  if (b > last >> lb) return;
  const int t0 = max((b << lb) - p.cached, 0), rows = min(((b + 1) << lb) - p.cached, p.rows) - t0;  // of the block, up to NT
  const int named = tid < rows ? a.s.row_req[p.row0 + t0 + tid] : -1;
  const int page = step_page(a.s, p.slot, b >> (kStepPageLog - lb));
  if (page < 0) return;
  const bool mine = h < a.Hkv;
  const int per = kStepPage >> lb, sub = b & (per - 1), tokens = min(a.block, last + 1 - (b << lb));
  const size_t head = ((size_t)a.layer * a.s.num_pages_total + page) * a.Hkv + h;
  float lo[N], hi[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    lo[i] = __int_as_float(0x7f800000);
    hi[i] = __int_as_float(0xff800000);
  }
  const int piece = t % PIECES, step = threads / PIECES;
  if (mine) {
    const uint4* src = reinterpret_cast<const uint4*>(a.k_cache) + (head * kStepPage + (size_t)sub * a.block) * PIECES + piece;
#pragma unroll 8
    for (int x = t / PIECES; x < tokens; x += step) {
      const uint4 u = src[(size_t)x * PIECES];
      const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float f = F32 ? __uint_as_float(w[i]) : __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        lo[i] = fminf(lo[i], f);  // of a number and NaN the number
        hi[i] = fmaxf(hi[i], f);
      }
    }
  }
  // the token groups of a unit are joined: within a warp, then over its warps
#pragma unroll
  for (int d = PIECES; d < 32; d *= 2)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      lo[i] = fminf(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], d));
      hi[i] = fmaxf(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], d));
    }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    lo_s[i * NT + tid] = lo[i];
    hi_s[i * NT + tid] = hi[i];
  }
  if (!__syncthreads_or(row_named(a.s, named, p.r))) return;  // no row falls into the block
  constexpr int FIRST = PIECES < 32 ? 32 : PIECES;  // threads of a unit that end with a piece
  const bool ends = t < FIRST && t < PIECES;
  float top = 0.f;
  if (ends) {
    for (int x = FIRST; x < threads; x += FIRST)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        lo[i] = fminf(lo[i], lo_s[i * NT + tid + x]);
        hi[i] = fmaxf(hi[i], hi_s[i * NT + tid + x]);
      }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (lo[i] > hi[i]) lo[i] = hi[i] = 0.f;
      top = fmaxf(top, fmaxf(fabsf(lo[i]), fabsf(hi[i])));
    }
  }
  // (PIECES <= 32: they are in the unit's first warp)
#pragma unroll
  for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  if (!ends || !mine) return;
  const int e = scale_exponent(top);
  const float down = power_of_two(-e);
  unsigned lw[N / 4], hw[N / 4];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int l = (int)fminf(fmaxf(floorf(lo[i] * down), -127.f), 127.f), g = (int)fminf(fmaxf(ceilf(hi[i] * down), -127.f), 127.f);
    if (i % 4 == 0) lw[i / 4] = hw[i / 4] = 0u;
    lw[i / 4] |= (unsigned)(l & 255) << (8 * (i % 4));
    hw[i / 4] |= (unsigned)(g & 255) << (8 * (i % 4));
  }
  const size_t at = head * per + sub;
  unsigned* dst = reinterpret_cast<unsigned*>(a.bounds + at * 2 * D + piece * N);
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    dst[i] = lw[i];
    dst[D / 4 + i] = hw[i];
  }
  if (t == 0) a.scales[at] = power_of_two(e);
}

template <int D, bool F32>
cudaError_t launch_t(const BoundsArgs& a, cudaStream_t s) {
  constexpr int PIECES = D * (F32 ? 4 : 2) / 16;
  int threads = 32;
  while (threads < NT && threads * 8 < a.block * PIECES) threads *= 2;
  const int heads = NT / threads;
  const dim3 grid((unsigned)(a.s.max_rows / a.block + 2 * a.s.n), (unsigned)((a.Hkv + heads - 1) / heads));
  return launch_step_kernel(k_bounds<D, F32>, grid, NT, 0, 1, s, a, threads, heads);
}

}  // namespace

cudaError_t launch_bounds(const BoundsArgs& a, cudaStream_t s) {
  if (a.s.n == 0 || a.s.max_rows == 0) return cudaSuccess;
  if (a.D == 128) return a.kv_f32 ? launch_t<128, true>(a, s) : launch_t<128, false>(a, s);
  if (a.D == 64) return a.kv_f32 ? launch_t<64, true>(a, s) : launch_t<64, false>(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace gp
