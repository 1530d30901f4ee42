// The blocks that each row attends to, by the bound that its queries reach over
// their keys.  For a row and KV head h with the queries q_g of its group:
//
//   e'  = the least whole number >= -100 with max |q| <= 127 * 2^e' (at most 100)
//   Q_g = round(q_g / 2^e'),  P = sum_g max(Q_g, 0),  N = sum_g min(Q_g, 0)
//   S_b = 2^e_b (P . hi_b + N . lo_b)
// (2^e' is the same for all blocks and left out).  Of the blocks [0, own], own the
// row's, the first `sink` and the last `recent` are taken, and of the others
// those of largest S, equal ones the lower first, `top` in all; ascending.
//
// Exact.  |P|, |N| <= 4 * 127, so they are fp16 numbers as the bounds are, and
// |P . hi + N . lo| <= 127 * 127 * 4 * 128 < 2^23: every partial sum of the product
// is a whole number that fp32 holds, in any order, and a score that power of two
// times such a number.  So the lists depend on no rounding, split or launch.
//
// One product of 16 blocks by 8 rows by 2 d (mma, fp16 in, fp32 out).  The 8 bit
// bounds go from global memory into its fragments: a lane takes 16 bytes of a
// block's row, four K steps' worth (K is summed over, so its order is free as
// long as P and N follow it), made fp16 by placing each byte under the exponent of
// 1024 and subtracting.  A tile of up to 8 rows of a request shares them.
// Scores stay in shared memory; a warp picks a row's blocks: the threshold by
// halving the range of the ordered bits, then one ordered pass.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "shared_limit.cuh"
#include "step.cuh"

namespace gp {
namespace {

constexpr int NT = 128;
constexpr int ROWS = 8;  // of a tile: the product's N

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two signed bytes (the lower or the upper two of w) as fp16: 0x6400 + (byte + 128) is 1024 + byte + 128.
__device__ __forceinline__ uint32_t two_halves(uint32_t flipped, uint32_t select) {
  const uint32_t u = __byte_perm(flipped, 0x64646464u, select);
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&u), __float2half2_rn(1152.f));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The order of floats as unsigned numbers (no NaN).
__device__ __forceinline__ unsigned ordered(float f) {
  const unsigned u = __float_as_uint(f + 0.f);  // -0 is 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A warp picks `want` of the keys [from, to) of `key` (larger first, equal ones
// the lower index first) and writes the list: the blocks [0, from), those picked,
// [to, end), then -1.  Needs 0 <= want < to - from.
__device__ __forceinline__ void pick(const unsigned* key, int from, int to, int end, int want, int32_t* out, int top) {
  const int lane = threadIdx.x & 31;
  // the largest threshold that at least `want` keys reach
  unsigned at_least = 0;
  if (want > 0)
    for (int bit = 31; bit >= 0; --bit) {
      const unsigned t = at_least | (1u << bit);
      int count = 0;
      for (int b = from + lane; b < to; b += 32) count += key[b] >= t;
      count = __reduce_add_sync(0xffffffffu, count);
      if (count >= want) at_least = t;
      if (count == want) break;  // exactly these
    }
  int above = 0;
  for (int b = from + lane; b < to; b += 32) above += key[b] > at_least;
  above = __reduce_add_sync(0xffffffffu, above);
  int ties = want - above;  // of the keys that equal it; the first ones
  for (int b = lane; b < from; b += 32) out[b] = b;
  int n = from;
  for (int b0 = from; b0 < to; b0 += 32) {
    const int b = b0 + lane;
    const bool more = want > 0 && b < to && key[b] > at_least, same = want > 0 && b < to && key[b] == at_least;
    const unsigned equal = __ballot_sync(0xffffffffu, same);
    const bool taken = more || (same && __popc(equal & ((1u << lane) - 1)) < ties);
    const unsigned kept = __ballot_sync(0xffffffffu, taken);
    if (taken) out[n + __popc(kept & ((1u << lane) - 1))] = b;
    n += __popc(kept);
    ties -= min(ties, __popc(equal));
  }
  for (int b = to + lane; b < end; b += 32) out[n + b - to] = b;
  n += end - to;
  for (int k = n + lane; k < top; k += 32) out[k] = -1;
}

template <int D, int G, bool F32>
__global__ void __launch_bounds__(NT) k_block_select(const __grid_constant__ SelectBlocksArgs a, int pitch) {
  extern __shared__ __align__(16) unsigned scores[];  // [ROWS][pitch], ordered bits
  __shared__ __align__(16) __half reach[ROWS][2 * D + 8];  // N, P of the tile's rows
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.y;
  const StepPiece p = find_piece(a.s, blockIdx.x, ROWS, 1);
  if (p.r < 0 || p.at * ROWS >= p.rows) return;
  const int t0 = p.at * ROWS, m = min(ROWS, p.rows - t0);  // rows of the tile
  const StepRow first = step_row(a.s, p.r, t0, tid == 0), last = step_row(a.s, p.r, t0 + m - 1, tid == 0);
  if (!first.live || !last.live) return;
  const size_t row0 = (size_t)p.row0 + t0;

  // P and N: a warp a row
  for (int x = warp; x < ROWS; x += NT / 32) {
    constexpr int E = D / 32;  // dimensions of a lane
    float q[G][E];
    float top = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int i = 0; i < E; ++i) {
        q[g][i] = 0.f;
        if (x < m) {
          const size_t at = ((row0 + x) * a.Hq + h * G + g) * D + lane + 32 * i;
          q[g][i] = F32 ? static_cast<const float*>(a.q)[at] : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at]);
          if (q[g][i] != q[g][i]) q[g][i] = 0.f;  // NaN asks for nothing
        }
        top = fmaxf(top, fabsf(q[g][i]));
      }
#pragma unroll
    for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float down = power_of_two(-scale_exponent(top));
#pragma unroll
    for (int i = 0; i < E; ++i) {
      float neg = 0.f, pos = 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float v = fminf(fmaxf(rintf(q[g][i] * down), -127.f), 127.f);
        neg += fminf(v, 0.f);
        pos += fmaxf(v, 0.f);
      }
      reach[x][lane + 32 * i] = __float2half_rn(neg);
      reach[x][D + lane + 32 * i] = __float2half_rn(pos);
    }
  }
  __syncthreads();

  const int lb = log2_of(a.block), lper = kStepPageLog - lb;  // blocks of a page
  const int some = max(0, (last.at >> lb) + 1 - a.recent);  // blocks that a row may have to choose from
  constexpr int CHUNKS = 2 * D / 64;
  uint32_t bq[CHUNKS][4][2];
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const uint2 v = *reinterpret_cast<const uint2*>(&reach[lane >> 2][64 * c + 16 * (lane & 3) + 4 * s]);
      bq[c][s][0] = v.x;
      bq[c][s][1] = v.y;
    }
  for (int b0 = 16 * warp; b0 < some; b0 += 16 * (NT / 32)) {
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    float scale[2];
    const uint4* src[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {  // this lane's two blocks
      const int b = min(b0 + (lane >> 2) + 8 * k, some - 1);
      const int page = max(step_page(a.s, first.slot, b >> lper), 0);
      const size_t at = (((((size_t)a.layer * a.s.num_pages_total + page) * a.Hkv) + h) << lper) + (b & ((1 << lper) - 1));
      src[k] = reinterpret_cast<const uint4*>(a.bounds + at * 2 * D) + (lane & 3);
      scale[k] = a.scales[at];
    }
    uint4 w[CHUNKS][2];
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      w[c][0] = src[0][4 * c];
      w[c][1] = src[1][4 * c];
    }
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const unsigned x[4] = {w[c][0].x, w[c][0].y, w[c][0].z, w[c][0].w}, y[4] = {w[c][1].x, w[c][1].y, w[c][1].z, w[c][1].w};
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint32_t u = x[s] ^ 0x80808080u, v = y[s] ^ 0x80808080u;
        const uint32_t f[4] = {two_halves(u, 0x4140), two_halves(v, 0x4140), two_halves(u, 0x4342), two_halves(v, 0x4342)};
        mma_16816(sum, f, bq[c][s][0], bq[c][s][1]);
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int b = b0 + (lane >> 2) + 8 * k, x = 2 * (lane & 3);
      if (b < some) {
        if (x < m) scores[(size_t)x * pitch + b] = ordered(sum[2 * k] * scale[k]);
        if (x + 1 < m) scores[(size_t)(x + 1) * pitch + b] = ordered(sum[2 * k + 1] * scale[k]);
      }
    }
  }
  __syncthreads();
  for (int x = warp; x < m; x += NT / 32) {
    const int end = ((first.at + x) >> lb) + 1;  // blocks that the row sees
    int32_t* out = a.blocks + ((row0 + x) * a.Hkv + h) * a.top;
    if (end <= a.top) {
      for (int k = lane; k < a.top; k += 32) out[k] = k < end ? k : -1;
    } else {
      pick(scores + (size_t)x * pitch, a.sink, end - a.recent, end, a.top - a.sink - a.recent, out, a.top);
    }
  }
}

template <int D, int G, bool F32>
cudaError_t launch_t(const SelectBlocksArgs& a, cudaStream_t s) {
  const int pitch = a.s.maxp * (kStepPage / a.block);
  const int smem = ROWS * pitch * 4;
  cudaError_t e = allow_shared<&k_block_select<D, G, F32>>(ROWS * 4096 * 4);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(a.s.max_rows / ROWS + a.s.n), (unsigned)a.Hkv);
  k_block_select<D, G, F32><<<grid, NT, smem, s>>>(a, pitch);
  return cudaGetLastError();
}
template <int D, bool F32>
cudaError_t launch_g(const SelectBlocksArgs& a, cudaStream_t s) {
  switch (a.Hq / a.Hkv) {
    case 2: return launch_t<D, 2, F32>(a, s);
    case 4: return launch_t<D, 4, F32>(a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_select_blocks(const SelectBlocksArgs& a, cudaStream_t s) {
  if (a.s.n == 0 || a.s.max_rows == 0) return cudaSuccess;
  if (a.D == 128) return a.q_f32 ? launch_g<128, true>(a, s) : launch_g<128, false>(a, s);
  if (a.D == 64) return a.q_f32 ? launch_g<64, true>(a, s) : launch_g<64, false>(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace gp
