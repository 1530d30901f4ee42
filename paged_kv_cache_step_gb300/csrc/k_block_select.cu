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
// Scores stay in shared memory; a warp picks a row's blocks with their keys in
// registers: the threshold bit by bit from the highest that differs, then one ordered
// pass.  Few tiles are shared by a cluster, whose scores go to its first CTA.
//
// Measured (32 + 8 heads, d = 128, blocks of 64, 32 of them): a decode step of 64 requests of
// 4 to 128 pages 13.5 us in a graph, where reading the bounds takes 4.5: latency; 4001 rows behind
// 12 007 tokens 57 us, bounded by instruction issue.  On the way: tiles of 8 rows, keys read from shared
// memory for every bit 141 us; in registers, tiles of 16 80 us; the products' row operand from
// shared memory, so that three CTAs fit on an SM, 64 us; four, at 64 registers a thread, 57 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "shared_limit.cuh"
#include "step.cuh"

namespace gp {
namespace {

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

// How many of a warp's keys reach t.
template <int N>
__device__ __forceinline__ int reaching(const unsigned (&key)[N], unsigned t) {
  int count = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) count += key[i] >= t;
  return __reduce_add_sync(0xffffffffu, count);
}

// The threshold that picks `want` >= 1 of a warp's keys, of more: the largest that at
// least so many reach; `ties`: how many of those that equal it are picked (all
// that reach it: -1).  Bit by bit from the highest in which the keys differ; two keys
// that are a part in 250 of their range apart need some ten bits.
template <typename Count>
__device__ __forceinline__ unsigned threshold(unsigned low, unsigned high, int want, int& ties, Count&& count) {
  ties = -1;
  if (low == high) {
    ties = want;
    return low;
  }
  const int top = 31 - __clz(low ^ high);
  unsigned t = high >> top >> 1 << top << 1;  // the bits that all keys share
  for (int bit = top; bit >= 0; --bit) {
    const int n = count(t | 1u << bit);
    if (n >= want) t |= 1u << bit;
    if (n == want) return t;
  }
  ties = want - (t == 0xffffffffu ? 0 : count(t + 1));
  return t;
}

// A warp picks `want` of the keys [from, to) (larger first, equal ones the lower index
// first) and writes the list: the blocks [0, from), those picked, [to, end), then -1.
// Needs 0 <= want < to - from <= 32 N.
template <int N>
__device__ __forceinline__ void pick(const unsigned* keys, int from, int to, int end, int want, int32_t* out, int top) {
  const int lane = threadIdx.x & 31;
  unsigned key[N], low = 0xffffffffu, high = 0u;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int b = from + 32 * i + lane;
    key[i] = b < to ? keys[b] : 0u;  // (no score is 0: the bits of a NaN)
    if (b < to) {
      low = min(low, key[i]);
      high = max(high, key[i]);
    }
  }
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  int ties = 0;
  unsigned t = 0xffffffffu;
  if (want > 0) t = threshold(low, high, want, ties, [&](unsigned x) { return reaching(key, x); });
  for (int b = lane; b < from; b += 32) out[b] = b;
  int n = from;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    bool taken = key[i] > t || (ties < 0 && key[i] == t);
    if (ties > 0) {
      const unsigned equal = __ballot_sync(0xffffffffu, key[i] == t);
      taken = taken || (key[i] == t && __popc(equal & ((1u << lane) - 1)) < ties);
      ties -= min(ties, __popc(equal));
    }
    const unsigned kept = __ballot_sync(0xffffffffu, taken);
    if (taken) out[n + __popc(kept & ((1u << lane) - 1))] = from + 32 * i + lane;
    n += __popc(kept);
  }
  for (int b = to + lane; b < end; b += 32) out[n + b - to] = b;
  n += end - to;
  for (int k = n + lane; k < top; k += 32) out[k] = -1;
}

// The same for more keys than registers hold.
__device__ __forceinline__ void pick_many(const unsigned* key, int from, int to, int end, int want, int32_t* out, int top) {
  const int lane = threadIdx.x & 31;
  unsigned low = 0xffffffffu, high = 0u;
  for (int b = from + lane; b < to; b += 32) {
    low = min(low, key[b]);
    high = max(high, key[b]);
  }
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  int ties = 0;
  unsigned t = 0xffffffffu;
  if (want > 0)
    t = threshold(low, high, want, ties, [&](unsigned x) {
      int count = 0;
      for (int b = from + lane; b < to; b += 32) count += key[b] >= x;
      return __reduce_add_sync(0xffffffffu, count);
    });
  for (int b = lane; b < from; b += 32) out[b] = b;
  int n = from;
  for (int b0 = from; b0 < to; b0 += 32) {
    const int b = b0 + lane;
    const unsigned k = b < to ? key[b] : 0u;
    bool taken = k > t || (ties < 0 && k == t);
    if (ties > 0) {
      const unsigned equal = __ballot_sync(0xffffffffu, k == t);
      taken = taken || (k == t && __popc(equal & ((1u << lane) - 1)) < ties);
      ties -= min(ties, __popc(equal));
    }
    const unsigned kept = __ballot_sync(0xffffffffu, taken);
    if (taken) out[n + __popc(kept & ((1u << lane) - 1))] = b;
    n += __popc(kept);
  }
  for (int b = to + lane; b < end; b += 32) out[n + b - to] = b;
  n += end - to;
  for (int k = n + lane; k < top; k += 32) out[k] = -1;
}

// ROWS: of a tile, 8 or 16.  Tiles of 8 rows (decode steps) wait on memory: half as
// many warps, each with the bounds of 32 blocks in flight, so that a step's tiles
// are on the GPU together.
template <int D, int G, bool F32, int ROWS>
__global__ void __launch_bounds__(16 * ROWS, 4) k_block_select(const __grid_constant__ SelectBlocksArgs a, int pitch) {
  constexpr int NT = 16 * ROWS, NW = NT / 32;
  constexpr int AHEAD = ROWS == 8 ? 2 : 1;  // products of 16 blocks whose bounds are loaded together
  constexpr int QR = ROWS / NW;             // rows of Q a warp
  constexpr int NN = ROWS / 8;  // products of 8 rows
  extern __shared__ __align__(16) unsigned scores[];  // [ROWS][pitch], ordered bits
  __shared__ __align__(16) __half reach[ROWS][2 * D + 4];  // N, P of the tile's rows (520 bytes apart: no bank twice)
  __shared__ int pages[256];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = a.splits, rank = blockIdx.x % C, item = blockIdx.x / C, h = item % a.Hkv;
  begin_step();
  const StepPiece p = find_piece(a.s, item / a.Hkv, log2_const(ROWS), 1, tid == 0);
  if (p.r < 0 || p.at * ROWS >= p.rows) return;  // (the whole cluster)
  const int t0 = p.at * ROWS, m = min(ROWS, p.rows - t0);  // rows of the tile
  const size_t row0 = (size_t)p.row0 + t0;

  // the rows' queries, a warp a row: loaded while their places are looked up
  constexpr int E = D / 32;  // dimensions of a lane
  float q[QR][G][E];
  int named[QR];
#pragma unroll
  for (int i = 0; i < QR; ++i) {
    const int x = warp + NW * i;
    named[i] = x < m ? a.s.row_req[row0 + x] : -1;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const size_t at = ((row0 + x) * a.Hq + h * G + g) * D + E * lane;
#pragma unroll
      for (int e = 0; e < E; ++e) q[i][g][e] = 0.f;
      if (x < m) {
        if constexpr (F32) {
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const float2 v = *reinterpret_cast<const float2*>(static_cast<const float*>(a.q) + at + e);
            q[i][g][e] = v.x;
            q[i][g][e + 1] = v.y;
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const unsigned v = *reinterpret_cast<const unsigned*>(static_cast<const __nv_bfloat16*>(a.q) + at + e);
            q[i][g][e] = __uint_as_float(v << 16);
            q[i][g][e + 1] = __uint_as_float(v & 0xffff0000u);
          }
        }
      }
    }
  }
  const int first = p.cached + t0, last = first + m - 1;  // the rows' slots
  if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int lb = log2_of(a.block), lper = kStepPageLog - lb;  // blocks of a page
  const int some = max(0, (last >> lb) + 1 - a.recent);    // blocks that a row may have to choose from
  for (int i = tid; i << lper < some; i += NT) pages[i] = max(step_page(a.s, p.slot, i), 0);

#pragma unroll
  for (int i = 0; i < QR; ++i) {
    float top = 0.f, odd = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        top = fmaxf(top, fabsf(q[i][g][e]));
        odd = fmaf(q[i][g][e], 0.f, odd);
      }
    if (odd != 0.f) {  // NaN asks for nothing
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (q[i][g][e] != q[i][g][e]) q[i][g][e] = 0.f;
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float down = power_of_two(-scale_exponent(top));
    float neg[E], pos[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      neg[e] = pos[e] = 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        // to the nearest whole number, ties to even: 1.5 * 2^23 has no room for more
        const float v = fminf(fmaxf(q[i][g][e] * down, -127.f), 127.f) + 12582912.f - 12582912.f;
        neg[e] += v;
        pos[e] += fmaxf(v, 0.f);
      }
      neg[e] -= pos[e];
    }
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      *reinterpret_cast<__half2*>(&reach[warp + NW * i][E * lane + e]) = __floats2half2_rn(neg[e], neg[e + 1]);
      *reinterpret_cast<__half2*>(&reach[warp + NW * i][D + E * lane + e]) = __floats2half2_rn(pos[e], pos[e + 1]);
    }
  }
  __syncthreads();

  constexpr int CHUNKS = 2 * D / 64;
  const __half* mine = &reach[lane >> 2][16 * (lane & 3)];
  uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(scores));  // of the cluster's first CTA
  if (C > 1) {
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(to) : "r"(to));
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // it has started
  }
  auto put = [&](int x, int b, float v) {
    const uint32_t at = to + 4u * (uint32_t)(x * pitch + b);
    if (C > 1) asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(ordered(v)) : "memory");
    else asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(ordered(v)) : "memory");
  };
  const int stride = 16 * NW * C;
  for (int b0 = 16 * (warp + NW * rank); b0 < some; b0 += AHEAD * stride) {
    float scale[AHEAD][2];
    uint4 w[AHEAD][CHUNKS][2];
#pragma unroll
    for (int t = 0; t < AHEAD; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // this lane's two blocks
        const int b = min(b0 + t * stride + (lane >> 2) + 8 * k, some - 1);
        const size_t at = (((((size_t)a.layer * a.s.num_pages_total + pages[b >> lper]) * a.Hkv) + h) << lper) + (b & ((1 << lper) - 1));
        const uint4* src = reinterpret_cast<const uint4*>(a.bounds + at * 2 * D) + (lane & 3);
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) w[t][c][k] = src[4 * c];
        scale[t][k] = a.scales[at];
      }
#pragma unroll
    for (int t = 0; t < AHEAD; ++t) {
      float sum[NN][4];
#pragma unroll
      for (int i = 0; i < NN; ++i) sum[i][0] = sum[i][1] = sum[i][2] = sum[i][3] = 0.f;
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) {
        const uint4 &x4 = w[t][c][0], &y4 = w[t][c][1];
        const unsigned x[4] = {x4.x, x4.y, x4.z, x4.w}, y[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const uint32_t u = x[s] ^ 0x80808080u, v = y[s] ^ 0x80808080u;
          const uint32_t f[4] = {two_halves(u, 0x4140), two_halves(v, 0x4140), two_halves(u, 0x4342), two_halves(v, 0x4342)};
#pragma unroll
          for (int i = 0; i < NN; ++i) {
            const uint2 v2 = *reinterpret_cast<const uint2*>(mine + 8 * i * (2 * D + 4) + 64 * c + 4 * s);
            mma_16816(sum[i], f, v2.x, v2.y);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < NN; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int b = b0 + t * stride + (lane >> 2) + 8 * k, x = 8 * i + 2 * (lane & 3);
          if (b < some) {
            if (x < m) put(x, b, sum[i][2 * k] * scale[t][k]);
            if (x + 1 < m) put(x + 1, b, sum[i][2 * k + 1] * scale[t][k]);
          }
        }
    }
  }
  if (C > 1) {
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (rank > 0) return;
  } else {
    __syncthreads();
  }
  unsigned live = 0u;
#pragma unroll
  for (int i = 0; i < QR; ++i) live |= (unsigned)row_named(a.s, named[i], p.r) << i;
#pragma unroll 1
  for (int i = 0; i < QR; ++i) {
    if (!(live >> i & 1u)) continue;
    const int x = warp + NW * i, end = ((first + x) >> lb) + 1;  // blocks that the row sees
    int32_t* out = a.blocks + ((row0 + x) * a.Hkv + h) * a.top;
    const unsigned* keys = scores + (size_t)x * pitch;
    const int to_b = end - a.recent, n = to_b - a.sink, want = a.top - a.sink - a.recent;
    if (end <= a.top) {
      for (int k = lane; k < a.top; k += 32) out[k] = k < end ? k : -1;
    } else if (n <= 128) {
      pick<4>(keys, a.sink, to_b, end, want, out, a.top);
    } else if (n <= 256) {
      pick<8>(keys, a.sink, to_b, end, want, out, a.top);
    } else if (n <= 512) {
      pick<16>(keys, a.sink, to_b, end, want, out, a.top);
    } else {
      pick_many(keys, a.sink, to_b, end, want, out, a.top);
    }
  }
}

template <int D, int G, bool F32, int ROWS>
cudaError_t launch_t(const SelectBlocksArgs& a, cudaStream_t s) {
  const int pitch = a.s.maxp * (kStepPage / a.block);
  cudaError_t e = allow_shared<&k_block_select<D, G, F32, ROWS>>(ROWS == 8 ? 8 * 4096 * 4 : kSelectShared);
  if (e != cudaSuccess) return e;
  return launch_step_kernel(k_block_select<D, G, F32, ROWS>, dim3((unsigned)(sparse_pieces(a.s, ROWS) * a.Hkv * a.splits)), 16 * ROWS, (size_t)ROWS * pitch * 4, a.splits, s, a, pitch);
}
template <int D, bool F32>
cudaError_t launch_g(const SelectBlocksArgs& a, cudaStream_t s) {
  const bool four = a.Hq / a.Hkv == 4;
  if (a.rows == 16) return four ? launch_t<D, 4, F32, 16>(a, s) : launch_t<D, 2, F32, 16>(a, s);
  return four ? launch_t<D, 4, F32, 8>(a, s) : launch_t<D, 2, F32, 8>(a, s);
}

}  // namespace

cudaError_t launch_select_blocks(const SelectBlocksArgs& a, cudaStream_t s) {
  if (a.s.n == 0 || a.s.max_rows == 0) return cudaSuccess;
  if (a.D == 128) return a.q_f32 ? launch_g<128, true>(a, s) : launch_g<128, false>(a, s);
  if (a.D == 64) return a.q_f32 ? launch_g<64, true>(a, s) : launch_g<64, false>(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace gp
