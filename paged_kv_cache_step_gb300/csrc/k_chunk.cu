// Causal attention of several new tokens a request over the paged cache, and
// the accumulated weights of it, on the CUDA cores (fp32 FMA): fp32 caches or
// queries, and every shape when it is asked for.  k_chunk_tc.cu has the
// tensor-core kernels.
//
// Token t of request r (query rows rotated, packed) sees the logical slots
// [0, cached + t + 1):  z = q . k / sqrt(d), a = softmax(z), out = sum a v,
// and W_i += sum over the tokens and the group's heads of a_i.
//
// A query row here is a (token, head of the group) pair: the G heads of a KV
// head share its keys, so a tile of 64 rows is 64 / G tokens.
//   attention  one CTA a tile: key tiles of 64 through shared memory, S by
//              4 x 4 register tiles, softmax in base 2 with a running maximum
//              and sum, out += P V.  Slots past the last token may hold any
//              bits; their V rows are zeroed as they are read.
//   weights    the sums over a column need every row's final maximum and sum,
//              so S is formed again, one CTA a tile of 64 keys, over the query
//              tiles that see it: a weight has one writer, and the sum's order
//              is fixed.
// Few tiles are cut into several items each, over the keys (weights: over the
// query tiles), to fill the SMs; their partials are joined by a kernel more.
// Bounded by the fp32 pipe: 2 d (2 + 1) flops a (row, key) pair.  The next K, V
// or query tile is on its way, in registers, while one is at work, and the FMAs
// are issued two at a time: 8000 tokens, 32 query and 8 KV heads, d = 128, fp32
// take 12.5 ms of attention (42 TFLOP/s) and 6.6 ms of weights (8.0 ms without),
// two requests of 1000 tokens behind 300, 16 and 8 heads, d = 64, 229 and 131 us
// (317 and 146).
#include <cuda_bf16.h>

#include <cstdint>

#include "chained.cuh"
#include "math2.cuh"
#include "weighted_kernels.h"

namespace gp {
namespace {

constexpr int NT = 256;  // 16 x 16 threads
constexpr int PAGE = 256;
constexpr int BR = CHUNK_ROWS, BK = CHUNK_KEYS;
constexpr float NEG = -1.0e30f;
static_assert(BR == 64 && BK == 64 && PAGE % BK == 0, "4 x 4 outputs a thread");

template <int D>
struct Smem {
  static constexpr int LD = D + 4;  // floats of a staged row: rows 4 banks apart
  float q[BR][LD];
  float kv[BK][LD];
  float p[BR][BK + 4];
  float m[BR], l[BR], f[BR];  // maximum, sum, the tile's rescale factor
};

template <bool F32>
__device__ __forceinline__ float4 load4(const void* base, size_t elt) {
  if constexpr (F32) {
    return *reinterpret_cast<const float4*>(static_cast<const float*>(base) + elt);
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(base) + elt);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
  }
}

// A thread's pieces of 64 rows of queries, K or V: fetched while the tile before
// is at work, put into shared memory when that is done.
template <int D>
struct Pieces {
  static constexpr int N = 64 * D / 4 / NT;
  float4 x[N];
  static __device__ __forceinline__ int row(int i) { return (threadIdx.x + i * NT) / (D / 4); }
  static __device__ __forceinline__ int col(int i) { return (threadIdx.x + i * NT) % (D / 4) * 4; }
  __device__ __forceinline__ void put(float (*dst)[D + 4]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) *reinterpret_cast<float4*>(&dst[row(i)][col(i)]) = x[i];
  }
};

// 64 query rows from token t0, scaled to base 2; rows past the request are 0.
template <int D>
__device__ __forceinline__ void fetch_rows(const ChunkArgs& a, const ChunkReq& rq, int h, int t0, Pieces<D>& to) {
  const float sc = 1.4426950408889634f / sqrtf((float)D);
#pragma unroll
  for (int i = 0; i < Pieces<D>::N; ++i) {
    const int row = Pieces<D>::row(i), t = t0 + row / a.G;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t < rq.nnew) {
      const size_t at = ((size_t)(rq.row0 + t) * a.Hq + h * a.G + row % a.G) * D + Pieces<D>::col(i);
      x = a.q_f32 ? load4<true>(a.q, at) : load4<false>(a.q, at);
    }
    to.x[i] = make_float4(sc * x.x, sc * x.y, sc * x.z, sc * x.w);
  }
}

// 64 rows of K or V from logical slot s0; rows from `total` on are 0.
template <int D>
__device__ __forceinline__ void fetch_keys(const ChunkArgs& a, const ChunkReq& rq, const void* cache, int h, int s0,
                                           int total, Pieces<D>& to) {
  int page = a.bt[rq.bt_off + s0 / PAGE];
  if (page < 0 || page >= a.num_pages_total) {
    if (threadIdx.x == 0) atomicOr(a.err, ERR_BAD_PAGE);
    page = 0;
  }
  const size_t base = ((((size_t)a.layer * a.num_pages_total + page) * a.Hkv + h) * PAGE + s0 % PAGE) * D;
#pragma unroll
  for (int i = 0; i < Pieces<D>::N; ++i) {
    const int row = Pieces<D>::row(i);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (s0 + row < total) {
      const size_t at = base + (size_t)row * D + Pieces<D>::col(i);
      x = a.kv_f32 ? load4<true>(cache, at) : load4<false>(cache, at);
    }
    to.x[i] = x;
  }
}

// s[i][j] = q row 4 ty + i . key tx + 16 j: the even and the odd products apart,
// two a step
template <int D>
__device__ __forceinline__ void scores(const Smem<D>& sm, int ty, int tx, float s[4][4]) {
  float2 z[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) z[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int d = 0; d < D; d += 4) {
    float4 q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = *reinterpret_cast<const float4*>(&sm.q[4 * ty + i][d]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 k = *reinterpret_cast<const float4*>(&sm.kv[tx + 16 * j][d]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        z[i][j] = fma2(make_float2(q[i].x, q[i].y), make_float2(k.x, k.y), z[i][j]);
        z[i][j] = fma2(make_float2(q[i].z, q[i].w), make_float2(k.z, k.w), z[i][j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = z[i][j].x + z[i][j].y;
}

template <int D>
__global__ void __launch_bounds__(NT, 2) k_chunk(const __grid_constant__ ChunkArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(raw);
  constexpr int DC = D / 64;  // float4 columns of the output a thread owns
  const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
  const ChunkTile tile = a.tiles[blockIdx.x];
  let_next_in();
  const ChunkReq rq = a.reqs[tile.r];
  const int total = rq.cached + rq.nnew;
  const int tokens = BR / a.G;
  const int last = min(tile.first + tokens, rq.nnew) - 1;  // last token of the tile
  const int end = min(rq.cached + last + 1, tile.to * BK);  // slots it sees, of this item
  Pieces<D> next, rows;
  fetch_keys<D>(a, rq, a.k_cache, tile.h, tile.from * BK, total, next);
  fetch_rows<D>(a, rq, tile.h, tile.first, rows);
  rows.put(sm.q);
  if (tid < BR) {
    sm.m[tid] = NEG;
    sm.l[tid] = 0.f;
  }
  float2 acc[4][DC][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < DC; ++c) acc[i][c][0] = acc[i][c][1] = make_float2(0.f, 0.f);
  for (int s0 = tile.from * BK; s0 < end; s0 += BK) {
    __syncthreads();  // the last tile's V and P are used
    next.put(sm.kv);
    __syncthreads();
    fetch_keys<D>(a, rq, a.v_cache, tile.h, s0, total, next);
    float s[4][4];
    scores<D>(sm, ty, tx, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 4 * ty + i;
      const int sees = rq.cached + tile.first + row / a.G;  // last slot the row sees
      float mx = NEG;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (s0 + tx + 16 * j > sees) s[i][j] = -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float old = sm.m[row], mn = fmaxf(old, mx);  // NEG while the row has seen no slot: its P is 0
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = ex2f(s[i][j] - mn);
        sm.p[row][tx + 16 * j] = p;
        sum += p;
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      __syncwarp();  // the row's old maximum has been read by its 16 threads
      if (tx == 0) {
        const float f = ex2f(old - mn);
        sm.f[row] = f;
        sm.m[row] = mn;
        sm.l[row] = fmaf(sm.l[row], f, sum);
      }
    }
    __syncthreads();  // K is used, P and the factors are written
    next.put(sm.kv);
    __syncthreads();
    if (s0 + BK < end) fetch_keys<D>(a, rq, a.k_cache, tile.h, s0 + BK, total, next);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = sm.f[4 * ty + i];
#pragma unroll
      for (int c = 0; c < DC; ++c)
#pragma unroll
        for (int x = 0; x < 2; ++x) acc[i][c][x] = mul2(acc[i][c][x], make_float2(f, f));
    }
    // four keys' weights a load: one at a time the reads of P alone took as long
    // as the FMAs
#pragma unroll 2
    for (int k = 0; k < BK; k += 4) {
      float p[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(&sm.p[4 * ty + i][k]);
        p[i][0] = x.x; p[i][1] = x.y; p[i][2] = x.z; p[i][3] = x.w;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int c = 0; c < DC; ++c) {
          const float4 v = *reinterpret_cast<const float4*>(&sm.kv[k + e][64 * c + 4 * tx]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 w = make_float2(p[i][e], p[i][e]);
            acc[i][c][0] = fma2(w, make_float2(v.x, v.y), acc[i][c][0]);
            acc[i][c][1] = fma2(w, make_float2(v.z, v.w), acc[i][c][1]);
          }
        }
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 4 * ty + i, t = tile.first + row / a.G;
    if (t >= rq.nnew) continue;
    if (tile.part >= 0) {
      float* po = a.part + (size_t)tile.part * chunk_tile_part_floats(D);
#pragma unroll
      for (int c = 0; c < DC; ++c)
        *reinterpret_cast<float4*>(po + (size_t)row * D + 64 * c + 4 * tx) =
            make_float4(acc[i][c][0].x, acc[i][c][0].y, acc[i][c][1].x, acc[i][c][1].y);
      if (tx == 0) {
        po[BR * D + row] = sm.m[row];
        po[BR * D + BR + row] = sm.l[row];
      }
      continue;
    }
    const int g = tile.h * a.G + row % a.G;
    const size_t at = (size_t)(rq.row0 + t) * a.Hq + g;
    const float inv = 1.f / sm.l[row];
    if (tx == 0 && a.stat) a.stat[at] = make_float2(sm.m[row], inv);
#pragma unroll
    for (int c = 0; c < DC; ++c) {
      const float o[4] = {acc[i][c][0].x * inv, acc[i][c][0].y * inv, acc[i][c][1].x * inv, acc[i][c][1].y * inv};
      const size_t e = at * D + 64 * c + 4 * tx;
      if (a.q_f32) {
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + e) = make_float4(o[0], o[1], o[2], o[3]);
      } else {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(o[0], o[1]), hi = __floats2bfloat162_rn(o[2], o[3]);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + e) =
            make_uint2(*reinterpret_cast<const unsigned*>(&lo), *reinterpret_cast<const unsigned*>(&hi));
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(NT) k_chunk_weights(const __grid_constant__ ChunkArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(raw);
  const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
  const ChunkTile tile = a.wtiles[blockIdx.x];
  let_next_in();
  const ChunkReq rq = a.reqs[tile.r];
  const int total = rq.cached + rq.nnew;
  const int tokens = BR / a.G, s0 = tile.first;
  if (rq.slot < 0 || rq.slot >= a.M) return;
  wait_for_previous();
  Pieces<D> rows;
  fetch_keys<D>(a, rq, a.k_cache, tile.h, s0, total, rows);
  rows.put(sm.kv);
  float w[4] = {0.f, 0.f, 0.f, 0.f};
  const int end = min(tile.to * tokens, rq.nnew);
  float2 st = make_float2(0.f, 0.f);
  auto fetch = [&](int t0) {
    fetch_rows<D>(a, rq, tile.h, t0, rows);
    const int t = t0 + tid / a.G;
    if (tid < BR) st = t < rq.nnew ? a.stat[(size_t)(rq.row0 + t) * a.Hq + tile.h * a.G + tid % a.G] : make_float2(0.f, 0.f);
  };
  fetch(tile.from * tokens);
  for (int t0 = tile.from * tokens; t0 < end; t0 += tokens) {
    __syncthreads();  // the last tile's rows are used
    rows.put(sm.q);
    if (tid < BR) {
      sm.m[tid] = st.x;
      sm.l[tid] = st.y;
    }
    __syncthreads();
    if (t0 + tokens < end) fetch(t0 + tokens);
    float s[4][4];
    scores<D>(sm, ty, tx, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 4 * ty + i, t = t0 + row / a.G;
      const float m = sm.m[row], inv = sm.l[row];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (t < rq.nnew && s0 + tx + 16 * j <= rq.cached + t) w[j] = fmaf(ex2f(s[i][j] - m), inv, w[j]);
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; ++j) sm.p[ty][tx + 16 * j] = w[j];
  __syncthreads();
  if (tid < BK && s0 + tid < total) {
    float sum = 0.f;
#pragma unroll
    for (int y = 0; y < 16; ++y) sum += sm.p[y][tid];
    if (tile.part >= 0) a.wpart[(size_t)tile.part * BK + tid] = sum;
    else a.weights[(((size_t)a.layer * a.M + rq.slot) * a.Hkv + tile.h) * a.cap + s0 + tid] += sum;
  }
}

// Joins the partials of a query tile: thread = four dimensions of a row.
template <int D>
__global__ void __launch_bounds__(D / 4) k_chunk_tile_join(const __grid_constant__ ChunkArgs a) {
  const ChunkTileJoin jn = a.joins[blockIdx.x];
  let_next_in();
  wait_for_previous();
  const ChunkReq rq = a.reqs[jn.r];
  const int row = blockIdx.y, t = jn.first + row / a.G;
  if (t >= rq.nnew) return;
  const float* base = a.part + (size_t)jn.part * chunk_tile_part_floats(D);
  float M = NEG;
#pragma unroll 8
  for (int p = 0; p < jn.n; ++p) M = fmaxf(M, __ldcg(base + p * chunk_tile_part_floats(D) + BR * D + row));
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int p = 0; p < jn.n; ++p) {
    const float* q = base + p * chunk_tile_part_floats(D);
    const float f = ex2f(__ldcg(q + BR * D + row) - M);  // 0 for a part of which the row sees nothing
    const float4 x = __ldcg(reinterpret_cast<const float4*>(q + (size_t)row * D) + threadIdx.x);
    l = fmaf(f, __ldcg(q + BR * D + BR + row), l);
    o = make_float4(fmaf(f, x.x, o.x), fmaf(f, x.y, o.y), fmaf(f, x.z, o.z), fmaf(f, x.w, o.w));
  }
  const float inv = 1.f / l;
  const size_t at = (size_t)(rq.row0 + t) * a.Hq + jn.h * a.G + row % a.G;
  if (threadIdx.x == 0 && a.stat) a.stat[at] = make_float2(M, inv);
  const size_t e = at * D + 4 * threadIdx.x;
  if (a.q_f32) {
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + e) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv), hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + e) =
        make_uint2(*reinterpret_cast<const unsigned*>(&lo), *reinterpret_cast<const unsigned*>(&hi));
  }
}

// Adds the partial sums of a key tile, in the order of its parts.
__global__ void __launch_bounds__(BK) k_chunk_tile_weights_join(const __grid_constant__ ChunkArgs a) {
  const ChunkTileJoin jn = a.wjoins[blockIdx.x];
  wait_for_previous();
  const ChunkReq rq = a.reqs[jn.r];
  const int i = jn.first + (int)threadIdx.x;
  if (i >= rq.cached + rq.nnew || rq.slot < 0 || rq.slot >= a.M) return;
  float* dst = a.weights + (((size_t)a.layer * a.M + rq.slot) * a.Hkv + jn.h) * a.cap + i;
  const float so_far = *dst;
  float w = 0.f;
#pragma unroll 8
  for (int p = 0; p < jn.n; ++p) w += __ldcg(a.wpart + (size_t)(jn.part + p) * BK + threadIdx.x);
  *dst = so_far + w;
}

cudaError_t launch_k(void (*kernel)(ChunkArgs), size_t smem, int grid, bool chained, const ChunkArgs& a, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  if (chained) return launch_chained(kernel, dim3((unsigned)grid), NT, smem, s, a);
  kernel<<<dim3((unsigned)grid), NT, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_chunk(const ChunkArgs& a, cudaStream_t s) {
  if (a.n_tiles == 0) return cudaSuccess;
  if (a.G < 1 || BR % a.G || (a.D != 64 && a.D != 128)) return cudaErrorInvalidValue;
  const cudaError_t e = a.D == 128 ? launch_k(k_chunk<128>, sizeof(Smem<128>), a.n_tiles, false, a, s)
                                   : launch_k(k_chunk<64>, sizeof(Smem<64>), a.n_tiles, false, a, s);
  if (e != cudaSuccess || a.n_joins == 0) return e;
  const dim3 grid((unsigned)a.n_joins, BR);
  return a.D == 128 ? launch_chained(k_chunk_tile_join<128>, grid, 32, 0, s, a)
                    : launch_chained(k_chunk_tile_join<64>, grid, 16, 0, s, a);
}

cudaError_t launch_chunk_weights(const ChunkArgs& a, cudaStream_t s) {
  if (a.n_wtiles == 0) return cudaSuccess;
  if (a.G < 1 || BR % a.G || (a.D != 64 && a.D != 128)) return cudaErrorInvalidValue;
  const cudaError_t e = a.D == 128 ? launch_k(k_chunk_weights<128>, sizeof(Smem<128>), a.n_wtiles, true, a, s)
                                   : launch_k(k_chunk_weights<64>, sizeof(Smem<64>), a.n_wtiles, true, a, s);
  if (e != cudaSuccess || a.n_wjoins == 0) return e;
  return launch_chained(k_chunk_tile_weights_join, dim3((unsigned)a.n_wjoins), BK, 0, s, a);
}

}  // namespace gp
