// Attention over listed blocks for one or a few rows of a request (decode steps,
// drafted tokens), bf16 caches and queries.  The formulas are k_sparse.cu's.
//
// Bounded by HBM: K and V of the listed blocks are read once for the 16 / G rows
// of a piece, whose G heads make the 16 rows of the product's A operand (mma with
// m = 16: a decode step fills G of them, at no cost: the products take a
// tenth of the time that the bytes do).  tcgen05 has nothing to add at M = 16.
//
// A cluster of `splits` CTAs a (piece, KV head).  Every CTA marks the blocks that
// the piece's rows list, as bits, and takes an even share of the blocks marked by
// any; a block's rows are those that list it.  (Of a single row the list itself.)  One warp streams the share through a ring of
// stages of 64 keys, K and V, by TMA (a box is a block of up to 64 tokens, 128-byte
// swizzle).  Four warps take 16 keys of a stage each:
//   S = Q K^T   16 x 16, ldmatrix of K
//   P = 2^(S c - m), c = log2(e) / sqrt(d), in two bf16 parts (2^-16 of a weight is
//   left; the output's own rounding is 2^-8), the running m and sum l in fp32
//   O += P V    16 x d, ldmatrix.trans of V, fp32 in registers
// with a maximum of its own a warp.  Warps and then the CTAs of the cluster are
// joined in shared memory: no scratch, no second launch, one fixed order.
//
// Measured (32 + 8 heads, d = 128, 32 blocks of 64): a decode step of 64 requests 88 us, 89 % of the
// copy rate (433 us on the CUDA cores); one request with 64 blocks 12.1 us, 8 of them from
// start to end of a CTA.  Two CTAs share an SM while a launch takes up to 115 KB of
// shared memory (d = 128: 110 KB with blocks of 64; 121 KB with G = 2, 256 pages and blocks
// of 16, where one fits).  A stage takes a CTA alone 1200 clocks, two on an SM 2300: memory.
#include <cuda_bf16.h>

#include <cstdint>

#include "math2.cuh"
#include "shared_limit.cuh"
#include "sparse_tc.cuh"

#include <algorithm>

namespace gp {
namespace {

using namespace tc;

constexpr int WARPS = 4;              // that compute
constexpr int NT = 32 * (WARPS + 1);  // and one that loads
constexpr int KEYS = 64;              // of a stage
constexpr int NST = 3;
constexpr float NEG = -1.0e30f;

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int D>
struct Sm {
  static constexpr int HALF = KEYS * 128;          // 64 dimensions of a stage's keys
  static constexpr int TILE = D / 64 * HALF;       // K or V of a stage
  static constexpr int RING = NST * 2 * TILE;
  static constexpr int PART = RING;                // float [16][D + 2]
  static constexpr int SEEN = PART + 16 * (D + 2) * 4;
  // then: int page[256]; unsigned any[words], seen[T][words]; int2 list[entries]
};

template <int D, int G>
__global__ void __launch_bounds__(NT, 2) k_sparse_mma(const __grid_constant__ SparseArgs a, const __grid_constant__ SparseMaps maps,
                                                      int words) {
  using L = Sm<D>;
  constexpr int T = 16 / G;  // rows of a piece
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = static_cast<uint32_t>(__cvta_generic_to_shared(sm));
  float* part = reinterpret_cast<float*>(sm + L::PART);
  int* pages = reinterpret_cast<int*>(sm + L::SEEN);  // first key row of a page in the map; -1
  unsigned* any_s = reinterpret_cast<unsigned*>(pages + 256);
  unsigned* seen = any_s + words;
  int2* list = reinterpret_cast<int2*>(any_s + (((T + 1) * words + 1) & ~1));  // first key row in the map; block | rows << 16
  __shared__ __align__(8) uint64_t bars[2 * NST];
  __shared__ int abort_s, total_s;
  __shared__ float m_s[WARPS][16], l_s[WARPS][16];
  volatile int* abort = &abort_s;
  const uint32_t bar0 = static_cast<uint32_t>(__cvta_generic_to_shared(bars));
  auto full = [&](int s) { return bar0 + 8u * (uint32_t)s; };
  auto empty = [&](int s) { return bar0 + 8u * (uint32_t)(NST + s); };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = a.splits, rank = blockIdx.x % C, unit = blockIdx.x / C, h = unit % a.Hkv;

  if (tid == NT - 1) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.v)) : "memory");
  }
  begin_step();
  const StepPiece p = find_piece(a.s, unit / a.Hkv, log2_const(T), 1, tid == 0);
  if (p.r < 0 || p.at * T >= p.rows) return;  // (the whole cluster)
  const int t0 = p.at * T, m = min(T, p.rows - t0);
  BlockLists<WARPS + 1, T> lists;
  lists.load(a, (size_t)p.row0 + t0, h, lists.rows_of(m), 0);
  const int first_at = p.cached + t0, last_at = first_at + m - 1;  // the rows' slots
  const size_t row0 = (size_t)p.row0 + t0;
  const int named = lane < m ? a.s.row_req[row0 + lane] : -1;
  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), WARPS);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    abort_s = 0;
  }
  for (int i = tid; i < (T + 1) * words; i += NT) any_s[i] = 0u;
  for (int i = tid; i <= last_at / kStepPage; i += NT) {
    const int page = a.s.tables[(size_t)p.slot * a.s.maxp + i];
    pages[i] = page >= 0 && page < a.s.num_pages_total
                   ? (int)((((size_t)a.layer * a.s.num_pages_total + page) * a.Hkv + h) * kStepPage) : -1;
  }
  __syncthreads();
  const unsigned live = __ballot_sync(0xffffffffu, row_named(a.s, named, p.r));  // the same in every warp
  if (!live) return;  // (the whole cluster)
  const int lb = log2_of(a.block), lper = kStepPageLog - lb;  // blocks of a page
  // this lane's rows of Q: (row / G)-th of the piece, head row % G
  uint32_t q[D / 16][4];
  if (warp < WARPS) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int x = (lane >> 2) + 8 * i;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                              ((row0 + x / G) * a.Hq + h * G + x % G) * D) + (lane & 3);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        q[k][i] = x / G < m ? src[8 * k] : 0u;
        q[k][i + 2] = x / G < m ? src[8 * k + 4] : 0u;
      }
    }
  }
  if (m == 1) {
    // one row: its list is the piece's
    if (warp == 0) {
      int n = 0, before = -1;
      for (int k0 = 0; k0 < a.top;) {
        const int b = lists.b[0];
        int last = __shfl_up_sync(0xffffffffu, b, 1);
        if (lane == 0) last = before;
        const unsigned ends = __ballot_sync(0xffffffffu, b < 0 || b <= last || b > first_at >> lb);
        const int some = ends ? __ffs(ends) - 1 : 32;
        if (lane < some) list[n + lane].y = b;
        n += some;
        before = __shfl_sync(0xffffffffu, b, 31);
        k0 += 32;
        if (ends || k0 >= a.top) break;
        lists.load(a, row0, h, 1u, k0);
      }
      if (lane == 0) total_s = n;
    }
  } else {
    unsigned mine = 0u;
#pragma unroll
    for (int i = 0; i < lists.N; ++i) mine |= (live >> (warp + i * (WARPS + 1)) & 1u) << i;
    lists.mark(a, row0, h, mine, first_at, lb, words, seen, any_s);
    __syncthreads();
    const int n = list_blocks<WARPS + 1>(any_s, words, [&](int e, int b) { list[e].y = b; });  // in order
    if (tid == 0) total_s = n;
  }
  __syncthreads();
  // this CTA's share
  const int from = (int)((int64_t)total_s * rank / C), n = (int)((int64_t)total_s * (rank + 1) / C) - from;
  list += from;
  for (int e = tid; e < n; e += NT) {
    const int b = list[e].y, page = pages[b >> lper];
    int rows = m == 1;
    if (m > 1)
      for (int x = 0; x < m; ++x) rows |= (int)(seen[x * words + (b >> 5)] >> (b & 31) & 1u) << x;
    if (page < 0) {  // the block is left out
      atomicOr(a.s.err, ERR_BAD_PAGE);
      rows = 0;
    }
    list[e] = make_int2(max(page, 0) + ((b << lb) & (kStepPage - 1)), b | rows << 16);
  }
  __syncthreads();

  const int lx = min(lb, 6), box = 1 << lx, boxes = KEYS >> lx, lof = lb - lx;  // a box, of a stage, log2 of those of a block
  int all = n << lof;                                                          // boxes of the share
  // without those of the last block past the rows
  while (all > 0 && ((list[(all - 1) >> lof].y & 0xffff) << lb) + (((all - 1) & ((1 << lof) - 1)) << lx) > last_at) --all;
  const int stages = (all + boxes - 1) >> (6 - lx);
  bool ok = true;
  float o[D / 8][4];
  float mx[2] = {NEG, NEG}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  if (warp == WARPS) {
    // ---- loads ----
    int s = 0;
    for (; s < stages; ++s) {
      const int slot = s % NST;
      if (s >= NST)
        ok = a.wait_limit != 0 && __all_sync(0xffffffffu, wait_phase(empty(slot), (uint32_t)((s / NST - 1) & 1), abort, a.wait_limit));
      if (!ok) break;
      const int have = min(boxes, all - s * boxes);
      if (lane == 0) mbar_expect_tx(full(slot), (uint32_t)(have * box * D * 4));
      __syncwarp();
      if (lane < have) {
        const int e = s * boxes + lane;
        const int y = list[e >> lof].x + ((e & ((1 << lof) - 1)) << lx);
        const uint32_t dst = sb + (uint32_t)(slot * 2 * L::TILE + lane * box * 128);
#pragma unroll
        for (int d = 0; d < D; d += 64) {
          tma_load_2d(dst + (uint32_t)(d / 64 * L::HALF), &maps.k, d, y, full(slot));
          tma_load_2d(dst + (uint32_t)(L::TILE + d / 64 * L::HALF), &maps.v, d, y, full(slot));
        }
      }
      __syncwarp();
    }
    if (!ok && lane == 0) {
      atomicOr(a.s.err, ERR_TIMEOUT);
      *abort = 1;
    }
    // every copy issued has landed before the CTA moves on (bounded)
    for (int x = s > NST ? s - NST : 0; x < s; ++x) drain_phase(full(x % NST), (uint32_t)((x / NST) & 1));
  } else {
    // ---- 16 keys a warp ----
    const float sc = 1.4426950408889634f / sqrtf((float)D);
    const int xr = lane & 7;
    const uint32_t krow = (uint32_t)(16 * warp + (lane >> 4) * 8 + xr) * 128u, kc = (uint32_t)(lane >> 3 & 1);
    const uint32_t vrow = (uint32_t)(16 * warp + (lane >> 3 & 1) * 8 + xr) * 128u, vc = (uint32_t)(lane >> 4);
    for (int s = 0; s < stages; ++s) {
      const int slot = s % NST;
      ok = __all_sync(0xffffffffu, wait_phase(full(slot), (uint32_t)((s / NST) & 1), abort, a.wait_limit));
      if (!ok) break;
      const int e = s * boxes + (16 * warp >> lx);
      const int y = e < all ? list[e >> lof].y : 0;
      if (y >> 16) {  // some row takes this block
        const uint32_t kt = sb + (uint32_t)(slot * 2 * L::TILE), vt = kt + (uint32_t)L::TILE;
        // logical slot of the warp's first key
        const int base = ((y & 0xffff) << lb) + ((e & ((1 << lof) - 1)) << lx) + (16 * warp & (box - 1));
        if (base + 15 > last_at) {  // slots past the piece's last row may hold any bits
          const int key = lane >> 1;
          if (base + key > last_at) {
#pragma unroll
            for (int d = 0; d < D / 64; ++d)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                *reinterpret_cast<uint4*>(sm + (size_t)slot * 2 * L::TILE + L::TILE + d * L::HALF + (16 * warp + key) * 128 +
                                          ((lane & 1) * 4 + i) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        float z[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t b[4];
          ldmatrix(b, kt + (uint32_t)(k / 4 * L::HALF) + krow + (((uint32_t)(2 * (k & 3)) + kc) ^ (uint32_t)xr) * 16u);
          mma_bf16(z[0], q[k][0], q[k][1], q[k][2], q[k][3], b[0], b[1]);
          mma_bf16(z[1], q[k][0], q[k][1], q[k][2], q[k][3], b[2], b[3]);
        }
        uint32_t ph[4], pl[4];
        float f[2];
        bool grow = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int x = ((lane >> 2) + 8 * i) / G;  // row of the piece
          // the last of the 16 keys that it sees
          const int lim = (y >> (16 + x) & 1) ? first_at + x - base : -1;
          float top = mx[i];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float& v = z[j >> 1][2 * i + (j & 1)];
            const int key = (j >> 1) * 8 + 2 * (lane & 3) + (j & 1);
            v = key <= lim ? v * sc : __int_as_float(0xff800000);
            top = fmaxf(top, v);
          }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          f[i] = ex2f(mx[i] - top);
          grow |= top > mx[i];
          mx[i] = top;
          float w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = ex2f(z[j >> 1][2 * i + (j & 1)] - top);
          l[i] = l[i] * f[i] + ((w[0] + w[1]) + (w[2] + w[3]));
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            ph[i + 2 * j] = pack2(w[2 * j], w[2 * j + 1]);
            pl[i + 2 * j] = pack2(w[2 * j] - __uint_as_float(ph[i + 2 * j] << 16),
                                  w[2 * j + 1] - __uint_as_float(ph[i + 2 * j] & 0xffff0000u));
          }
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[i][0] *= f[0];
            o[i][1] *= f[0];
            o[i][2] *= f[1];
            o[i][3] *= f[1];
          }
        }
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t b[4];
          ldmatrix_t(b, vt + (uint32_t)(k / 4 * L::HALF) + vrow + (((uint32_t)(2 * (k & 3)) + vc) ^ (uint32_t)xr) * 16u);
          mma_bf16(o[2 * k], ph[0], ph[1], ph[2], ph[3], b[0], b[1]);
          mma_bf16(o[2 * k + 1], ph[0], ph[1], ph[2], ph[3], b[2], b[3]);
          mma_bf16(o[2 * k], pl[0], pl[1], pl[2], pl[3], b[0], b[1]);
          mma_bf16(o[2 * k + 1], pl[0], pl[1], pl[2], pl[3], b[2], b[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(slot));
    }
    if (!ok && lane == 0) {
      atomicOr(a.s.err, ERR_TIMEOUT);
      *abort = 1;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if ((lane & 3) == 0) {
        m_s[warp][(lane >> 2) + 8 * i] = mx[i];
        l_s[warp][(lane >> 2) + 8 * i] = l[i];
      }
    }
  }
  __syncthreads();  // the ring is at rest
  // ---- the warps' outputs joined ----
  float* acc = reinterpret_cast<float*>(sm);  // [WARPS][16][D + 4]
  if (warp < WARPS) {
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        *reinterpret_cast<float2*>(acc + ((size_t)warp * 16 + (lane >> 2) + 8 * j) * (D + 4) + 8 * i + 2 * (lane & 3)) =
            make_float2(o[i][2 * j], o[i][2 * j + 1]);
  }
  __syncthreads();
  const int rows = m * G;
  for (int x = tid; x < rows * D; x += NT) {
    const int r = x / D, d = x % D;
    float top = NEG, y = 0.f, sum = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) top = fmaxf(top, m_s[w][r]);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float f = ex2f(m_s[w][r] - top);
      y = fmaf(acc[((size_t)w * 16 + r) * (D + 4) + d], f, y);
      sum = fmaf(l_s[w][r], f, sum);
    }
    part[r * (D + 2) + d] = y;
    if (d == 0) {
      part[r * (D + 2) + D] = top;
      part[r * (D + 2) + D + 1] = abort_s ? -1.f : sum;  // (a sum is never negative)
    }
  }
  auto meet = [&] {
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  };
  if (C > 1) meet();
  else __syncthreads();
  auto of = [&](int r, const float* x) {  // *x of CTA r of the cluster
    if (C == 1) return *x;
    uint32_t there;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(there)
                 : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(x))), "r"(r));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(there) : "memory");
    return v;
  };
  for (int x = 2 * (rank * NT + tid); x < rows * D; x += 2 * C * NT) {
    const int r = x / D, d = x % D;
    if (!(live >> (r / G) & 1u)) continue;
    const float* at = part + r * (D + 2);
    float top = NEG, y0 = 0.f, y1 = 0.f, sum = 0.f;
    bool whole = true;
    for (int c = 0; c < C; ++c) top = fmaxf(top, of(c, at + D));
    for (int c = 0; c < C; ++c) {
      const float f = ex2f(of(c, at + D) - top), lc = of(c, at + D + 1);
      y0 = fmaf(of(c, at + d), f, y0);
      y1 = fmaf(of(c, at + d + 1), f, y1);
      sum = fmaf(lc, f, sum);
      whole = whole && !(lc < 0.f);
    }
    if (!whole) continue;  // a CTA gave up: the row stays as it was
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + ((row0 + r / G) * a.Hq + h * G + r % G) * D + d) =
        pack2(y0 * inv, y1 * inv);
  }
  if (C > 1) meet();  // no CTA leaves while another reads it
}

template <int D, int G>
cudaError_t launch_t(const SparseArgs& a, const SparseMaps& maps, cudaStream_t s) {
  constexpr int T = 16 / G;
  const int most = a.s.maxp * (kStepPage / a.block), words = (most + 31) / 32;
  const int entries = (int)std::min<int64_t>((int64_t)T * a.top, most);
  const int smem = 1024 + Sm<D>::SEEN + 4 * 256 + 4 * (((T + 1) * words + 1) & ~1) + 8 * entries;
  cudaError_t e = allow_shared<&k_sparse_mma<D, G>>(1024 + Sm<D>::SEEN + 4 * 256 + 4 * (T + 1) * 128 + 8 * 4096);
  if (e != cudaSuccess) return e;
  if (a.splits > 8 && (e = allow_large_clusters<&k_sparse_mma<D, G>>()) != cudaSuccess) return e;
  return launch_step_kernel(k_sparse_mma<D, G>, dim3((unsigned)(sparse_pieces(a.s, T) * a.Hkv * a.splits)), NT, (size_t)smem, a.splits, s, a, maps, words);
}

}  // namespace

cudaError_t launch_sparse_mma(const SparseArgs& a, const SparseMaps& maps, cudaStream_t s) {
  if (a.s.n == 0 || a.s.max_rows == 0) return cudaSuccess;
  const int G = a.Hq / a.Hkv;
  if (a.D == 128) return G == 4 ? launch_t<128, 4>(a, maps, s) : launch_t<128, 2>(a, maps, s);
  if (a.D == 64) return G == 4 ? launch_t<64, 4>(a, maps, s) : launch_t<64, 2>(a, maps, s);
  return cudaErrorInvalidValue;
}

}  // namespace gp
