// Attention over listed blocks for many rows of a request (prompts), on the tensor
// cores (tcgen05): bf16 caches and queries.  The formulas are k_sparse.cu's.
//
// A piece is 128 / G rows of a request; with the G heads of a KV head they make the
// 128 rows of a product.  The piece goes through the blocks that any of its rows
// lists, each loaded once; a row takes weight 0 in a block that it does not list, by
// a bias of its exponent.  Neighbouring rows list much the same blocks, so this
// reads and multiplies a few times what one row alone needs, where a pass of
// its own for each row reads all of it from L2 every time.
//
// Per stage of 64 keys:
//   S = Q K^T        128 x 64, fp32 in TMEM, double buffered
//   P = 2^(S c - m)  in two bf16 parts over S (2^-15 of a weight is left, as
//                    k_chunk_tc.cu's), a maximum followed only when it grows by
//                    more than 24: O is then rescaled in TMEM
//   O += P V         128 x d, both parts, V MN-major as TMA left it
// A CTA holds 256 of the 512 columns of TMEM (O d, S and P twice 64) and half of
// the shared memory (101 to 115 KB with blocks of 64 and more, d = 128; 125 KB with 256
// pages in blocks of 16, G = 4, where one CTA fits), so that two CTAs share an SM: one's softmax runs beside the
// other's products, and one's start beside the other's work.  The products are
// issued as S0 S1 O0 S2 O1 S3 ..., so that a CTA's softmax finds the next S done; K and
// V come through one ring in that order.
//   warps 0-3   softmax (thread = row = TMEM lane), then the outputs
//   warp 4      lists the blocks, then loads K and V (TMA, a box a block of up to 64)
//   warp 5      issues the products
// Products of 64 keys are bounded by shared memory: S takes 48 clocks a step for Q and K
// at 128 bytes a clock, 384 a stage, the two parts of P 512; 870 clocks a stage and SM are
// measured.  4001 rows behind 12 007 tokens, 32 + 8 heads, d = 128, 32 blocks of 64 a row: 325 us
// for 473 GFLOP, 75 % of the measured bf16 rate; row by row in k_sparse_mma.cu 1094 us.  A CTA alone
// takes 1300 clocks a stage, its start 8500 (lists, pages), its outputs 3000.
// Every wait is bounded: on expiry the CTA records ERR_TIMEOUT, waits for what it
// has in flight, frees its TMEM and returns; rows that it has part in stay as they were.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstdint>

#include "math2.cuh"
#include "shared_limit.cuh"
#include "sparse_tc.cuh"
#include "tc_rows.cuh"

namespace gp {
namespace {

using namespace tc;

constexpr int NT = 192;
constexpr int KEYS = 64;  // of a stage
constexpr int TMEM_COLS = 256;
constexpr float NEG = -1.0e30f;
constexpr float LAZY = 24.f;  // base-2 growth of a maximum that is not followed

template <int D>
struct Sm {
  static constexpr int HALF = KEYS * 128;     // 64 dimensions of a stage's keys
  static constexpr int TILE = D / 64 * HALF;  // K or V of a stage
  static constexpr int NST = 512 / D;         // tiles in flight: 64 KB
  static constexpr int QHALF = 128 * 128;     // 64 dimensions of the rows of Q
  static constexpr int Q = NST * TILE;
  static constexpr int RING = Q + D / 64 * QHALF;
  // then: int page[256]; unsigned any[words], seen[T][words]; uint16_t list[blocks]
};

template <int D, int G>
__global__ void __launch_bounds__(NT, 2) k_sparse_tc(const __grid_constant__ SparseArgs a, const __grid_constant__ SparseMaps maps,
                                                     const __grid_constant__ CUtensorMap qmap, int words) {
  using L = Sm<D>;
  constexpr int T = 128 / G, NST = L::NST;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = static_cast<uint32_t>(__cvta_generic_to_shared(sm));
  int* pages = reinterpret_cast<int*>(sm + L::RING);  // first key row of a page in the map; -1
  unsigned* any_s = reinterpret_cast<unsigned*>(pages + 256);
  unsigned* seen = any_s + words;
  uint16_t* list = reinterpret_cast<uint16_t*>(seen + T * words);
  __shared__ __align__(8) uint64_t bars[2 * NST + 7];
  __shared__ int abort_s, bad_s;
  __shared__ uint32_t tmem_s;
  __shared__ float2 ml_s[128];  // a row's maximum and sum
  __shared__ bool live_s[T];    // the row takes part
  volatile int* abort = &abort_s;
  const uint32_t bar0 = static_cast<uint32_t>(__cvta_generic_to_shared(bars));
  auto full = [&](int s) { return bar0 + 8u * (uint32_t)s; };
  auto empty = [&](int s) { return bar0 + 8u * (uint32_t)(NST + s); };
  auto s_ready = [&](int s) { return bar0 + 8u * (uint32_t)(2 * NST + (s & 1)); };
  auto p_ready = [&](int s) { return bar0 + 8u * (uint32_t)(2 * NST + 2 + (s & 1)); };
  const uint32_t o_done = bar0 + 8u * (uint32_t)(2 * NST + 4), mma_done = o_done + 8u, q_full = o_done + 16u;  // o_done: once a stage
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const int C = a.splits, rank = blockIdx.x % C, item = blockIdx.x / C, h = item % a.Hkv;

  begin_step();
  const StepPiece p = find_piece(a.s, item / a.Hkv, log2_const(T), 1, tid == 0);
  if (p.r < 0 || p.at * T >= p.rows) return;  // (the whole cluster)
  const int t0 = p.at * T, m_rows = min(T, p.rows - t0);
  BlockLists<NT / 32, T> lists;
  lists.load(a, (size_t)p.row0 + t0, h, lists.rows_of(m_rows), 0);
  const int first_at = p.cached + t0, last_at = first_at + m_rows - 1;  // the rows' slots
  const size_t row0 = (size_t)p.row0 + t0;
  const int named = tid < m_rows ? a.s.row_req[row0 + tid] : -1;
  const int lb = log2_of(a.block), lper = kStepPageLog - lb;  // blocks of a page

  if (tid == 0) {
    for (int i = 0; i < 2 * NST + 7; ++i)  // p_ready: four warps
      mbar_init(bar0 + 8u * (uint32_t)i, i == 2 * NST + 2 || i == 2 * NST + 3 ? 4u : 1u);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    abort_s = bad_s = 0;
    // the G heads of the piece's rows (and of what follows them: a row of the
    // products that is no row of the piece is never looked at)
    mbar_expect_tx(q_full, (uint32_t)(D / 64 * L::QHALF));
    for (int d = 0; d < D; d += 64)
      tma_load_3d(sb + (uint32_t)(L::Q + d / 64 * L::QHALF), &qmap, d, h * G, (int)row0, q_full);
  }
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(&tmem_s))),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  for (int i = tid; i < (T + 1) * words; i += NT) any_s[i] = 0u;
  for (int i = tid; i <= last_at / kStepPage; i += NT) {
    const int page = a.s.tables[(size_t)p.slot * a.s.maxp + i];
    pages[i] = page >= 0 && page < a.s.num_pages_total
                   ? (int)((((size_t)a.layer * a.s.num_pages_total + page) * a.Hkv + h) * kStepPage) : -1;
  }
  if (tid < T) live_s[tid] = row_named(a.s, named, p.r);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)tmem_s);
  for (int i = tid; i <= last_at / kStepPage; i += NT)
    if (pages[i] < 0) bad_s = 1;
  const uint32_t ts = tmem + D, to = tmem;  // columns: O, S and P of even and of odd stages
  const int owned = warp + lane * (NT / 32);  // row `lane` of this warp's lists
  lists.mark(a, row0, h, __ballot_sync(0xffffffffu, lane < lists.N && owned < T && live_s[min(owned, T - 1)]), first_at, lb, words,
             seen, any_s);
  const int tok = tid / G, sees = first_at + tok;  // of softmax threads
  const bool valid = warp < 4 && live_s[min(tok, T - 1)];
  const size_t at = ((row0 + tok) * a.Hq + h * G + tid % G) * D;
  const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
  __syncthreads();
  if (bad_s) {  // blocks on a page outside the pool are left out
    if (warp == 0)
      for (int w = 0; w < words; ++w) {
        const bool out = (any_s[w] >> lane & 1u) && pages[(w * 32 + lane) >> lper] < 0;
        const unsigned drop = __ballot_sync(0xffffffffu, out);
        if (lane == 0 && drop) {
          atomicOr(a.s.err, ERR_BAD_PAGE);
          any_s[w] &= ~drop;
        }
      }
    __syncthreads();
  }
  // the blocks that any row lists, in order
  const int count = list_blocks<NT / 32>(any_s, words, [&](int e, int b) { list[e] = (uint16_t)b; });
  __syncthreads();
  const int lx = min(lb, 6), box = 1 << lx, boxes = KEYS >> lx, lof = lb - lx;  // a box, of a stage, log2 of those of a block
  // this CTA's share of the list, in boxes
  const int from = (int)((int64_t)count * rank / C);
  int all = uniform((int)((int64_t)count * (rank + 1) / C) - from) << lof;
  list += from;
  // first logical slot of box e
  auto slot_of = [&](int e) { return ((int)list[e >> lof] << lb) + ((e & ((1 << lof) - 1)) << lx); };
  while (all > 0 && slot_of(all - 1) > last_at) --all;  // boxes of the last block past the rows
  all = uniform(all);
  const int stages = (all + boxes - 1) >> (6 - lx);
  bool ok = true;
  auto timed_out = [&] {
    atomicOr(a.s.err, ERR_TIMEOUT);
    *abort = 1;
  };

  if (warp == 4) {
    // ---- loads ----
    int c = 0;  // tiles issued
    auto load = [&](const CUtensorMap* map, int s) {
      const int slot = c % NST;
      if (c >= NST)
        ok = ok && a.wait_limit != 0 &&
             __all_sync(0xffffffffu, wait_phase(empty(slot), (uint32_t)((c / NST - 1) & 1), abort, a.wait_limit));
      if (!ok) return;
      const int have = min(boxes, all - s * boxes);
      if (lane == 0) mbar_expect_tx(full(slot), (uint32_t)(have * box * D * 2));
      __syncwarp();
      if (lane < have) {
        const int at0 = slot_of(s * boxes + lane), y = pages[at0 >> kStepPageLog] + (at0 & (kStepPage - 1));
        const uint32_t dst = sb + (uint32_t)(slot * L::TILE + lane * box * 128);
#pragma unroll
        for (int d = 0; d < D; d += 64) tma_load_2d(dst + (uint32_t)(d / 64 * L::HALF), map, d, y, full(slot));
      }
      __syncwarp();
      ++c;
    };
    if (stages > 0) load(&maps.k, 0);
    if (stages > 1) load(&maps.k, 1);
    for (int s = 0; s < stages && ok; ++s) {
      load(&maps.v, s);
      if (s + 2 < stages) load(&maps.k, s + 2);
    }
    if (!ok && lane == 0) timed_out();
    // every copy issued has landed before the CTA moves on (bounded)
    for (int x = c > NST ? c - NST : 0; x < c; ++x) drain_phase(full(x % NST), (uint32_t)((x / NST) & 1));
    drain_phase(q_full, 0u);
  } else if (warp == 5) {
    // ---- products ----
    tc_fence_after();
    auto wait = [&](uint32_t bar, int phase) {
      ok = ok && __all_sync(0xffffffffu, wait_phase(bar, (uint32_t)(phase & 1), abort, a.wait_limit));
    };
    int c = 0;  // tiles used
    auto tile = [&] { return sb + (uint32_t)(c % NST * L::TILE); };
    auto score = [&](int s) {
      wait(full(c % NST), c / NST);
      if (!ok) return;
      tc_fence_after();
      const uint64_t q0 = sw128_desc(sb + (uint32_t)L::Q), k0 = sw128_desc(tile());
#pragma unroll
      for (int e = 0; e < D / 16; ++e)
        mma_ss(ts + (uint32_t)(64 * (s & 1)), q0 + (uint64_t)(((e >> 2) * L::QHALF + (e & 3) * 32) >> 4),
               k0 + (uint64_t)(((e >> 2) * L::HALF + (e & 3) * 32) >> 4), idesc(KEYS, false), e > 0 ? 1u : 0u);
      commit(s_ready(s));
      commit(empty(c++ % NST));
    };
    wait(q_full, 0);
    if (stages > 0 && ok) score(0);
    if (stages > 1 && ok) score(1);
    for (int s = 0; s < stages && ok; ++s) {
      wait(full(c % NST), c / NST);
      wait(p_ready(s), s >> 1);
      if (!ok) break;
      tc_fence_after();
      const uint64_t v0 = sw128_mn_desc(tile(), L::HALF);
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int part = 0; part < 2; ++part)
          mma_ts(to, ts + (uint32_t)(64 * (s & 1) + 32 * part + 8 * e), v0 + (uint64_t)(e * 2048 >> 4), idesc(D, true),
                 s == 0 && e == 0 && part == 0 ? 0u : 1u);
      commit(o_done);
      commit(empty(c++ % NST));
      if (s + 2 < stages) score(s + 2);  // over P, which the products before it have read
    }
    if (!ok) {
      if (lane == 0) timed_out();
      __threadfence_block();  // the others see it before mma_done
      __syncwarp();
    }
    // every product issued has completed before TMEM is released (bounded)
    commit(mma_done);
    drain_phase(mma_done, 0u);
    __syncwarp();
  } else {
    // ---- softmax: thread = row ----
    const float sc = 1.4426950408889634f / sqrtf((float)D);
    const uint32_t my_o = to + lanes;
    const unsigned* mine = seen + min(tok, T - 1) * words;
    float m = NEG, l = 0.f;
    for (int s = 0; s < stages; ++s) {
      // the row's part in each 16 keys of the stage
      bool in[4];
      const bool tail = s + 1 == stages;
      const int end = min(s * boxes + boxes, all);  // past the stage's last box
      const bool partly = tail || slot_of(end - 1) + box - 1 > first_at;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = s * boxes + (16 * i >> lx);
        in[i] = false;
        if (e < all) {
          const int b = list[e >> lof];
          in[i] = mine[b >> 5] >> (b & 31) & 1u;
        }
      }
      const uint32_t my_s = ts + lanes + (uint32_t)(64 * (s & 1));
      ok = __all_sync(0xffffffffu, wait_phase(s_ready(s), (uint32_t)(s >> 1 & 1), abort, a.wait_limit));
      if (!ok) break;
      tc_fence_after();
      uint32_t r[2][32];
      tmem_load32(my_s, r[0]);
      tmem_load32(my_s + 32u, r[1]);
      tmem_wait_ld();
      tmem_arrived(r[0]);
      tmem_arrived(r[1]);
      if (partly) {
        // slots that not every row sees, and places that no block filled, which may
        // hold any bits
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = s * boxes + (16 * i >> lx);
          const int base = e < all ? slot_of(e) + (16 * i & (box - 1)) : 0;
          const int keep = in[i] ? sees - base : -1;
#pragma unroll
          for (int c = 0; c < 16; ++c)
            if (c > keep) r[i / 2][16 * (i & 1) + c] = 0xff800000u;  // -inf
        }
      }
      float top = NEG;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t* x = r[i / 2] + 16 * (i & 1);
        float mx = max3(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]));
#pragma unroll
        for (int c = 3; c < 15; c += 2) mx = max3(mx, __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
        mx = fmaxf(mx, __uint_as_float(x[15]));
        top = fmaxf(top, in[i] ? sc * mx : NEG);
      }
      if (s == 0) {
        m = fmaxf(m, top);
      } else {
        const bool grow = top > m + LAZY;
        if (__any_sync(0xffffffffu, grow)) {
          // O is at rest once the products with the last P have completed (those before
          // it completed before this S)
          ok = __all_sync(0xffffffffu, wait_phase(o_done, (uint32_t)((s - 1) & 1), abort, a.wait_limit));
          if (!ok) break;
          tc_fence_after();
          const float mn = grow ? top : m, f = ex2f(m - mn);
          m = mn;
          l *= f;
#pragma unroll 1
          for (int d = 0; d < D; d += 32) {
            uint32_t o[32];
            tmem_load32(my_o + (uint32_t)d, o);
            tmem_wait_ld();
            tmem_arrived(o);
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
            tmem_store32(my_o + (uint32_t)d, o);
          }
        }
      }
      const float2 sc2 = make_float2(sc, sc);
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float bias = in[2 * q + c / 8] ? -m : __int_as_float(0xff800000);
          float2 z = fma2(make_float2(__uint_as_float(r[q][2 * c]), __uint_as_float(r[q][2 * c + 1])), sc2, make_float2(bias, bias));
          z.x = ex2f(z.x);
          z.y = ex2f(z.y);
          sum[c & 1] = add2(sum[c & 1], z);
          hi[c] = __byte_perm(__float_as_uint(z.x), __float_as_uint(z.y), 0x7632);  // the upper halves
          z = less_bf16(z, hi[c]);
          lo[c] = pack_bf16(z.x, z.y);
        }
        tmem_store16(my_s + (uint32_t)(16 * q), hi);
        tmem_store16(my_s + (uint32_t)(32 + 16 * q), lo);
      }
      l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      if (tail) {  // weight 0 times any bits is not 0: those rows of V are cleared
        const int c = 2 * stages - 1, slot = c % NST, key = tid >> 1;  // the last tile
        ok = __all_sync(0xffffffffu, wait_phase(full(slot), (uint32_t)((c / NST) & 1), abort, a.wait_limit));
        if (!ok) break;
        const int e = s * boxes + (key >> lx);
        if (e >= all || slot_of(e) + (key & (box - 1)) > last_at) {
          unsigned char* v = sm + (size_t)slot * L::TILE + (size_t)key * 128 + (tid & 1) * 64;
#pragma unroll
          for (int d = 0; d < D / 64; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) reinterpret_cast<uint4*>(v + (size_t)d * L::HALF)[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_ready(s));
    }
    // (o_done may be two stages behind; products that were given up are done too)
    if (ok) ok = __all_sync(0xffffffffu, wait_phase(mma_done, 0u, abort, a.wait_limit) && !*abort);
    if (ok) {
      tc_fence_after();
      const float inv = C > 1 ? 1.f : l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
      for (int d = 0; d < D; d += 32) {
        uint32_t o[32];
        if (stages > 0) {
          tmem_load32(my_o + (uint32_t)d, o);
          tmem_wait_ld();
          tmem_arrived(o);
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = 0u;
        }
        if (C > 1) {
          float4* dst = reinterpret_cast<float4*>(sm + ((size_t)tid * (D + 4) + d) * 4);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]), __uint_as_float(o[4 * e + 2]),
                                 __uint_as_float(o[4 * e + 3]));
        } else if (valid) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at + d);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              u[k] = pack_bf16(__uint_as_float(o[8 * e + 2 * k]) * inv, __uint_as_float(o[8 * e + 2 * k + 1]) * inv);
            dst[e] = make_uint4(u[0], u[1], u[2], u[3]);
          }
        }
        __syncwarp();
      }
      ml_s[tid] = make_float2(m, l);
    } else if (lane == 0) {
      timed_out();
    }
    tmem_wait_st();  // a loop that was left between a store and its wait
  }
  tc_fence_before();
  __syncthreads();
  if (C > 1) {
    // ---- the shares joined: a warp a row, each CTA its rows ----
    if (abort_s && tid < 128) ml_s[tid] = make_float2(NEG, -1.f);  // (a sum is never negative)
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    auto there = [&](const void* x, int r) {  // *x of CTA r of the cluster
      uint32_t y;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(y) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(x))), "r"(r));
      return y;
    };
    for (int x = rank + C * warp; x < m_rows * G; x += C * (NT / 32)) {
      if (!live_s[x / G]) continue;
      float top = NEG, sum = 0.f, y[D / 32];
      bool whole = true;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) y[i] = 0.f;
      for (int r = 0; r < C; ++r) {
        float mr, lr;
        asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(mr), "=f"(lr) : "r"(there(&ml_s[x], r)) : "memory");
        const float mn = fmaxf(top, mr), f = ex2f(top - mn), g = ex2f(mr - mn);
        top = mn;
        sum = sum * f + lr * g;
        whole = whole && !(lr < 0.f);
        const uint32_t at0 = there(sm + ((size_t)x * (D + 4) + lane * (D / 32)) * 4, r);
        float v[D / 32];
        if constexpr (D == 128) {
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(at0) : "memory");
        } else {
          asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "r"(at0) : "memory");
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) y[i] = y[i] * f + v[i] * g;
      }
      if (!whole) continue;  // a CTA gave up
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + ((row0 + x / G) * a.Hq + h * G + x % G) * D) +
                      lane * (D / 64);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) dst[i] = pack_bf16(y[2 * i] * inv, y[2 * i + 1] * inv);
    }
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");  // no CTA leaves while another reads it
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  }
  if (warp == 5) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
  }
}

template <int D, int G>
cudaError_t launch_t(const SparseArgs& a, const SparseMaps& maps, const CUtensorMap& qmap, cudaStream_t s) {
  constexpr int T = 128 / G;
  const int most = a.s.maxp * (kStepPage / a.block), words = (most + 31) / 32;
  const int smem = 1024 + Sm<D>::RING + 4 * 256 + 4 * (T + 1) * words + 2 * most;
  cudaError_t e = allow_shared<&k_sparse_tc<D, G>>(1024 + Sm<D>::RING + 4 * 256 + 4 * (T + 1) * 128 + 2 * 4096);
  if (e != cudaSuccess) return e;
  return launch_step_kernel(k_sparse_tc<D, G>, dim3((unsigned)(sparse_pieces(a.s, T) * a.Hkv * a.splits)), NT, (size_t)smem, a.splits, s, a, maps, qmap, words);
}

}  // namespace

cudaError_t launch_sparse_tc(const SparseArgs& a, const SparseMaps& maps, const CUtensorMap& qmap, cudaStream_t s) {
  if (a.s.n == 0 || a.s.max_rows == 0) return cudaSuccess;
  const int G = a.Hq / a.Hkv;
  if (a.D == 128) return G == 4 ? launch_t<128, 4>(a, maps, qmap, s) : launch_t<128, 2>(a, maps, qmap, s);
  if (a.D == 64) return G == 4 ? launch_t<64, 4>(a, maps, qmap, s) : launch_t<64, 2>(a, maps, qmap, s);
  return cudaErrorInvalidValue;
}

}  // namespace gp
