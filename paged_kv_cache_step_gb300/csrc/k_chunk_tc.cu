// Causal attention of several new tokens a request over the paged cache, and
// the accumulated weights of it, on the tensor cores (tcgen05, sm_103a): bf16
// caches and queries.  The formulas are k_chunk.cu's.
//
// Attention.  A query tile is 128 rows, 128 / G tokens of the G heads of a KV
// head (they share its keys).  Per key tile of 128 slots
//   S = Q K^T        128 x 128, K = d, fp32 in TMEM
//   P = 2^(S c - m)  c = log2(e) / sqrt(d), in two bf16 parts over S in TMEM
//   O += P V         128 x d, K = 128 for each part, P from TMEM, V MN-major as
//                    TMA left it
// with the maximum m of the first tile, moved only when a row's has grown by
// more than 24 (a factor 2^24, which the exponents of fp32 and bf16 hold
// easily): O is then rescaled in TMEM by the warp that found it, between two
// products.
// P's first part is its upper 16 bits, the second the rest rounded to bf16: a
// weight keeps 2^-15 of itself, where the output's own rounding is 2^-8.  One
// bf16 part alone takes 522 us instead of the 680 below, and is off by up to 2^-8
// of sum a |v|: more than the output's rounding where values cancel.  The rest is
// formed by a mixed-precision FMA of the packed first part (masked out and added
// instead: 755 us; a rounded first part: 695).  The sum l is of the unrounded fp32
// weights.
//
// One CTA per SM walks a list of items that the host cut into even shares.
// Two softmax groups of 128 threads (thread = row = TMEM lane) alternate on
// the tensor core: while one computes P, the other's products run.  They hold
// two query tiles (the K and V tiles then serve 256 rows), or, where a request
// has one tile left, the even and odd key tiles of that one (a launch of its
// own).  A query tile in several parts leaves partials (O, m, l) that another
// kernel joins.
//   warp 0       producer: Q tiles, and the K and V tiles through a ring
//   warp 1       MMA issuer
//   warps 4-7    softmax of group 0, then its epilogue;  warps 8-11 group 1
// TMEM: S0 S1 (128 columns each, the parts of P over 64 each), O0 O1.
//
// Weights.  W_i += sum over rows of 2^(S_ri c - L_r) needs the final
// L_r = m_r + log2 l_r of every row (rounded to fp32 once, as the logit is), so S
// is formed again, transposed: S^T = K Q^T, so that a thread (TMEM lane) owns
// a key and adds up half of its columns in registers: no atomics, one writer a
// weight.  -L / c joins S^T as one more K = 16 step, ones times its three bf16
// parts (24 bits): read from shared memory by every thread instead, it took
// four times its bytes of the bandwidth that the products need there (291 us
// against 272 then for 6007 tokens behind 4099, 32 heads, d = 128).  An item is a
// page (two key tiles) against a range of query tiles, S^T double buffered, K
// tiles kept and the next item's loaded meanwhile.
//   warp 0       producer;  warps 1, 2  MMA issuers, one a key tile
//   warp 3       L of the query tiles;  warps 4-19  sums
//
// Measured (bf16, d = 128, 32 query and 8 KV heads): those 6007 tokens take 680
// us of attention (80 % of the measured bf16 rate, of the 6 d flops a pair that the
// two parts take) and 270 us of weights; 106 drafted tokens of 16 requests over
// 85 831 cached ones 80 and 38 us, where reading K and V once takes 52 us and K
// again 26.  What bounds the attention is the chain S - softmax - O of a group,
// beside products of 1536 clocks a tile.  Tried when P was one part (510 us then)
// and slower: two threads a row (583 us), an issuer a group (554 us), weights under
// the old maximum while the new one is found (562 us), S double buffered in steps
// of 64 keys (717 us: products of 64 columns read A again for half as much).
//
// Every wait is bounded (by the caller's limit, one second of clock cycles unless a
// test sets less): on expiry the CTA records ERR_TIMEOUT, raises an abort flag that
// ends every role's loop, waits (bounded by the full second) for its copies, products
// and TMEM stores in flight, frees its TMEM and returns.
#include <cuda.h>
#include <cuda_bf16.h>

#include <cstdint>

#include "chained.cuh"
#include "math2.cuh"
#include "tc_rows.cuh"
#include "weighted_kernels.h"

namespace gp {
namespace {

using namespace tc;

constexpr int PAGE = 256;
constexpr int NT = 384;   // attention: four warps of the pipeline, two softmax groups of four
constexpr int WNT = 640;  // weights: four warps of the pipeline, four summing groups
constexpr int TK = 128;
constexpr int TMEM_COLS = 512;
constexpr float NEG = -1.0e30f;
constexpr float LAZY = 24.f;                 // base-2 growth of a maximum that is not followed

// Registers of the calling warpgroup (all of its warps call it).  The shares add
// up to what the block was launched with.
template <int N>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Bounded wait; gives up when the limit passes or *abort is set.  (A try may itself
// wait for a while; a limit of 0 is looked at by the producers, before they try.)
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const volatile int* abort, long long limit) {
  if (mbar_try(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (*abort || clock64() - t0 > limit) return false;
    if (mbar_try(bar, parity)) return true;
  }
}
// The wait for what a role has in flight before it ends.
__device__ __forceinline__ void drain_bar(uint32_t bar, uint32_t parity) {
  const int zero = 0;
  wait_bar(bar, parity, &zero, kDefaultWaitLimit);
}

template <typename T>
__device__ __forceinline__ T load_item(const T* p) {
  static_assert(sizeof(T) == 32, "two 16-byte loads");
  union {
    int4 v[2];
    T t;
  } u;
  u.v[0] = __ldg(reinterpret_cast<const int4*>(p));
  u.v[1] = __ldg(reinterpret_cast<const int4*>(p) + 1);
  return u.t;
}
__device__ __forceinline__ ChunkReq load_req(const ChunkReq* p) {
  static_assert(sizeof(ChunkReq) == 24, "row0, four ints");
  ChunkReq q;
  const int2* s = reinterpret_cast<const int2*>(p);
  const int2 a = __ldg(s), b = __ldg(s + 1), c = __ldg(s + 2);
  q.row0 = (int64_t)(((uint64_t)(uint32_t)a.y << 32) | (uint32_t)a.x);
  q.cached = b.x;
  q.nnew = b.y;
  q.slot = c.x;
  q.bt_off = c.y;
  return q;
}

// The key row of tile `t` of a request in the cache's tensor map.
__device__ __forceinline__ int key_row(const ChunkTcArgs& a, const ChunkReq& rq, int h, int t) {
  int pg = __ldg(a.bt + rq.bt_off + (t >> 1));
  if (pg < 0 || pg >= a.num_pages_total) {
    atomicOr(a.err, ERR_BAD_PAGE);
    pg = 0;
  }
  return (int)((((size_t)a.layer * a.num_pages_total + pg) * a.Hkv + h) * PAGE + (t & 1) * TK);
}

// What an item's groups do: `n` key tiles, of which group x takes cnt[x].
struct Work {
  int n, cnt[2];
};
template <int G, bool KEYS>
__device__ __forceinline__ Work work_of(const ChunkItem& it, const ChunkReq& rq) {
  constexpr int TOK = 128 / G;
  Work w;
  w.n = it.ke - it.kb;
  if (KEYS) {
    w.cnt[0] = (w.n + 1) / 2;
    w.cnt[1] = w.n / 2;
  } else {
    // the first tile's last token sees fewer slots than the second's
    const int see = (rq.cached + min(it.t0 + TOK, rq.nnew) + TK - 1) / TK;
    w.cnt[0] = min(max(see - it.kb, 0), w.n);
    w.cnt[1] = it.alone ? 0 : w.n;
  }
  return w;
}

// KEYS: one query tile, its even key tiles the first group's and the odd ones
// the second's; else two query tiles, every key tile for both.
template <int D, bool KEYS>
struct Sm {
  static constexpr int TILE = TK * D * 2;             // a Q, K or V tile
  static constexpr int HALF = TK * 128;               // its span of 64 columns
  static constexpr int NQT = KEYS ? 1 : 2;            // query tiles
  static constexpr int NST = (D == 128 ? 7 : 12) - NQT;  // K and V tiles in flight
  static constexpr size_t Q = 0;
  static constexpr size_t ST = NQT * (size_t)TILE;
  static constexpr size_t BARS = ST + (size_t)NST * TILE;
  // full[NST], empty[NST], q_full, q_empty, s_ready[2], p_ready[2], o_done[2], o_free[2], p_half[2], mma_done
  static constexpr int NBARS = 2 * NST + 13;
  static constexpr size_t MISC = BARS + 8 * NBARS;
  static constexpr size_t BYTES = MISC + 64 + 1024;   // + alignment slack
};

template <int D, int G, bool KEYS>
__global__ void __launch_bounds__(NT, 1) k_chunk_tc(const __grid_constant__ ChunkTcArgs a) {
  using L = Sm<D, KEYS>;
  constexpr int NST = L::NST, TOK = 128 / G;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = static_cast<uint32_t>(__cvta_generic_to_shared(sm));
  int* misc = reinterpret_cast<int*>(sm + L::MISC);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(misc);
  volatile int* abort = misc + 1;
  const uint32_t bar0 = sb + (uint32_t)L::BARS;
  auto full = [&](int s) { return bar0 + 8u * (uint32_t)s; };
  auto empty = [&](int s) { return bar0 + 8u * (uint32_t)(NST + s); };
  const uint32_t q_full = bar0 + 8u * (uint32_t)(2 * NST), q_empty = q_full + 8u;
  auto s_ready = [&](int x) { return q_full + 8u * (uint32_t)(2 + x); };
  auto p_ready = [&](int x) { return q_full + 8u * (uint32_t)(4 + x); };
  auto o_done = [&](int x) { return q_full + 8u * (uint32_t)(6 + x); };
  auto o_free = [&](int x) { return q_full + 8u * (uint32_t)(8 + x); };
  auto p_half = [&](int x) { return q_full + 8u * (uint32_t)(10 + x); };
  const uint32_t mma_done = q_full + 96u;

  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const ChunkItem* items = KEYS ? a.kitems : a.items;
  const int32_t* begin = KEYS ? a.kbegin : a.begin;
  const int i0 = uniform(begin[blockIdx.x]), i1 = uniform(begin[blockIdx.x + 1]);
  let_next_in();
  if (tid == 0) {
    for (int i = 0; i < L::NBARS; ++i) {
      const int b = i - 2 * NST;  // p_ready, o_free, p_half: the group's four warps; else one arrival
      const int n = b == 4 || b == 5 || (b >= 8 && b <= 11) ? 4 : 1;
      mbar_init(bar0 + 8u * (uint32_t)i, (uint32_t)n);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    *abort = 0;
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(tmem_holder))),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_holder);
  wait_for_previous();  // (of two attention launches the second is chained)
  auto timed_out = [&] {
    atomicOr(a.err, ERR_TIMEOUT);
    *abort = 1;
  };

  // 128 x 88 + 256 x 208 registers = the 384 x 168 of the launch
  if (warp < 4) {
    registers_down<88>();
    if (warp == 0) {
      // ---- producer ----------------------------------------------------------
      if (lane == 0) {
        int c = 0, nq = 0;  // tiles and items issued
        bool ok = true;
        const bool patient = a.wait_limit != 0;
        for (int i = i0; i < i1 && ok; ++i) {
          const ChunkItem it = load_item(items + i);
          const ChunkReq rq = load_req(a.reqs + it.r);
          const Work w = work_of<G, KEYS>(it, rq);
          auto tile = [&](const CUtensorMap* map, int t) {
            if (!ok) return;
            const int s = c % NST;
            if (c >= NST && !(ok = patient && wait_bar(empty(s), (uint32_t)((c / NST - 1) & 1), abort, a.wait_limit))) return;
            const int y = key_row(a, rq, it.h, t);
            const uint32_t dst = sb + (uint32_t)(L::ST + (size_t)s * L::TILE);
            mbar_expect_tx(full(s), L::TILE);
#pragma unroll
            for (int x = 0; x < D; x += 64) tma_load_2d(dst + (uint32_t)(x / 64 * L::HALF), map, x, y, full(s));
            ++c;
          };
          // the query tiles' place is free only when the item before has formed its
          // last S: the first key tiles are on their way before
          auto queries = [&] {
            if (!ok || (nq > 0 && !(ok = patient && wait_bar(q_empty, (uint32_t)((nq - 1) & 1), abort, a.wait_limit)))) return;
            const int nqt = KEYS || it.alone ? 1 : 2;
            mbar_expect_tx(q_full, (uint32_t)(nqt * L::TILE));
            for (int x = 0; x < nqt; ++x)
#pragma unroll
              for (int d = 0; d < D; d += 64)
                tma_load_3d(sb + (uint32_t)(L::Q + (size_t)x * L::TILE + d / 64 * L::HALF), &a.qmap, d, it.h * G,
                            (int)rq.row0 + it.t0 + x * TOK, q_full);
            ++nq;
          };
          if (KEYS) {
            tile(&a.kmap, it.kb);
            if (w.cnt[1] > 0) tile(&a.kmap, it.kb + 1);
            for (int j = 0; j < w.cnt[0]; ++j) {
              tile(&a.vmap, it.kb + 2 * j);
              if (j == 0) queries();
              if (j + 1 < w.cnt[0]) tile(&a.kmap, it.kb + 2 * j + 2);
              if (j < w.cnt[1]) tile(&a.vmap, it.kb + 2 * j + 1);
              if (j + 1 < w.cnt[1]) tile(&a.kmap, it.kb + 2 * j + 3);
            }
          } else {
            for (int j = it.kb; j < it.ke; ++j) {
              tile(&a.kmap, j);
              tile(&a.vmap, j);
              if (j == it.kb) queries();
            }
          }
        }
        if (!ok) timed_out();
        // every copy issued has landed before the CTA moves on (bounded)
        for (int x = c > NST ? c - NST : 0; x < c; ++x) drain_bar(full(x % NST), (uint32_t)((x / NST) & 1));
        if (nq > 0) drain_bar(q_full, (uint32_t)((nq - 1) & 1));
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---- MMA issuer --------------------------------------------------------------
      int c = 0, nq = 0;      // tiles of the ring, items
      int ns[2] = {0, 0};     // products P V per group
      int no[2] = {0, 0};     // items per group
      bool ok = true;
      auto wait = [&](uint32_t bar, int phase) {
        ok = ok && __all_sync(0xffffffffu, wait_bar(bar, (uint32_t)(phase & 1), abort, a.wait_limit));
      };
      auto stage = [&](int k) { return sb + (uint32_t)(L::ST + (size_t)(k % NST) * L::TILE); };
      auto arrived = [&](int k) { wait(full(k % NST), k / NST); };
      auto score = [&](int x, int k) {  // S of group x from the K tile k
        arrived(k);
        if (!ok) return;
        tc_fence_after();
        const uint64_t q0 = sw128_desc(sb + (uint32_t)(L::Q + (KEYS ? 0 : (size_t)x * L::TILE)));
        const uint64_t k0 = sw128_desc(stage(k));
#pragma unroll
        for (int e = 0; e < D / 16; ++e) {
          const uint64_t off = (uint64_t)(((e >> 2) * L::HALF + (e & 3) * 32) >> 4);
          mma_ss(tmem + (uint32_t)(x * 128), q0 + off, k0 + off, idesc(TK, false), e > 0 ? 1u : 0u);
        }
        commit(s_ready(x));
      };
      // O of group x from its P and the V tile k, in two steps: the second half of
      // P is still being computed when the first 64 keys' product starts
      auto value = [&](int x, int k, bool first, bool last, int& n, int& items_done) {
        arrived(k);
        if (first && items_done > 0) wait(o_free(x), items_done - 1);
        wait(p_half(x), n);
        const uint64_t v0 = sw128_mn_desc(stage(k), L::HALF);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (half) wait(p_ready(x), n);
          if (!ok) return;
          tc_fence_after();
#pragma unroll
          for (int e = 4 * half; e < 4 * half + 4; ++e)
#pragma unroll
            for (int part = 0; part < 2; ++part)
              mma_ts(tmem + (uint32_t)(256 + x * 128), tmem + (uint32_t)(x * 128 + part * 64 + e * 8),
                     v0 + (uint64_t)(e * 2048 >> 4), idesc(D, true), first && e == 0 && part == 0 ? 0u : 1u);
        }
        ++n;
        if (last) {
          commit(o_done(x));
          ++items_done;
        }
      };
      for (int i = i0; i < i1 && ok; ++i) {
        const ChunkItem it = load_item(items + i);
        Work w = work_of<G, KEYS>(it, load_req(a.reqs + it.r));
        w.n = uniform(w.n);
        w.cnt[0] = uniform(w.cnt[0]);
        w.cnt[1] = uniform(w.cnt[1]);
        wait(q_full, nq++);
        if constexpr (KEYS) {
          int at = c;  // every tile serves one group; used in the order of the loads
          auto S = [&](int x, bool last) {
            score(x, at);
            if (!ok) return;
            commit(empty(at++ % NST));
            if (last) commit(q_empty);
          };
          auto V = [&](int x, int j) {
            value(x, at, j == 0, j + 1 == w.cnt[x], ns[x], no[x]);
            if (ok) commit(empty(at++ % NST));
          };
          S(0, w.n == 1);
          if (w.cnt[1] > 0 && ok) S(1, w.n == 2);
          for (int j = 0; j < w.cnt[0] && ok; ++j) {
            V(0, j);
            if (j + 1 < w.cnt[0] && ok) S(0, 2 * j + 3 == w.n);
            if (j < w.cnt[1] && ok) V(1, j);
            if (j + 1 < w.cnt[1] && ok) S(1, 2 * j + 4 == w.n);
          }
        } else {
          // K tile j is c + 2 j, V tile j the one after it; the first group may see
          // fewer tiles, the second have no query tile
          const bool two = w.cnt[1] > 0;
          if (w.cnt[0] > 0) score(0, c);
          if (two) score(1, c);
          if (!ok) break;
          commit(empty(c % NST));
          if (w.n == 1) commit(q_empty);
          for (int j = 0; j < w.n && ok; ++j) {
            const int kv = c + 2 * j + 1;
            if (j < w.cnt[0]) {
              value(0, kv, j == 0, j + 1 == w.cnt[0], ns[0], no[0]);
              if (ok && j + 1 < w.cnt[0]) score(0, kv + 1);
            }
            if (two) value(1, kv, j == 0, j + 1 == w.n, ns[1], no[1]);
            if (!ok) break;
            commit(empty(kv % NST));
            if (j + 1 < w.n) {
              if (two) score(1, kv + 1);
              if (!ok) break;
              commit(empty((kv + 1) % NST));
              if (j + 2 == w.n) commit(q_empty);
            }
          }
        }
        c += 2 * w.n;
      }
      if (!ok && lane == 0) timed_out();
      // every product issued has completed before TMEM is released (bounded)
      commit(mma_done);
      drain_bar(mma_done, 0u);
      __syncwarp();
    }
  } else {
    registers_up<208>();
    // ---- softmax and epilogue: thread = row ------------------------------------
    const int x = (warp - 4) >> 2, quad = warp & 3, row = 32 * quad + lane;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const uint32_t ts = tmem + lanes + (uint32_t)(x * 128), to = tmem + lanes + (uint32_t)(256 + x * 128);
    const float sc = 1.4426950408889634f / sqrtf((float)D);
    auto zero_rows = [&](int k, bool past) {  // this thread's row of the V tile k
      if (past) {
        unsigned char* v = sm + L::ST + (size_t)(k % NST) * L::TILE + (size_t)row * 128;
#pragma unroll
        for (int d = 0; d < D / 64; ++d)
#pragma unroll
          for (int e = 0; e < 8; ++e) reinterpret_cast<uint4*>(v + (size_t)d * L::HALF)[e] = make_uint4(0u, 0u, 0u, 0u);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    };
    int ns = 0, no = 0;  // tiles and items of this group
    int c = 0;           // tiles of all items (the ring's)
    bool ok = true;
    for (int i = i0; i < i1 && ok; ++i) {
      const ChunkItem it = load_item(items + i);
      const ChunkReq rq = load_req(a.reqs + it.r);
      const Work w = work_of<G, KEYS>(it, rq);
      const int total = rq.cached + rq.nnew;
      const int cnt = w.cnt[x];
      const int first = it.t0 + (KEYS ? 0 : x * TOK);  // the tile's first token
      const int t = first + row / G;
      const int sees = rq.cached + t;                     // last slot the row sees
      // the last key tile may hold slots past the request's tokens: their weights
      // are 0, but 0 x inf or NaN would reach O; their V rows are zeroed (by both
      // groups when both take the tile: neither waits for the other)
      auto last_of = [&](int kt) { return kt + 1 == it.ke && kt * TK + TK > total; };
      // a warp whose rows are all past the request's tokens computes nothing: its
      // rows of P hold any bits, and spoil only its rows of O
      const bool live = first + 32 * quad / G < rq.nnew;
      float m = NEG, l = 0.f;
      for (int j = 0; j < cnt; ++j) {
        const int kt = it.kb + (KEYS ? 2 * j + x : j);  // key tile
        ok = __all_sync(0xffffffffu, wait_bar(s_ready(x), (uint32_t)(ns & 1), abort, a.wait_limit));
        if (!ok) break;
        tc_fence_after();
        if (!live) {
          if (last_of(kt)) {
            const int k = c + 2 * w.n - 1;
            ok = __all_sync(0xffffffffu, wait_bar(full(k % NST), (uint32_t)((k / NST) & 1), abort, a.wait_limit));
            if (!ok) break;
            zero_rows(k, kt * TK + row >= total);
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(p_half(x));
            mbar_arrive(p_ready(x));
          }
          ++ns;
          continue;
        }
        uint32_t r[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_load32(ts + (uint32_t)(32 * q), r[q]);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_arrived(r[q]);
        if (kt * TK + TK - 1 > rq.cached + first) {  // some row of the tile does not see all of these keys
          const int keep = sees - kt * TK;           // columns 0 .. keep are seen
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * q + e > keep) r[q][e] = 0xff800000u;  // -inf
        }
        float mx[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          mx[q] = max3(__uint_as_float(r[q][0]), __uint_as_float(r[q][1]), __uint_as_float(r[q][2]));
#pragma unroll
          for (int e = 3; e < 31; e += 2) mx[q] = max3(mx[q], __uint_as_float(r[q][e]), __uint_as_float(r[q][e + 1]));
          mx[q] = fmaxf(mx[q], __uint_as_float(r[q][31]));
        }
        const float top = sc * fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (j == 0) {
          m = fmaxf(m, top);
        } else {
          const bool grow = top > m + LAZY;
          if (__any_sync(0xffffffffu, grow)) {
            // the products issued before this S have completed: O is at rest
            const float mn = grow ? top : m, f = ex2f(m - mn);
            m = mn;
            l *= f;
#pragma unroll 1
            for (int d = 0; d < D; d += 32) {
              uint32_t o[32];
              tmem_load32(to + (uint32_t)d, o);
              tmem_wait_ld();
              tmem_arrived(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_store32(to + (uint32_t)d, o);
            }
          }
        }
        const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(-m, -m);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        auto weigh = [&](int q) {  // 32 keys' weights, both parts over the logits
          uint32_t p[16], rest[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float2 z = fma2(make_float2(__uint_as_float(r[q][2 * e]), __uint_as_float(r[q][2 * e + 1])), sc2, nm2);
            z.x = ex2f(z.x);
            z.y = ex2f(z.y);
            sum[e & 1] = add2(sum[e & 1], z);
            p[e] = __byte_perm(__float_as_uint(z.x), __float_as_uint(z.y), 0x7632);  // the upper halves
            z = less_bf16(z, p[e]);
            rest[e] = pack_bf16(z.x, z.y);
          }
          tmem_store16(ts + (uint32_t)(16 * q), p);
          tmem_store16(ts + (uint32_t)(64 + 16 * q), rest);
        };
        weigh(0);
        weigh(1);
        if (last_of(kt)) {
          const int k = c + 2 * w.n - 1;  // the item's last load
          ok = __all_sync(0xffffffffu, wait_bar(full(k % NST), (uint32_t)((k / NST) & 1), abort, a.wait_limit));
          if (!ok) break;
          zero_rows(k, kt * TK + row >= total);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_half(x));
        weigh(2);
        weigh(3);
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready(x));
        ++ns;
      }
      if (!ok) break;
      // ---- epilogue ----
      const int part = x == 0 ? it.part_a : it.part_b;
      const bool valid = t < rq.nnew;
      if (cnt == 0) {  // nothing of this range is seen by the tile, or there is no second part
        if (!KEYS && part >= 0) {
          float* po = a.part + (size_t)part * chunk_part_floats(D) + 128 * D;
          po[row] = NEG;
          po[128 + row] = 0.f;
        }
      } else {
        ok = __all_sync(0xffffffffu, wait_bar(o_done(x), (uint32_t)(no & 1), abort, a.wait_limit));
        if (!ok) break;
        tc_fence_after();
        const size_t at = (size_t)(rq.row0 + t) * a.Hq + it.h * G + row % G;
        const float inv = 1.f / l;
#pragma unroll 1
        for (int d = 0; d < D; d += 32) {
          uint32_t o[32];
          tmem_load32(to + (uint32_t)d, o);
          tmem_wait_ld();
          tmem_arrived(o);
          if (valid && part < 0) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at * D + d);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t u[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                u[k] = pack_bf16(__uint_as_float(o[8 * e + 2 * k]) * inv, __uint_as_float(o[8 * e + 2 * k + 1]) * inv);
              dst[e] = make_uint4(u[0], u[1], u[2], u[3]);
            }
          } else if (valid) {
            uint4* dst = reinterpret_cast<uint4*>(a.part + (size_t)part * chunk_part_floats(D)) + (size_t)(d / 4) * 128 + row;
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[(size_t)e * 128] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
          __syncwarp();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_free(x));
        ++no;
        if (valid && part < 0 && a.lse) a.lse[at] = m + log2f(l);
        if (part >= 0) {
          float* po = a.part + (size_t)part * chunk_part_floats(D) + 128 * D;
          po[row] = m;
          po[128 + row] = l;
        }
      }
      c += 2 * w.n;
    }
    if (!ok && lane == 0) timed_out();
    tmem_wait_st();  // a loop that was left between a store and its wait
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
  }
}

// Joins the partials of a query tile: thread = (row, slice of d).
template <int D, int G>
__global__ void __launch_bounds__(256) k_chunk_join(const __grid_constant__ ChunkTcArgs a) {
  const ChunkJoin jn = load_item(a.joins + blockIdx.x);
  let_next_in();
  wait_for_previous();
  const ChunkReq rq = load_req(a.reqs + jn.r);
  const int row = threadIdx.x & 127, half = threadIdx.x >> 7;
  const int t = jn.t0 + row / G;
  if (t >= rq.nnew) return;
  const float* base = a.part + (size_t)jn.first * chunk_part_floats(D);
  float M = NEG;
#pragma unroll 8
  for (int p = 0; p < jn.n; ++p) M = fmaxf(M, __ldcg(base + p * chunk_part_floats(D) + 128 * D + row));
  float l = 0.f;
  float4 acc[2] = {};
  const int d0 = (blockIdx.y * 2 + half) * 8;  // eight dimensions
#pragma unroll 4
  for (int p = 0; p < jn.n; ++p) {
    const float* q = base + p * chunk_part_floats(D);
    const float lp = __ldcg(q + 128 * D + 128 + row);
    // a part that the row does not see has no sum, and its O may not be there
    const float f = lp > 0.f ? ex2f(__ldcg(q + 128 * D + row) - M) : 0.f;
    l = fmaf(f, lp, l);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float4 o = __ldcg(reinterpret_cast<const float4*>(q) + (size_t)(d0 / 4 + e) * 128 + row);
      if (f == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
      acc[e].x = fmaf(f, o.x, acc[e].x);
      acc[e].y = fmaf(f, o.y, acc[e].y);
      acc[e].z = fmaf(f, o.z, acc[e].z);
      acc[e].w = fmaf(f, o.w, acc[e].w);
    }
  }
  const float inv = 1.f / l;
  const size_t at = (size_t)(rq.row0 + t) * a.Hq + jn.h * G + row % G;
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at * D + d0) =
      make_uint4(pack_bf16(acc[0].x * inv, acc[0].y * inv), pack_bf16(acc[0].z * inv, acc[0].w * inv),
                 pack_bf16(acc[1].x * inv, acc[1].y * inv), pack_bf16(acc[1].z * inv, acc[1].w * inv));
  if (d0 == 0 && a.lse) a.lse[at] = M + log2f(l);
}

// ---- weights -----------------------------------------------------------------

template <int D>
struct SmW {
  static constexpr int TILE = TK * D * 2;
  static constexpr int HALF = TK * 128;
  static constexpr int NQ = D == 128 ? 2 : 6;          // query tiles in flight
  static constexpr int ROW16 = 128 * 32;               // an operand of 128 rows of 16
  static constexpr size_t K = 0;                       // two pages, two tiles each
  static constexpr size_t Q = 4 * (size_t)TILE;
  static constexpr size_t ONES = Q + (size_t)NQ * TILE;
  static constexpr size_t LSE = ONES + ROW16;          // [2]
  static constexpr size_t HALVES = LSE + 2 * ROW16;    // float [2][128]
  static constexpr size_t BARS = HALVES + 2 * 128 * 4;
  // k_full[2], k_empty[2], q_full[NQ], q_empty[NQ], t_full[2], t_empty[2], s_ready[2][2], s_free[2][2], mma_done[2]
  static constexpr int NBARS = 8 + 2 * NQ + 8 + 2;
  static constexpr size_t MISC = BARS + 8 * NBARS;
  static constexpr size_t BYTES = MISC + 64;           // the base is aligned to 1 KiB by its declaration
  static_assert(BYTES <= 232448, "227 KiB a CTA");
};

// An operand of 128 rows of 16 without swizzle: 8 x 16-byte blocks, the two of a
// row's halves 128 bytes apart, the next eight rows 256.
__device__ __forceinline__ int row16(int row) { return (row >> 3) * 256 + (row & 7) * 16; }
__device__ __forceinline__ uint64_t row16_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(128 >> 4) << 16) | ((uint64_t)(256 >> 4) << 32) |
         ((uint64_t)1 << 46);
}

template <int D, int G>
__global__ void __launch_bounds__(WNT, 1) k_chunk_weights_tc(const __grid_constant__ ChunkTcArgs a) {
  using L = SmW<D>;
  constexpr int NQ = L::NQ, TOK = 128 / G;
  extern __shared__ __align__(1024) unsigned char smem_base[];
  unsigned char* sm = smem_base;
  const uint32_t sb = static_cast<uint32_t>(__cvta_generic_to_shared(sm));
  if (sb & 1023u) {  // the swizzled tiles need it; there is no room to align here
    if (threadIdx.x == 0) atomicOr(a.err, ERR_BAD_COUNT);
    return;
  }
  int* misc = reinterpret_cast<int*>(sm + L::MISC);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(misc);
  volatile int* abort = misc + 1;
  volatile int* fail = misc + 2;  // [2] a wait of a key tile's threads gave up
  const uint32_t bar0 = sb + (uint32_t)L::BARS;
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  auto k_full = [&](int b) { return bar(b); };
  auto k_empty = [&](int b) { return bar(2 + b); };
  auto q_full = [&](int s) { return bar(4 + s); };
  auto q_empty = [&](int s) { return bar(4 + NQ + s); };
  auto t_full = [&](int b) { return bar(4 + 2 * NQ + b); };
  auto t_empty = [&](int b) { return bar(6 + 2 * NQ + b); };
  auto s_ready = [&](int x, int b) { return bar(8 + 2 * NQ + 2 * x + b); };
  auto s_free = [&](int x, int b) { return bar(12 + 2 * NQ + 2 * x + b); };
  auto mma_done = [&](int x) { return bar(16 + 2 * NQ + x); };

  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const int i0 = uniform(a.wbegin[blockIdx.x]), i1 = uniform(a.wbegin[blockIdx.x + 1]);
  let_next_in();
  if (tid == 0) {
    for (int i = 0; i < L::NBARS; ++i) {
      int n = i == 2 || i == 3 || (i >= 4 + NQ && i < 4 + 2 * NQ) ? 2 : 1;  // k_empty, q_empty: both issuers
      if (i >= 6 + 2 * NQ && i < 8 + 2 * NQ) n = 2;    // t_empty: both issuers
      if (i >= 12 + 2 * NQ && i < 16 + 2 * NQ) n = 8;  // s_free: the warps of a key tile
      mbar_init(bar(i), (uint32_t)n);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    *abort = 0;
    fail[0] = 0;
    fail[1] = 0;
  }
  // the constant parts of the operands that carry L (row16 has their layout)
  for (int row = tid; row < 128; row += WNT) {
    unsigned char* at = sm + row16(row);
    *reinterpret_cast<uint4*>(at + L::ONES) = make_uint4(0x3f803f80u, 0x00003f80u, 0u, 0u);  // 1, 1, 1, 0, ...
    *reinterpret_cast<uint4*>(at + L::ONES + 128) = make_uint4(0u, 0u, 0u, 0u);
    for (int b = 0; b < 2; ++b) *reinterpret_cast<uint4*>(at + L::LSE + b * L::ROW16 + 128) = make_uint4(0u, 0u, 0u, 0u);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(tmem_holder))),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_holder);
  wait_for_previous();  // the statistics are the attention's; the weights may be an earlier call's
  auto timed_out = [&] {
    atomicOr(a.err, ERR_TIMEOUT);
    *abort = 1;
  };

  if (warp == 0) {
    // ---- producer: an item's two K tiles, then its query tiles -------------------
    if (lane == 0) {
      int c = 0, n = 0;  // query tiles and pages issued
      bool ok = true;
      const bool patient = a.wait_limit != 0;
      for (int i = i0; i < i1 && ok; ++i) {
        const WeightItem it = load_item(a.witems + i);
        const ChunkReq rq = load_req(a.reqs + it.r);
        for (int pg = it.page; pg < it.page + it.pages; ++pg) {
          const int b = n & 1;
          if (n >= 2 && !(ok = patient && wait_bar(k_empty(b), (uint32_t)((n / 2 - 1) & 1), abort, a.wait_limit))) break;
          const int y = key_row(a, rq, it.h, 2 * pg);
          mbar_expect_tx(k_full(b), 2 * L::TILE);
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int d = 0; d < D; d += 64)
              tma_load_2d(sb + (uint32_t)(L::K + (size_t)(2 * b + x) * L::TILE + d / 64 * L::HALF), &a.kmap, d, y + x * TK,
                          k_full(b));
          ++n;
          for (int q = it.qb; q < it.qe; ++q, ++c) {
            const int s = c % NQ;
            if (c >= NQ && !(ok = patient && wait_bar(q_empty(s), (uint32_t)((c / NQ - 1) & 1), abort, a.wait_limit))) break;
            mbar_expect_tx(q_full(s), L::TILE);
#pragma unroll
            for (int d = 0; d < D; d += 64)
              tma_load_3d(sb + (uint32_t)(L::Q + (size_t)s * L::TILE + d / 64 * L::HALF), &a.qmap, d, it.h * G,
                          (int)rq.row0 + q * TOK, q_full(s));
          }
          if (!ok) break;
        }
      }
      if (!ok) timed_out();
      for (int x = c > NQ ? c - NQ : 0; x < c; ++x) drain_bar(q_full(x % NQ), (uint32_t)((x / NQ) & 1));
      for (int x = n > 2 ? n - 2 : 0; x < n; ++x) drain_bar(k_full(x & 1), (uint32_t)((x / 2) & 1));
    }
    __syncwarp();
  } else if (warp < 3) {
    // ---- MMA issuers, one a key tile -----------------------------------------------
    const int x = warp - 1;
    int c = 0, n = 0;
    bool ok = true;
    auto wait = [&](uint32_t b, int phase) {
      ok = ok && __all_sync(0xffffffffu, wait_bar(b, (uint32_t)(phase & 1), abort, a.wait_limit));
    };
    for (int i = i0; i < i1 && ok; ++i) {
      const WeightItem it = load_item(a.witems + i);
      const int pages = uniform(it.pages), tiles = uniform(it.qe - it.qb);
      for (int pg = 0; pg < pages && ok; ++pg, ++n) {
        const int b = n & 1;
        wait(k_full(b), n / 2);
        const uint64_t k0 = sw128_desc(sb + (uint32_t)(L::K + (size_t)(2 * b + x) * L::TILE));
        for (int q = 0; q < tiles && ok; ++q, ++c) {
          const int s = c % NQ, z = c & 1;
          wait(q_full(s), c / NQ);
          if (c >= 2) wait(s_free(x, z), c / 2 - 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t q0 = sw128_desc(sb + (uint32_t)(L::Q + (size_t)s * L::TILE));
          wait(t_full(z), c / 2);
          if (!ok) break;
#pragma unroll
          for (int e = 0; e < D / 16; ++e) {
            const uint64_t off = (uint64_t)(((e >> 2) * L::HALF + (e & 3) * 32) >> 4);
            mma_ss(tmem + (uint32_t)(x * 256 + z * 128), k0 + off, q0 + off, idesc(128, false), e > 0 ? 1u : 0u);
          }
          mma_ss(tmem + (uint32_t)(x * 256 + z * 128), row16_desc(sb + (uint32_t)L::ONES),
                 row16_desc(sb + (uint32_t)(L::LSE + z * L::ROW16)), idesc(128, false), 1u);
          commit(t_empty(z));
          commit(s_ready(x, z));
          commit(q_empty(s));
        }
        if (ok) commit(k_empty(b));
      }
    }
    if (!ok && lane == 0) timed_out();
    commit(mma_done(x));
    drain_bar(mma_done(x), 0u);
    __syncwarp();
  } else if (warp == 3) {
    // ---- -L / c of the query tiles, in three bf16 parts ---------------------------
    const float inv_sc = sqrtf((float)D) / 1.4426950408889634f;
    int c = 0;
    bool ok = true;
    for (int i = i0; i < i1 && ok; ++i) {
      const WeightItem it = load_item(a.witems + i);
      const ChunkReq rq = load_req(a.reqs + it.r);
      for (int pg = 0; pg < it.pages && ok; ++pg)
        for (int q = it.qb; q < it.qe; ++q, ++c) {
          const int b = c & 1;
          float v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int row = 32 * k + lane, t = q * TOK + row / G;
            v[k] = t < rq.nnew ? -inv_sc * __ldcg(a.lse + (size_t)(rq.row0 + t) * a.Hq + it.h * G + row % G) : 0.f;
          }
          if (c >= 2) ok = __all_sync(0xffffffffu, wait_bar(t_empty(b), (uint32_t)((c / 2 - 1) & 1), abort, a.wait_limit));
          if (!ok) break;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float h1 = __bfloat162float(__float2bfloat16_rn(v[k]));
            const float h2 = __bfloat162float(__float2bfloat16_rn(v[k] - h1));
            *reinterpret_cast<uint4*>(sm + L::LSE + b * L::ROW16 + row16(32 * k + lane)) =
                make_uint4(pack_bf16(h1, h2), pack_bf16(v[k] - h1 - h2, 0.f), 0u, 0u);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(t_full(b));
        }
    }
    if (!ok && lane == 0) timed_out();
  } else if (warp >= 4) {
    // ---- sums: thread = (key, half of the columns) ---------------------------------
    const int x = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1, quad = warp & 3, key = 32 * quad + lane;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16;
    const float sc = 1.4426950408889634f / sqrtf((float)D);
    const float2 sc2 = make_float2(sc, sc);
    float* other = reinterpret_cast<float*>(sm + L::HALVES) + x * 128 + key;  // the upper half's sum
    int c = 0;
    bool ok = true;
    for (int i = i0; i < i1 && ok; ++i) {
      const WeightItem it = load_item(a.witems + i);
      const ChunkReq rq = load_req(a.reqs + it.r);
      for (int pg = it.page; pg < it.page + it.pages && ok; ++pg) {
        const int slot_i = pg * PAGE + x * TK + key;  // this thread's logical slot
        // the weight so far is on its way while the products run
        auto mine = [&] { return half == 0 && slot_i < rq.cached + rq.nnew && rq.slot >= 0 && rq.slot < a.M; };
        auto weight = [&] { return a.weights + (((size_t)a.layer * a.M + rq.slot) * a.Hkv + it.h) * a.cap + slot_i; };
        const float so_far = it.part < 0 && mine() ? *weight() : 0.f;
        float2 w[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        for (int q = it.qb; q < it.qe; ++q, ++c) {
          const int z = c & 1;
          ok = __all_sync(0xffffffffu, wait_bar(s_ready(x, z), (uint32_t)((c / 2) & 1), abort, a.wait_limit));
          if (!ok) break;
          tc_fence_after();
          // of this half's columns lo .. hi - 1 count: rows of tokens that see the slot and exist
          const int lo = (slot_i - rq.cached - q * TOK) * G - half * 64, hi = (rq.nnew - q * TOK) * G - half * 64;
          if (hi > 0) {
            uint32_t r[2][32];
#pragma unroll
            for (int h = 0; h < 2; ++h)
              tmem_load32(tmem + lanes + (uint32_t)(x * 256 + z * 128 + half * 64 + h * 32), r[h]);
            tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < 2; ++h) tmem_arrived(r[h]);
            if (__any_sync(0xffffffffu, lo > 0 || hi < 64)) {
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (32 * h + e < lo || 32 * h + e >= hi) r[h][e] = 0xff800000u;  // -inf
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                float2 u = mul2(make_float2(__uint_as_float(r[h][4 * e]), __uint_as_float(r[h][4 * e + 1])), sc2);
                float2 v = mul2(make_float2(__uint_as_float(r[h][4 * e + 2]), __uint_as_float(r[h][4 * e + 3])), sc2);
                u.x = ex2f(u.x);
                u.y = ex2f(u.y);
                v.x = ex2f(v.x);
                v.y = ex2f(v.y);
                w[e & 1] = add2(w[e & 1], u);
                w[2 + (e & 1)] = add2(w[2 + (e & 1)], v);
              }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(s_free(x, z));
          }
        }
        // the two halves of a key's sum meet (both groups of threads come here,
        // whether a wait gave up or not)
        float sum = ((w[0].x + w[0].y) + (w[1].x + w[1].y)) + ((w[2].x + w[2].y) + (w[3].x + w[3].y));
        if (half) *other = sum;
        if (!ok) fail[x] = 1;  // written only before the barrier: all of the key tile's threads agree
        asm volatile("bar.sync %0, 256;" ::"r"(1 + x) : "memory");
        ok = !fail[x];
        if (!half) sum += *other;
        asm volatile("bar.sync %0, 256;" ::"r"(1 + x) : "memory");
        if (!ok) break;
        if (half) continue;
        if (it.part >= 0) a.wpart[(size_t)it.part * PAGE + x * TK + key] = sum;
        else if (mine()) *weight() = so_far + sum;
      }
    }
    if (!ok && lane == 0) timed_out();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
  }
}

// Adds the partial sums of a page, in the order of its parts.
__global__ void __launch_bounds__(PAGE) k_chunk_weights_join(const __grid_constant__ ChunkTcArgs a) {
  const WeightJoin jn = load_item(a.wjoins + blockIdx.x);
  wait_for_previous();
  const ChunkReq rq = load_req(a.reqs + jn.r);
  const int i = jn.page * PAGE + (int)threadIdx.x;
  if (i >= rq.cached + rq.nnew || rq.slot < 0 || rq.slot >= a.M) return;
  float* dst = a.weights + (((size_t)a.layer * a.M + rq.slot) * a.Hkv + jn.h) * a.cap + i;
  const float so_far = *dst;
  float w = 0.f;
#pragma unroll 8
  for (int p = 0; p < jn.n; ++p) w += __ldcg(a.wpart + (size_t)(jn.first + p) * PAGE + threadIdx.x);
  *dst = so_far + w;
}

template <int D, int G, bool KEYS>
cudaError_t attention_launch(const ChunkTcArgs& a, int grid, bool chained, cudaStream_t s) {
  if (grid == 0) return cudaSuccess;
  constexpr int smem = (int)Sm<D, KEYS>::BYTES;
  const cudaError_t e = cudaFuncSetAttribute(k_chunk_tc<D, G, KEYS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  if (chained) return launch_chained(k_chunk_tc<D, G, KEYS>, dim3((unsigned)grid), NT, smem, s, a);
  k_chunk_tc<D, G, KEYS><<<dim3((unsigned)grid), NT, smem, s>>>(a);
  return cudaGetLastError();
}
template <int D, int G>
cudaError_t attention(const ChunkTcArgs& a, cudaStream_t s) {
  cudaError_t e = attention_launch<D, G, false>(a, a.grid, false, s);
  if (e == cudaSuccess) e = attention_launch<D, G, true>(a, a.kgrid, a.grid > 0, s);
  if (e != cudaSuccess || a.n_joins == 0) return e;
  return launch_chained(k_chunk_join<D, G>, dim3((unsigned)a.n_joins, D / 16), 256, 0, s, a);
}
template <int D, int G>
cudaError_t weights(const ChunkTcArgs& a, cudaStream_t s) {
  cudaError_t e =
      cudaFuncSetAttribute(k_chunk_weights_tc<D, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SmW<D>::BYTES);
  if (e != cudaSuccess) return e;
  e = launch_chained(k_chunk_weights_tc<D, G>, dim3((unsigned)a.wgrid), WNT, SmW<D>::BYTES, s, a);
  if (e != cudaSuccess || a.n_wjoins == 0) return e;
  return launch_chained(k_chunk_weights_join, dim3((unsigned)a.n_wjoins), PAGE, 0, s, a);
}

}  // namespace

cudaError_t launch_chunk_tc(const ChunkTcArgs& a, cudaStream_t s) {
  if (a.grid + a.kgrid < 1 || !chunk_tc_shape(a.D, a.G)) return cudaErrorInvalidValue;
  if (a.D == 128) return a.G == 4 ? attention<128, 4>(a, s) : attention<128, 2>(a, s);
  return a.G == 4 ? attention<64, 4>(a, s) : attention<64, 2>(a, s);
}
cudaError_t launch_chunk_weights_tc(const ChunkTcArgs& a, cudaStream_t s) {
  if (a.wgrid < 1 || !chunk_tc_shape(a.D, a.G)) return cudaErrorInvalidValue;
  if (a.D == 128) return a.G == 4 ? weights<128, 4>(a, s) : weights<128, 2>(a, s);
  return a.G == 4 ? weights<64, 4>(a, s) : weights<64, 2>(a, s);
}

}  // namespace gp
