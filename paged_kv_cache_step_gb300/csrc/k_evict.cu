// Eviction by accumulated attention weight, per (request, layer, KV head):
// the `recent` last tokens stay, and of the others the keep - recent of the
// largest accumulated weight (equal weights: the lower slot); the kept rows
// of K, V and the weights move, in order, to the logical slots [0, keep).
//
// Two kernels:
//   select  one CTA a unit: radix select (11 + 11 + 10 bits of an
//           order-preserving key, fewer when a bin is kept whole) of the
//           threshold, then one ordered pass that writes the kept slot of every
//           rank, and how many slots are kept below the first slot of every
//           move item.
//   move    in place, many warps a unit.  An item is evict_rows consecutive
//           ranks -- target slots [kR, (k+1)R), consecutive rows of one page --
//           so its rows are always all wanted, and its K and V pass through
//           16 KB of shared memory: asynchronous copies in, a bulk copy out.
//           Writing item k destroys the rows that live in those slots; the
//           kept ones among them have ranks <= their slots, so they belong
//           to items <= k.  Warps take the items in order (a ticket), read
//           their rows at once, raise the item's flag, and only then wait for
//           the flags of the (at most two) items whose rows they will
//           overwrite: a reader never waits, so the lowest item not yet read
//           is always read, and every wait ends.  Waits are bounded all the
//           same.  Fourteen warps an SM keep 224 KB of items on their way, each
//           at a step of its own (ticket, kept slots, pages, rows, flags).
//           Items are numbered across the units: unit by unit, most of a unit's
//           items were in flight at once and waited for one another's reads
//           (4.8 TB/s against 6.4).
// Bounded by HBM: kept rows are read and written once.  Ten requests of 77 671
// tokens to 37 %, 32 layers of 8 heads, d = 128, bf16: 7.5 GB moved in 1176 us, 6.4
// TB/s, 94 % of the copy rate, after 99 us of selection (which is bound by the
// issue of its passes over the keys in shared memory: three at most that count
// digits, and the ordered one).
#include <cstdint>

#include "chained.cuh"
#include "weighted_kernels.h"

namespace gp {
namespace {

constexpr int PAGE = 256;
constexpr int SNT = 512;    // select
constexpr int BINS = 2048;  // a digit of 11 bits
constexpr int MWARPS = 14;         // move: warps of a CTA, one CTA per SM,
constexpr int STAGE = 16 * 1024;   // each with an item's K and V rows

// Order-preserving key of a weight; -0 counts as 0, NaN as the largest.
__device__ __forceinline__ unsigned okey(float v) {
  if (v != v) return 0xffffffffu;
  const unsigned u = __float_as_uint(v + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// A warp has consecutive words (32 slots each) of the unit.  STAGED: the keys
// are formed once and stay in shared memory for the passes over them, else the
// weights are read again at each.  (In registers, 16 a thread, they left one CTA an
// SM: 96 us against 70 for 1024 units of 8192 slots, read again each pass.)
template <bool STAGED>
__global__ void __launch_bounds__(SNT) k_evict_select(const __grid_constant__ EvictArgs a) {
  constexpr int SWARP = SNT / 32, PER_BIN = BINS / SNT;
  extern __shared__ unsigned staged[];
  __shared__ unsigned hist[BINS];
  __shared__ unsigned wsum[SWARP], weq[SWARP];
  __shared__ unsigned s_bin, s_above;
  __shared__ bool s_whole;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int units = a.L * a.Hkv;
  const int r = blockIdx.x / units, unit = blockIdx.x % units;
  const EvictReq rq = a.reqs[r];
  let_next_in();
  if (blockIdx.x == 0 && tid == 0) *a.ticket = 0ull;
  if (rq.items == 0) return;  // nothing to evict
  const int nw = (rq.T + 31) / 32;
  const float* w0 = a.weights + (((size_t)(unit / a.Hkv) * a.M + rq.slot) * a.Hkv + unit % a.Hkv) * a.cap;
  const int ncand = rq.T - rq.recent;
  const unsigned need = (unsigned)(rq.keep - rq.recent);  // 0 <= need < ncand
  const int per = (nw + SWARP - 1) / SWARP, wa = min(nw, warp * per), wb = min(nw, wa + per);
  if constexpr (STAGED) {
    for (int i = tid; i < ncand; i += 8 * SNT) {  // eight loads in flight
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = i + j * SNT < ncand ? w0[i + j * SNT] : 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j * SNT < ncand) staged[i + j * SNT] = okey(v[j]);
    }
  }
  unsigned* flags = a.flags + rq.item0 + (size_t)unit * rq.items;
  for (int k = tid; k < rq.items; k += SNT) flags[k] = 0u;
  // f(word, key) for words [from, to) in order; the key counts where slot < ncand
  auto each_word = [&](int from, int to, auto&& f) {
    if constexpr (STAGED) {
#pragma unroll 4
      for (int w = from; w < to; ++w) f(w, 32 * w + lane < ncand ? staged[32 * w + lane] : 0u);
    } else {
      for (int w = from; w < to; w += 8) {  // eight loads in flight
        unsigned k[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int s = 32 * (w + j) + lane;
          k[j] = w + j < to && s < ncand ? okey(w0[s]) : 0u;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (w + j < to) f(w + j, k[j]);
      }
    }
  };
  if (need == 0) __syncthreads();  // the keys are staged (the passes below begin with a barrier)

  // ---- the need-th largest key: prefix, and how many keys lie above it ----
  // `whole`: the keys of the prefix's last bin are just as many as still wanted,
  // so all of them are kept and the digits left need not be known
  unsigned prefix = 0u, mask_bits = 0u, above = 0u;
  bool whole = false;
  if (need > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3 && !whole; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const unsigned digit = pass == 2 ? 1023u : 2047u;
      for (int b = tid; b < BINS; b += SNT) hist[b] = 0u;
      __syncthreads();
      each_word(wa, wb, [&](int w, unsigned k) {
        if (32 * w + lane < ncand && (k & mask_bits) == prefix) atomicAdd(&hist[(k >> shift) & digit], 1u);
      });
      __syncthreads();
      // thread t owns the PER_BIN bins from BINS - 1 - PER_BIN t down
      unsigned c[PER_BIN], own = 0u;
#pragma unroll
      for (int j = 0; j < PER_BIN; ++j) {
        c[j] = hist[BINS - 1 - PER_BIN * tid - j];
        own += c[j];
      }
      unsigned inc = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      if (lane == 31) wsum[warp] = inc;
      __syncthreads();
      unsigned cum = inc - own;
      for (int w = 0; w < warp; ++w) cum += wsum[w];
      const unsigned want = need - above;
      if (cum < want && want <= cum + own) {  // one thread: the bins' counts sum to at least `want`
        bool found = false;
#pragma unroll
        for (int j = 0; j < PER_BIN; ++j) {
          if (!found && want <= cum + c[j]) {
            found = true;
            s_bin = (unsigned)(BINS - 1 - PER_BIN * tid - j);
            s_above = cum;
            s_whole = want == cum + c[j];
          }
          cum += c[j];
        }
      }
      __syncthreads();
      prefix |= s_bin << shift;
      mask_bits |= digit << shift;
      above += s_above;
      whole = s_whole;
    }
  }
  const unsigned thr = prefix, take_eq = whole ? 0u : need - above;  // of the keys equal to thr, the first take_eq

  // ---- the ordered pass ------------------------------------------------------
  // lane j holds the bits of the warp's words j, j + 32, ...: the slots kept
  // whatever the ties, and the ties
  constexpr int BLOCKS = 65536 / 32 / SWARP / 32;  // of 32 words a warp, at most
  unsigned sure[BLOCKS], tie[BLOCKS];
#pragma unroll
  for (int b = 0; b < BLOCKS; ++b) {
    sure[b] = tie[b] = 0u;
    const int first = wa + 32 * b;
    each_word(first, min(first + 32, wb), [&](int w, unsigned k) {
      const int s = 32 * w + lane;
      const bool cand = s < ncand && need > 0;
      const unsigned bs = __ballot_sync(0xffffffffu, cand ? (whole ? k >= thr : k > thr) : s >= ncand && s < rq.T);
      const unsigned bt = __ballot_sync(0xffffffffu, cand && !whole && k == thr);
      if (w - first == lane) {
        sure[b] = bs;
        tie[b] = bt;
      }
    });
  }
  unsigned cnt = 0u, eqs = 0u;
#pragma unroll
  for (int b = 0; b < BLOCKS; ++b) {
    cnt += __popc(sure[b]);
    eqs += __popc(tie[b]);
  }
  cnt = __reduce_add_sync(0xffffffffu, cnt);
  eqs = __reduce_add_sync(0xffffffffu, eqs);
  __syncthreads();  // wsum has been read above
  if (lane == 0) {
    wsum[warp] = cnt;
    weq[warp] = eqs;
  }
  __syncthreads();
  unsigned before = 0u, eq_before = 0u;  // kept slots and ties before this warp's words
  for (int w = 0; w < warp; ++w) {
    before += wsum[w];
    eq_before += weq[w];
  }
  before += min(eq_before, take_eq);
  const int rlog = 31 - __clz(evict_rows(a.row_bytes));  // rows of an item, a power of two
  uint16_t* idx = a.idx + rq.idx_off + (size_t)unit * rq.idx_pitch;
  int32_t* pre = a.pre + rq.pre_off + (size_t)unit * (rq.items + 1);
  // the kept slots go out through shared memory, in whole lines
  uint16_t* list = STAGED ? reinterpret_cast<uint16_t*>(staged + (ncand + 3) / 4 * 4) : idx;
#pragma unroll
  for (int b = 0; b < BLOCKS; ++b) {
    if (wa + 32 * b >= wb) break;
    const int w = wa + 32 * b + lane;
    // ties before this lane's word, then the ties of it that are kept: its first ones
    unsigned eq = __popc(tie[b]), inc = eq;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const unsigned eq_mine = eq_before + inc - eq, room = take_eq > eq_mine ? take_eq - eq_mine : 0u;
    unsigned t = tie[b];
    for (; eq > room; --eq) t &= ~(0x80000000u >> __clz(t));
    eq_before += __shfl_sync(0xffffffffu, inc, 31);
    unsigned kept = sure[b] | t;
    const unsigned n = __popc(kept);
    inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    unsigned rank = before + inc - n;  // kept slots before this lane's word
    before += __shfl_sync(0xffffffffu, inc, 31);
    if (w < wb) {
      if (rlog < 5) {  // 16 rows an item: two items a word
        if (2 * w <= rq.items) pre[2 * w] = (int32_t)rank;
        if (2 * w + 1 <= rq.items) pre[2 * w + 1] = (int32_t)(rank + __popc(kept & 0xffffu));
      } else if (((32 * w) & ((1 << rlog) - 1)) == 0 && (32 * w) >> rlog <= rq.items) {
        pre[(32 * w) >> rlog] = (int32_t)rank;
      }
    }
    for (; kept; kept &= kept - 1u) list[rank++] = (uint16_t)(32 * w + __ffs(kept) - 1);
  }
  if (tid == 0 && rq.items << rlog >= 32 * nw) pre[rq.items] = rq.keep;
  if constexpr (STAGED) {
    __syncthreads();
    uint4* dst = reinterpret_cast<uint4*>(idx);  // every unit's list starts on 16 bytes
    const uint4* src = reinterpret_cast<const uint4*>(list);
    for (int i = tid; i < (rq.keep + 7) / 8; i += SNT) dst[i] = src[i];
  }
}

__device__ __forceinline__ unsigned ld_acquire(const unsigned* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_relaxed(unsigned* p, unsigned v) {
  asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

template <int RB>
__global__ void __launch_bounds__(32 * MWARPS, 1) k_evict_move(const __grid_constant__ EvictArgs a) {
  constexpr int R = evict_rows(RB);        // rows of an item
  constexpr int PIECES = RB / 16;          // 16-byte pieces of a row
  constexpr int LOADS = R * PIECES / 32;   // pieces of K (and of V) a lane copies
  constexpr int OWN = (R + 31) / 32;       // rows a lane looks up
  static_assert((R % 32 == 0 || R == 16) && PAGE % R == 0 && 2 * R * RB == STAGE, "item shape");
  extern __shared__ __align__(128) unsigned char stages[];
  const int lane = threadIdx.x & 31;
  unsigned char* stage = stages + (size_t)(threadIdx.x >> 5) * STAGE;  // this warp's K rows, then V rows
  const uint32_t st = static_cast<uint32_t>(__cvta_generic_to_shared(stage));
  unsigned char* kc = static_cast<unsigned char*>(a.k_cache);
  unsigned char* vc = static_cast<unsigned char*>(a.v_cache);
  unsigned moved = 0u;
  bool fail = false, stored = false;
  uint64_t once;  // L2 policy of rows that are not read again
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
  auto take = [&] {  // the next item, in every lane
    unsigned long long t = 0ull;
    if (lane == 0) t = atomicAdd(a.ticket, 1ull);
    return (int64_t)__shfl_sync(0xffffffffu, t, 0);
  };
  struct Item {
    int64_t id;
    int k, rows;
    bool any, clear;      // some row moves; the target slots' rows are known to be read
    int wait0, wait1;     // items whose flags that takes, -1: none
    size_t dst;           // byte offset of the targets in K (and V)
    float* wrow;
    unsigned* flags;
    int src[OWN];         // the lane's rows lane, lane + 32, ...: slot,
    long long off[OWN];   // byte offset, -1: no row,
    float wv[OWN];        // weight
    unsigned stay;        // bit o: the row stays where it is
  };
  EvictReq rq{};
  int64_t rq_end = -1;  // first item past rq's
  auto look_up = [&](int64_t id) {
    Item it;
    it.id = id;
    it.any = false;
    if (id >= a.items) return it;
    if (id >= rq_end) {  // items come in order: mostly the request of the last one
      int lo = 0, hi = a.n;  // reqs[lo].item0 <= id < reqs[hi].item0
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.reqs[mid].item0 <= id) lo = mid;
        else hi = mid;
      }
      rq = a.reqs[lo];
      rq_end = rq.item0 + (int64_t)rq.items * a.L * a.Hkv;
    }
    const int units = a.L * a.Hkv;
    const int unit = (int)((id - rq.item0) % units), k = (int)((id - rq.item0) / units);
    const int layer = unit / a.Hkv, h = unit % a.Hkv;
    const int32_t* ob = a.old_bt + rq.bt_off;
    const int32_t* pre = a.pre + rq.pre_off + (size_t)unit * (rq.items + 1);
    const size_t lbase = (size_t)layer * a.num_pages_total;
    it.k = k;
    it.rows = min(R, rq.keep - k * R);
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
      const int r = lane + 32 * o;
      it.src[o] = r < it.rows ? (int)a.idx[rq.idx_off + (size_t)unit * rq.idx_pitch + k * R + r] : -1;
    }
    const int p0 = pre[k], p1 = pre[k + 1];
    const int dpage = a.new_bt[rq.bt_off + k * R / PAGE];  // an item's targets share a page
    const bool same_page = ob[k * R / PAGE] == dpage;
    it.dst = ((lbase + dpage) * a.Hkv + h) * (size_t)(PAGE * RB) + (size_t)(k * R % PAGE) * RB;
    it.wrow = a.weights + (((size_t)layer * a.M + rq.slot) * a.Hkv + h) * a.cap;
    it.flags = a.flags + rq.item0 + (size_t)unit * rq.items;
    // the kept rows in the target slots have ranks p0 .. p1 - 1: two items at most, none above k
    it.wait0 = p1 > p0 && p0 / R < k ? p0 / R : -1;
    it.wait1 = p1 > p0 && (p1 - 1) / R != p0 / R && (p1 - 1) / R < k ? (p1 - 1) / R : -1;
    const int mine = lane == 0 ? it.wait0 : lane == 1 ? it.wait1 : -1;
    it.clear = __all_sync(0xffffffffu, mine < 0 || (a.wait_limit > 0 && ld_acquire(it.flags + max(mine, 0)) != 0u));
    it.stay = 0u;
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
      if (it.src[o] < 0 || (same_page && it.src[o] == k * R + lane + 32 * o)) it.stay |= 1u << o;
      it.off[o] = -1;
      it.wv[o] = 0.f;
      if (it.src[o] >= 0) {
        it.off[o] = (long long)(((lbase + ob[it.src[o] / PAGE]) * a.Hkv + h) * (size_t)(PAGE * RB) +
                                (size_t)(it.src[o] % PAGE) * RB);
        it.wv[o] = it.wrow[it.src[o]];
      }
    }
    it.any = __any_sync(0xffffffffu, it.stay != (1u << OWN) - 1u);
    return it;
  };
  wait_for_previous();
  Item it = look_up(take());
  while (it.id < a.items && !fail) {
    // ---- read: consecutive lanes copy consecutive pieces of a row ----
    if (it.any) {
      if (stored && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the stage is free
      __syncwarp();
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int row = (32 * i + lane) / PIECES, q = (32 * i + lane) % PIECES;
        const long long at = __shfl_sync(0xffffffffu, it.off[i / PIECES], row & 31);
        if (at >= 0) {
          const uint32_t d = st + (uint32_t)(row * RB + q * 16);
          asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(d), "l"(kc + at + q * 16),
                       "l"(once)
                       : "memory");
          asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(d + (uint32_t)(R * RB)),
                       "l"(vc + at + q * 16), "l"(once)
                       : "memory");
        }
      }
    }
    // the next item's ticket, slots and pages come with the rows.  The items
    // before it are read all the same: this warp reads its own before it waits.
    const Item next = look_up(take());
    if (it.any) {
      asm volatile("cp.async.wait_all;" ::: "memory");
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the rows are stored from there by a bulk copy
    }
    __threadfence();  // every lane's reads come before the flag
    __syncwarp();
    if (lane == 0) st_relaxed(it.flags + it.k, 1u);  // a release, with the fence
    if (it.any) {
      // ---- the rows that live in the target slots have been read ----
      if (!it.clear) {
        const int mine = lane == 0 ? it.wait0 : lane == 1 ? it.wait1 : -1;
        if (mine >= 0) {
          const long long t0 = clock64();
          bool ok = false;
          while (!ok) {
            if (clock64() - t0 >= a.wait_limit) break;
            ok = ld_acquire(it.flags + mine) != 0u;
          }
          fail = !ok;
        }
        fail = __any_sync(0xffffffffu, fail);
        if (fail) break;
      }
      // ---- write: the targets are consecutive ----
      if (lane == 0) {
        const uint32_t bytes = (uint32_t)(it.rows * RB);
        asm volatile("fence.proxy.async;" ::: "memory");  // after what the flags told
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(kc + it.dst), "r"(st), "r"(bytes)
                     : "memory");
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(vc + it.dst),
                     "r"(st + (uint32_t)(R * RB)), "r"(bytes)
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
      stored = true;
#pragma unroll
      for (int o = 0; o < OWN; ++o)
        if (!((it.stay >> o) & 1u)) {
          it.wrow[it.k * R + lane + 32 * o] = it.wv[o];
          ++moved;
        }
    }
    it = next;
  }
  if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  if (fail && lane == 0) atomicOr(a.err, ERR_TIMEOUT);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) moved += __shfl_xor_sync(0xffffffffu, moved, o);
  if (lane == 0 && moved) atomicAdd(a.moved, (unsigned long long)moved);
}

template <int RB>
cudaError_t launch_rb(const EvictArgs& a, cudaStream_t s) {
  constexpr int smem = MWARPS * STAGE;
  const cudaError_t e = cudaFuncSetAttribute(k_evict_move<RB>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t grid = a.items < (int64_t)a.sms ? a.items : (int64_t)a.sms;
  return launch_chained(k_evict_move<RB>, dim3((unsigned)grid), 32 * MWARPS, smem, s, a);
}

}  // namespace

cudaError_t launch_evict_select(const EvictArgs& a, cudaStream_t s) {
  if (a.n == 0) return cudaSuccess;
  const int64_t grid = (int64_t)a.n * a.L * a.Hkv;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  // a key and a place in the list of kept slots each, and the list's last piece
  const size_t smem = (sizeof(unsigned) + sizeof(uint16_t)) * (size_t)a.longest + 64;
  constexpr size_t most = 208 * 1024;
  if (smem > most) {  // over 35 488 slots
    k_evict_select<false><<<dim3((unsigned)grid), SNT, 0, s>>>(a);
  } else {
    // the limit is the function's, whoever launches it: always the same, so that a
    // thread with a shorter request does not lower it between here and the launch
    const cudaError_t e = cudaFuncSetAttribute(k_evict_select<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return e;
    k_evict_select<true><<<dim3((unsigned)grid), SNT, smem, s>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_evict_move(const EvictArgs& a, cudaStream_t s) {
  if (a.items == 0) return cudaSuccess;
  if (a.wait_limit < 0) return cudaErrorInvalidValue;
  switch (a.row_bytes) {
    case 128: return launch_rb<128>(a, s);
    case 256: return launch_rb<256>(a, s);
    case 512: return launch_rb<512>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace gp
