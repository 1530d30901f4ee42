// Eviction by accumulated attention weight, per (request, layer, KV head):
// the `recent` last tokens stay, and of the others the keep - recent of the
// largest accumulated weight (equal weights: the lower slot); the kept rows
// of K, V and the weights move, in order, to the logical slots [0, keep).
//
// Two kernels:
//   select  one CTA a unit: radix select (11 + 11 + 10 bits of an
//           order-preserving key) of the threshold, then one ordered pass that
//           writes the keep mask, the kept slot of every rank, and how many
//           slots are kept below the first slot of every move item.
//   move    in place, many CTAs a unit.  An item is evict_rows consecutive
//           ranks -- target slots [kR, (k+1)R) -- so its rows are always all
//           wanted, and its 32 KB of K and V pass through registers.
//           Writing item k destroys the rows that live in those slots; the
//           kept ones among them have ranks <= their slots, so they belong
//           to items <= k.  CTAs take the items in order (a ticket), read
//           their rows at once, raise the item's flag, and only then wait for
//           the flags of the (at most two) items whose rows they will
//           overwrite: a reader never waits, so the lowest item not yet read
//           is always read, and every wait ends.  Waits are bounded all the
//           same.
// Bounded by HBM: kept rows are read and written once.
#include <cstdint>

#include "weighted_kernels.h"

namespace gp {
namespace {

constexpr int PAGE = 256;
constexpr int SNT = 512;  // select
constexpr int SWARP = SNT / 32;
constexpr int BINS = 2048;
constexpr int MNT = 256;  // move

// Order-preserving key of a weight; -0 counts as 0, NaN as the largest.
__device__ __forceinline__ unsigned okey(float v) {
  if (v != v) return 0xffffffffu;
  const unsigned u = __float_as_uint(v + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(SNT) k_evict_select(const __grid_constant__ EvictArgs a) {
  __shared__ unsigned hist[BINS];
  __shared__ unsigned wsum[SWARP], weq[SWARP];
  __shared__ unsigned s_bin, s_above;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int units = a.L * a.Hkv;
  const int r = blockIdx.x / units, unit = blockIdx.x % units;
  const EvictReq rq = a.reqs[r];
  if (blockIdx.x == 0 && tid == 0) *a.ticket = 0ull;
  uint32_t* mask = a.masks + rq.mask_off + (size_t)unit * rq.words;
  const int nw = (rq.T + 31) / 32;
  for (int w = nw + tid; w < rq.words; w += SNT) mask[w] = 0u;
  if (rq.items == 0) {  // nothing to evict
    for (int w = tid; w < nw; w += SNT) mask[w] = rq.T - 32 * w >= 32 ? 0xffffffffu : (1u << (rq.T - 32 * w)) - 1u;
    return;
  }
  unsigned* flags = a.flags + rq.item0 + (size_t)unit * rq.items;
  for (int k = tid; k < rq.items; k += SNT) flags[k] = 0u;
  const float* w0 = a.weights + (((size_t)(unit / a.Hkv) * a.M + rq.slot) * a.Hkv + unit % a.Hkv) * a.cap;
  const int ncand = rq.T - rq.recent;
  const unsigned need = (unsigned)(rq.keep - rq.recent);  // 0 <= need < ncand

  // ---- the need-th largest key: prefix, and how many keys lie above it ----
  unsigned prefix = 0u, mask_bits = 0u, above = 0u;
  if (need > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const unsigned digit = pass == 2 ? 1023u : 2047u;
      for (int b = tid; b < BINS; b += SNT) hist[b] = 0u;
      __syncthreads();
      for (int i = tid; i < ncand; i += SNT) {
        const unsigned k = okey(w0[i]);
        if ((k & mask_bits) == prefix) atomicAdd(&hist[(k >> shift) & digit], 1u);
      }
      __syncthreads();
      // thread t owns the four bins from BINS - 1 - 4 t down
      unsigned c[4], own = 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c[j] = hist[BINS - 1 - 4 * tid - j];
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
        int j = 0;
        while (j < 3 && cum + c[j] < want) cum += c[j++];
        s_bin = (unsigned)(BINS - 1 - 4 * tid - j);
        s_above = cum;
      }
      __syncthreads();
      prefix |= s_bin << shift;
      mask_bits |= digit << shift;
      above += s_above;
      __syncthreads();
    }
  }
  const unsigned thr = prefix, take_eq = need - above;  // of the keys equal to thr, the first take_eq

  // ---- the ordered pass: a warp has consecutive words ------------------------
  const int per = (nw + SWARP - 1) / SWARP, wa = min(nw, warp * per), wb = min(nw, wa + per);
  unsigned cnt = 0u, eqs = 0u;  // kept whatever the ties, and ties
  for (int w = wa; w < wb; ++w) {
    const int s = 32 * w + lane;
    const unsigned k = s < ncand && need > 0 ? okey(w0[s]) : 0u;
    const bool sure = (s >= ncand && s < rq.T) || (s < ncand && need > 0 && k > thr);
    cnt += __popc(__ballot_sync(0xffffffffu, sure));
    eqs += __popc(__ballot_sync(0xffffffffu, s < ncand && need > 0 && k == thr));
  }
  if (lane == 0) {
    wsum[warp] = cnt;
    weq[warp] = eqs;
  }
  __syncthreads();
  unsigned sure_before = 0u, eq_before = 0u;
  for (int w = 0; w < warp; ++w) {
    sure_before += wsum[w];
    eq_before += weq[w];
  }
  const int R = evict_rows(a.row_bytes);
  uint16_t* idx = a.idx + rq.idx_off + (size_t)unit * rq.keep;
  int32_t* pre = a.pre + rq.pre_off + (size_t)unit * (rq.items + 1);
  for (int w = wa; w < wb; ++w) {
    const int s = 32 * w + lane;
    const unsigned k = s < ncand && need > 0 ? okey(w0[s]) : 0u;
    const bool sure = (s >= ncand && s < rq.T) || (s < ncand && need > 0 && k > thr);
    const bool tie = s < ncand && need > 0 && k == thr;
    const unsigned below = (1u << lane) - 1u;
    const unsigned bt = __ballot_sync(0xffffffffu, tie);
    const bool kept = sure || (tie && eq_before + __popc(bt & below) < take_eq);
    const unsigned bk = __ballot_sync(0xffffffffu, kept);
    const unsigned rank = sure_before + min(eq_before, take_eq);  // kept slots before this word
    if (kept) idx[rank + __popc(bk & below)] = (uint16_t)s;
    if (lane == 0) {
      mask[w] = bk;
      if ((32 * w) % R == 0 && 32 * w / R <= rq.items) pre[32 * w / R] = (int32_t)rank;
    }
    sure_before += __popc(__ballot_sync(0xffffffffu, sure));
    eq_before += __popc(bt);
  }
  if (tid == 0 && rq.items * R >= 32 * nw) pre[rq.items] = rq.keep;
}

__device__ __forceinline__ unsigned ld_acquire(const unsigned* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_release(unsigned* p, unsigned v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

template <int RB>
__global__ void __launch_bounds__(MNT) k_evict_move(const __grid_constant__ EvictArgs a) {
  constexpr int R = evict_rows(RB);   // rows of an item
  constexpr int PIECES = RB / 16;     // 16-byte pieces of a row
  constexpr int PER = R * PIECES / MNT;  // pieces of K (and of V) a thread carries
  static_assert(PER * MNT == R * PIECES && R <= MNT && R % 32 == 0 && PAGE % R == 0, "item shape");
  __shared__ unsigned long long s_item;
  __shared__ int s_src[R];  // source slot, -1: the row stays where it is
  __shared__ int s_fail;
  const int tid = threadIdx.x;
  unsigned char* kc = static_cast<unsigned char*>(a.k_cache);
  unsigned char* vc = static_cast<unsigned char*>(a.v_cache);
  unsigned moved = 0u;
  if (tid == 0) s_fail = 0;
  for (;;) {
    if (tid == 0) s_item = atomicAdd(a.ticket, 1ull);
    __syncthreads();
    const int64_t item = (int64_t)s_item;
    if (item >= a.items) break;
    int lo = 0, hi = a.n;  // reqs[lo].item0 <= item < reqs[hi].item0
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.reqs[mid].item0 <= item) lo = mid;
      else hi = mid;
    }
    const EvictReq rq = a.reqs[lo];
    const int unit = (int)((item - rq.item0) / rq.items), k = (int)((item - rq.item0) % rq.items);
    const int layer = unit / a.Hkv, h = unit % a.Hkv;
    const int rows = min(R, rq.keep - k * R);
    const int32_t* ob = a.old_bt + rq.bt_off;
    const int32_t* nb = a.new_bt + rq.bt_off;
    const int dpage = nb[k * R / PAGE];  // an item's targets share a page
    const bool same_page = ob[k * R / PAGE] == dpage;
    if (tid < rows) {
      const int s = a.idx[rq.idx_off + (size_t)unit * rq.keep + k * R + tid];
      s_src[tid] = s == k * R + tid && same_page ? -1 : s;
    }
    __syncthreads();
    const size_t lbase = (size_t)layer * a.num_pages_total;
    float* wrow = a.weights + (((size_t)layer * a.M + rq.slot) * a.Hkv + h) * a.cap;
    // ---- read ----
    uint4 kv[PER], vv[PER];
    float wv = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int p = tid + i * MNT, row = p / PIECES, q = p % PIECES;
      const int s = row < rows ? s_src[row] : -1;
      if (s >= 0) {
        const size_t off = ((lbase + ob[s / PAGE]) * a.Hkv + h) * (size_t)(PAGE * RB) + (size_t)(s % PAGE) * RB + q * 16;
        kv[i] = *reinterpret_cast<const uint4*>(kc + off);
        vv[i] = *reinterpret_cast<const uint4*>(vc + off);
      }
    }
    const bool wmove = tid < rows && s_src[tid] >= 0;
    if (wmove) wv = wrow[s_src[tid]];
    // the block's reads come before the flag: barrier, then a release at GPU scope
    __syncthreads();
    const int32_t* pre = a.pre + rq.pre_off + (size_t)unit * (rq.items + 1);
    unsigned* flags = a.flags + rq.item0 + (size_t)unit * rq.items;
    if (tid == 0) {
      __threadfence();
      st_release(flags + k, 1u);
    }
    // ---- the rows that live in the target slots have been read ----
    if (tid < 2) {
      const int p0 = pre[k], p1 = pre[k + 1];
      const int j = p0 / R + tid;  // items p0 / R .. (p1 - 1) / R, two at most, none above k
      if (p1 > p0 && j <= (p1 - 1) / R && j < k) {
        const long long t0 = clock64();
        bool ok = a.wait_limit > 0 && ld_acquire(flags + j) != 0u;
        while (!ok) {
          if (clock64() - t0 >= a.wait_limit) break;
          ok = ld_acquire(flags + j) != 0u;
        }
        if (!ok) atomicOr(&s_fail, 1);
      }
    }
    __syncthreads();
    if (s_fail) break;  // read after the barrier: all threads leave together
    // ---- write ----
    const size_t dbase = ((lbase + dpage) * a.Hkv + h) * (size_t)(PAGE * RB) + (size_t)(k * R % PAGE) * RB;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int p = tid + i * MNT, row = p / PIECES;
      if (row < rows && s_src[row] >= 0) {
        *reinterpret_cast<uint4*>(kc + dbase + (size_t)p * 16) = kv[i];
        *reinterpret_cast<uint4*>(vc + dbase + (size_t)p * 16) = vv[i];
      }
    }
    if (wmove) {
      wrow[k * R + tid] = wv;
      ++moved;
    }
    __syncthreads();  // s_src and s_item are rewritten
  }
  if (tid == 0 && s_fail) atomicOr(a.err, ERR_TIMEOUT);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) moved += __shfl_xor_sync(0xffffffffu, moved, o);
  if ((tid & 31) == 0 && moved) atomicAdd(a.moved, (unsigned long long)moved);
}

template <int RB>
cudaError_t launch_rb(const EvictArgs& a, cudaStream_t s) {
  int per_sm = 0;
  const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k_evict_move<RB>, MNT, 0);
  if (e != cudaSuccess) return e;
  const int64_t grid = a.items < (int64_t)per_sm * a.sms ? a.items : (int64_t)per_sm * a.sms;
  k_evict_move<RB><<<dim3((unsigned)grid), MNT, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_evict_select(const EvictArgs& a, cudaStream_t s) {
  if (a.n == 0) return cudaSuccess;
  const int64_t grid = (int64_t)a.n * a.L * a.Hkv;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  k_evict_select<<<dim3((unsigned)grid), SNT, 0, s>>>(a);
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
