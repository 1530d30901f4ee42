// Host side of the operators around accumulated attention weights: new tokens
// into the cache, causal attention of several new tokens a request, and the
// eviction by the weights.  (gp_decode_attention_weighted shares
// gp_decode_attention's host code in growpage.cpp.)  Validates, plans and
// uploads descriptors; every device step runs in the kernels.
#include "growpage.h"

#include <cuda_runtime.h>

#include <cstring>
#include <vector>

#include "engine.h"
#include "weighted_kernels.h"

using namespace gp;

namespace {

// A call's tables laid out one after the other, 16-byte aligned.
struct Layout {
  size_t bytes = 0;
  size_t take(size_t n) {
    const size_t at = bytes;
    bytes += (n + 15) & ~size_t(15);
    return at;
  }
};

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// The checks that the calls over new tokens share: every request bound and
// listed once, its cached and new tokens inside its pages.  *rows: packed rows.
gp_status check_new_tokens(gp_ctx* c, int32_t layer, int32_t n, const gp_request* reqs, const int32_t* num_cached,
                           const int32_t* num_new, int64_t* rows) {
  const gp_config& g = c->cfg;
  if (layer < 0 || layer >= g.num_layers) return fail(c, GP_ERR_INVALID, "layer %d", layer);
  if (n < 0 || n > g.max_slots) return fail(c, GP_ERR_INVALID, "n = %d outside [0, max_slots]", n);
  *rows = 0;
  if (n == 0) return GP_OK;
  if (!reqs || !num_cached || !num_new) return fail(c, GP_ERR_INVALID, "null argument");
  gp_status st;
  std::vector<uint8_t> bound(g.max_slots, 0);
  for (int r = 0; r < n; ++r) {
    if ((st = validate_request(c, reqs[r], r, true)) != GP_OK) return st;
    if (bound[reqs[r].slot]) return fail(c, GP_ERR_INVALID, "slot %d appears twice", reqs[r].slot);
    bound[reqs[r].slot] = 1;
    if (num_cached[r] < 0 || num_new[r] < 0 ||
        (int64_t)num_cached[r] + num_new[r] > (int64_t)reqs[r].num_pages * kPage)
      return fail(c, GP_ERR_INVALID, "request %d: %d cached and %d new tokens do not fit its %d pages", r,
                  num_cached[r], num_new[r], reqs[r].num_pages);
    *rows += num_new[r];
  }
  return GP_OK;
}

}  // namespace

gp_status gp_append_tokens(gp_ctx* c, int32_t layer, int32_t n, const gp_request* reqs, const int32_t* num_cached,
                           const int32_t* num_new, const void* q_dev, const void* k_dev, const void* v_dev,
                           void* q_rot_dev, float* weights_dev) {
  if (!c) return GP_ERR_INVALID;
  gp_status st;
  const gp_config& g = c->cfg;
  int64_t rows = 0;
  if ((st = check_new_tokens(c, layer, n, reqs, num_cached, num_new, &rows)) != GP_OK) return st;
  if (rows == 0) return ready_call(c);
  if (!k_dev || !v_dev || (q_dev == nullptr) != (q_rot_dev == nullptr))
    return fail(c, GP_ERR_INVALID, "null keys or values, or only one of q and q_rot");
  if (misaligned(q_dev) || misaligned(k_dev) || misaligned(v_dev) || misaligned(q_rot_dev) ||
      misaligned(c->k_cache) || misaligned(c->v_cache))
    return fail(c, GP_ERR_INVALID, "queries, keys, values and caches must be 16-byte aligned");
  // the pages written: private, and each in one request only
  int64_t pages = 0;
  int live = 0;
  begin_page_check(c);
  for (int r = 0; r < n; ++r) {
    if (num_new[r] == 0) continue;
    ++live;
    const int p0 = num_cached[r] / kPage, p1 = (num_cached[r] + num_new[r] - 1) / kPage;
    pages += p1 - p0 + 1;
    for (int j = p0; j <= p1; ++j) {
      const int32_t pg = reqs[r].block_table[j];
      if (c->refcnt[pg] != 1)
        return fail(c, GP_ERR_INVALID, "request %d: block %d is on page %d, which %d requests share", r, j, pg,
                    c->refcnt[pg]);
      if (std::exchange(c->page_seen[pg], c->check) == c->check)
        return fail(c, GP_ERR_INVALID, "page %d is written by two requests", pg);
    }
  }
  if ((st = ready_call(c)) != GP_OK) return st;
  if ((st = wait_shared_pages(c, n, reqs)) != GP_OK) return st;
  Layout lay;
  const size_t at_req = lay.take(sizeof(AppendReq) * (size_t)live), at_bt = lay.take(sizeof(int32_t) * (size_t)pages);
  StagingSlot* slot = nullptr;
  if ((st = staging_take(c, lay.bytes, &slot)) != GP_OK) return st;
  char* host = static_cast<char*>(slot->pinned);
  AppendReq* hr = reinterpret_cast<AppendReq*>(host + at_req);
  int32_t* hb = reinterpret_cast<int32_t*>(host + at_bt);
  int64_t row = 0;
  int at = 0, k = 0;
  for (int r = 0; r < n; ++r) {
    if (num_new[r] == 0) continue;
    hr[k++] = {reqs[r].pos, row, num_cached[r], num_new[r], reqs[r].slot, at};
    row += num_new[r];
    for (int j = num_cached[r] / kPage; j <= (num_cached[r] + num_new[r] - 1) / kPage; ++j)
      hb[at++] = reqs[r].block_table[j];
  }
  if ((st = staging_upload(c, *slot, lay.bytes)) != GP_OK) return st;
  AppendArgs a{};
  a.k_cache = c->k_cache;
  a.v_cache = c->v_cache;
  a.kv_f32 = g.kv_dtype == GP_DTYPE_F32;
  a.q_f32 = g.q_dtype == GP_DTYPE_F32;
  a.num_pages_total = g.num_pages;
  a.layer = layer;
  a.Hq = g.num_q_heads;
  a.Hkv = g.num_kv_heads;
  a.D = g.head_dim;
  a.M = g.max_slots;
  a.cap = (int64_t)g.max_pages_per_req * kPage;
  a.reqs = reinterpret_cast<const AppendReq*>(static_cast<char*>(slot->dev.p) + at_req);
  a.bt = reinterpret_cast<const int32_t*>(static_cast<char*>(slot->dev.p) + at_bt);
  a.n = live;
  a.rows = (int)rows;
  a.q = q_dev;
  a.k = k_dev;
  a.v = v_dev;
  a.q_rot = q_rot_dev;
  a.weights = weights_dev;
  a.inv_freq = c->inv_freq;
  a.err = c->err_dev;
  st = timed_launch(c, GP_KERNEL_APPEND, "append_tokens", [&] { return launch_append(a, c->stream); });
  if (st != GP_OK) return st;
  for (int r = 0; r < n; ++r)  // a demand result over the old rows is stale
    if (num_new[r] > 0) ++c->slot_gen[reqs[r].slot];
  return GP_OK;
}

gp_status gp_chunk_attention(gp_ctx* c, int32_t layer, int32_t n, const gp_request* reqs, const int32_t* num_cached,
                             const int32_t* num_new, const void* q_dev, void* out_dev, float* weights_dev) {
  if (!c) return GP_ERR_INVALID;
  gp_status st;
  const gp_config& g = c->cfg;
  const int G = g.num_q_heads / g.num_kv_heads, Hkv = g.num_kv_heads;
  int64_t rows = 0;
  if ((st = check_new_tokens(c, layer, n, reqs, num_cached, num_new, &rows)) != GP_OK) return st;
  if (rows == 0) return ready_call(c);
  if (!q_dev || !out_dev) return fail(c, GP_ERR_INVALID, "null argument");
  if (misaligned(q_dev) || misaligned(out_dev) || misaligned(c->k_cache) || misaligned(c->v_cache))
    return fail(c, GP_ERR_INVALID, "queries, outputs and caches must be 16-byte aligned");
  if ((st = ready_call(c)) != GP_OK) return st;
  if ((st = wait_shared_pages(c, n, reqs)) != GP_OK) return st;
  const int maxp = g.max_pages_per_req, tokens = CHUNK_ROWS / G;
  // query tiles, those that see most first; key tiles, the first (seen by most) first
  std::vector<ChunkTile> tiles, wtiles;
  for (int r = 0; r < n; ++r) {
    if (num_new[r] == 0) continue;
    for (int t = (num_new[r] - 1) / tokens * tokens; t >= 0; t -= tokens)
      for (int h = 0; h < Hkv; ++h) tiles.push_back({r, h, t, 0});
    if (weights_dev)
      for (int s = 0; s < num_cached[r] + num_new[r]; s += CHUNK_KEYS)
        for (int h = 0; h < Hkv; ++h) wtiles.push_back({r, h, s, 0});
  }
  Layout lay;
  const size_t at_req = lay.take(sizeof(ChunkReq) * (size_t)n), at_bt = lay.take(sizeof(int32_t) * (size_t)n * maxp);
  const size_t at_tiles = lay.take(sizeof(ChunkTile) * tiles.size());
  const size_t at_wtiles = lay.take(sizeof(ChunkTile) * wtiles.size());
  if (weights_dev && (st = ensure(c, c->wstat, sizeof(float2) * (size_t)rows * g.num_q_heads)) != GP_OK) return st;
  StagingSlot* slot = nullptr;
  if ((st = staging_take(c, lay.bytes, &slot)) != GP_OK) return st;
  char* host = static_cast<char*>(slot->pinned);
  int64_t row = 0;
  for (int r = 0; r < n; ++r) {
    reinterpret_cast<ChunkReq*>(host + at_req)[r] = {row, num_cached[r], num_new[r], reqs[r].slot, r * maxp};
    row += num_new[r];
    std::memcpy(host + at_bt + sizeof(int32_t) * (size_t)r * maxp, reqs[r].block_table,
                sizeof(int32_t) * reqs[r].num_pages);
  }
  std::memcpy(host + at_tiles, tiles.data(), sizeof(ChunkTile) * tiles.size());
  std::memcpy(host + at_wtiles, wtiles.data(), sizeof(ChunkTile) * wtiles.size());
  if ((st = staging_upload(c, *slot, lay.bytes)) != GP_OK) return st;
  const char* dev = static_cast<char*>(slot->dev.p);
  ChunkArgs a{};
  a.k_cache = c->k_cache;
  a.v_cache = c->v_cache;
  a.kv_f32 = g.kv_dtype == GP_DTYPE_F32;
  a.q_f32 = g.q_dtype == GP_DTYPE_F32;
  a.num_pages_total = g.num_pages;
  a.layer = layer;
  a.Hq = g.num_q_heads;
  a.Hkv = Hkv;
  a.D = g.head_dim;
  a.G = G;
  a.M = g.max_slots;
  a.cap = (int64_t)maxp * kPage;
  a.reqs = reinterpret_cast<const ChunkReq*>(dev + at_req);
  a.n = n;
  a.bt = reinterpret_cast<const int32_t*>(dev + at_bt);
  a.tiles = reinterpret_cast<const ChunkTile*>(dev + at_tiles);
  a.n_tiles = (int)tiles.size();
  a.wtiles = reinterpret_cast<const ChunkTile*>(dev + at_wtiles);
  a.n_wtiles = (int)wtiles.size();
  a.q = q_dev;
  a.out = out_dev;
  a.stat = weights_dev ? static_cast<float2*>(c->wstat.p) : nullptr;
  a.weights = weights_dev;
  a.err = c->err_dev;
  st = timed_launch(c, GP_KERNEL_CHUNK, "chunk_attention", [&] { return launch_chunk(a, c->stream); });
  if (st != GP_OK || !weights_dev) return st;
  return timed_launch(c, GP_KERNEL_WEIGHTS, "chunk_weights", [&] { return launch_chunk_weights(a, c->stream); });
}

gp_status gp_evict_weighted(gp_ctx* c, int32_t n, gp_request* reqs, const int32_t* num_tokens,
                            const int32_t* keep_tokens, float* weights_dev) {
  if (!c) return GP_ERR_INVALID;
  gp_status st;
  const gp_config& g = c->cfg;
  if (n < 0 || n > g.max_slots) return fail(c, GP_ERR_INVALID, "n = %d outside [0, max_slots]", n);
  if (n == 0) return ready_call(c);
  if (!reqs || !num_tokens || !keep_tokens || !weights_dev) return fail(c, GP_ERR_INVALID, "null argument");
  if (misaligned(c->k_cache) || misaligned(c->v_cache))
    return fail(c, GP_ERR_INVALID, "the caches must be 16-byte aligned");
  const int units = units_of(c), maxp = g.max_pages_per_req;
  const int row_bytes = g.head_dim * elt_bytes(g.kv_dtype), R = evict_rows(row_bytes);
  std::vector<uint8_t> bound(g.max_slots, 0);
  size_t cow = 0;
  int64_t mask_words = 0, idx_count = 0, items = 0, pre_count = 0;
  std::vector<EvictReq> er(n);
  for (int r = 0; r < n; ++r) {
    if ((st = validate_request(c, reqs[r], r, true)) != GP_OK) return st;
    if (bound[reqs[r].slot]) return fail(c, GP_ERR_INVALID, "slot %d appears twice", reqs[r].slot);
    bound[reqs[r].slot] = 1;
    const int T = num_tokens[r], keep = keep_tokens[r];
    if (T < 0 || T > reqs[r].num_pages * kPage)
      return fail(c, GP_ERR_INVALID, "request %d: num_tokens %d outside [0, %d]", r, T, reqs[r].num_pages * kPage);
    if (keep < 1) return fail(c, GP_ERR_INVALID, "request %d: keep_tokens %d, at least 1", r, keep);
    EvictReq& e = er[r];
    e = EvictReq{};
    e.slot = reqs[r].slot;
    e.T = T;
    e.keep = keep;
    e.recent = std::min(g.recent_window, keep);
    e.bt_off = r * maxp;
    e.words = reqs[r].num_pages * (kPage / 32);
    e.mask_off = mask_words;
    mask_words += (int64_t)units * e.words;
    e.idx_off = idx_count;
    e.item0 = items;
    e.pre_off = pre_count;
    if (T <= keep) continue;  // nothing to evict: its tables and rows stay as they are
    e.items = (keep + R - 1) / R;
    idx_count += (int64_t)units * keep;
    items += (int64_t)units * e.items;
    pre_count += (int64_t)units * (e.items + 1);
    for (int j = 0; j < reqs[r].num_pages; ++j) cow += c->refcnt[reqs[r].block_table[j]] > 1;
  }
  if ((st = ready_call(c)) != GP_OK) return st;
  if (cow > c->free_pages.size())
    return fail(c, GP_ERR_NO_PAGES, "copy-on-write needs %zu fresh pages, %zu free", cow, c->free_pages.size());
  // an earlier compaction may still run on the side stream, and its scratch is used again here
  if ((st = join_compaction(c)) != GP_OK) return st;
  if ((st = join_select(c)) != GP_OK) return st;
  Layout lay, scratch;
  const size_t at_req = lay.take(sizeof(EvictReq) * (size_t)n);
  const size_t at_old = lay.take(sizeof(int32_t) * (size_t)n * maxp), at_new = lay.take(sizeof(int32_t) * (size_t)n * maxp);
  const size_t at_idx = scratch.take(sizeof(uint16_t) * (size_t)idx_count);
  const size_t at_pre = scratch.take(sizeof(int32_t) * (size_t)pre_count);
  const size_t at_flags = scratch.take(sizeof(unsigned) * (size_t)items), at_ticket = scratch.take(sizeof(unsigned long long));
  if ((st = ensure(c, c->masks, sizeof(uint32_t) * (size_t)mask_words)) != GP_OK) return st;
  if ((st = ensure(c, c->evict, scratch.bytes)) != GP_OK) return st;
  StagingSlot* slot = nullptr;
  if ((st = staging_take(c, lay.bytes, &slot)) != GP_OK) return st;
  char* host = static_cast<char*>(slot->pinned);
  std::memcpy(host + at_req, er.data(), sizeof(EvictReq) * (size_t)n);
  int32_t* old_bt = reinterpret_cast<int32_t*>(host + at_old);
  int32_t* new_bt = reinterpret_cast<int32_t*>(host + at_new);
  // copy-on-write targets as in Compress & Hold (cannot fail now): lowest id first, ascending logical order
  for (int r = 0; r < n; ++r)
    for (int j = 0; j < reqs[r].num_pages; ++j) {
      const int32_t pg = reqs[r].block_table[j];
      int32_t to = pg;
      if (er[r].items && c->refcnt[pg] > 1) gp_page_alloc(c, &to);
      old_bt[(size_t)r * maxp + j] = pg;
      new_bt[(size_t)r * maxp + j] = to;
    }
  auto roll_back = [&](gp_status why) {
    for (int r = 0; r < n; ++r)
      for (int j = 0; j < reqs[r].num_pages; ++j)
        if (new_bt[(size_t)r * maxp + j] != old_bt[(size_t)r * maxp + j])
          gp_page_unref(c, new_bt[(size_t)r * maxp + j]);
    return why;
  };
  if ((st = staging_upload(c, *slot, lay.bytes)) != GP_OK) return roll_back(st);
  const char* dev = static_cast<char*>(slot->dev.p);
  char* scr = static_cast<char*>(c->evict.p);
  EvictArgs a{};
  a.k_cache = c->k_cache;
  a.v_cache = c->v_cache;
  a.num_pages_total = g.num_pages;
  a.L = g.num_layers;
  a.Hkv = g.num_kv_heads;
  a.M = g.max_slots;
  a.row_bytes = row_bytes;
  a.cap = (int64_t)maxp * kPage;
  a.reqs = reinterpret_cast<const EvictReq*>(dev + at_req);
  a.n = n;
  a.old_bt = reinterpret_cast<const int32_t*>(dev + at_old);
  a.new_bt = reinterpret_cast<const int32_t*>(dev + at_new);
  a.weights = weights_dev;
  a.masks = static_cast<uint32_t*>(c->masks.p);
  a.idx = reinterpret_cast<uint16_t*>(scr + at_idx);
  a.pre = reinterpret_cast<int32_t*>(scr + at_pre);
  a.flags = reinterpret_cast<unsigned*>(scr + at_flags);
  a.ticket = reinterpret_cast<unsigned long long*>(scr + at_ticket);
  a.items = items;
  a.sms = c->sms;
  a.moved = c->moved_dev;
  a.err = c->err_dev;
  a.wait_limit = c->wait_limit_evict;
  cudaStream_t ks = c->stream;
  auto on_stream = [&](cudaError_t e) {
    return e == cudaSuccess ? GP_OK : fail(c, GP_ERR_CUDA, "evict: %s", cudaGetErrorString(e));
  };
  if (c->cstream) {  // beside the decoding, after everything the engine stream holds (App. E.3)
    if ((st = on_stream(cudaEventRecord(c->ev_ready, c->stream))) != GP_OK) return roll_back(st);
    if ((st = on_stream(cudaStreamWaitEvent(c->cstream, c->ev_ready, 0))) != GP_OK) return roll_back(st);
    ks = c->cstream;
  }
  st = timed_launch_on(c, ks, GP_KERNEL_EVICT_SELECT, "evict_select", [&] { return launch_evict_select(a, ks); });
  if (st == GP_OK)
    st = timed_launch_on(c, ks, GP_KERNEL_EVICT, "evict_move", [&] { return launch_evict_move(a, ks); });
  if (c->cstream) cudaEventRecord(slot->free, ks);  // the side stream reads the staged tables
  if (st != GP_OK) return roll_back(st);  // no row has moved: the selection writes scratch alone
  if (c->cstream) {
    GP_CUDA(c, cudaEventRecord(c->ev_done, ks));
    c->compaction_pending = true;
    c->pending_pages.clear();
    for (int r = 0; r < n; ++r)
      for (int j = 0; j < reqs[r].num_pages; ++j) {
        c->pending_pages.insert(old_bt[(size_t)r * maxp + j]);
        c->pending_pages.insert(new_bt[(size_t)r * maxp + j]);
      }
  }
  c->last_compress.assign(n, CompressRec{});
  for (int r = 0; r < n; ++r) {
    for (int j = 0; j < reqs[r].num_pages; ++j) {
      const int32_t from = old_bt[(size_t)r * maxp + j], to = new_bt[(size_t)r * maxp + j];
      if (to == from) continue;
      reqs[r].block_table[j] = to;
      gp_page_unref(c, from);
      ++c->stats.cow_pages;
    }
    if (er[r].items) ++c->slot_gen[reqs[r].slot];
    c->last_compress[r].num_pages = reqs[r].num_pages;
    c->last_compress[r].mask_off = er[r].mask_off;
  }
  return GP_OK;
}
