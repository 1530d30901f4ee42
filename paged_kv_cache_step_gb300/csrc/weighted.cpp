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

bool misaligned(const void* p, unsigned to = 16) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Whether two buffers of `bytes` share any.
bool overlap(const void* p, const void* q, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + bytes && b < a + bytes;
}

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

// ---- work of the tensor-core chunk kernels --------------------------------------

// Work laid end to end and cut into one even share a CTA, of at least `least`.
// A job is `n` tiles that cost `cost` each, `times` of them alike one after the
// other; every piece of a job costs `fixed` more.  A piece is tiles [from, to)
// of one job, or `times` whole ones.  begin: the first piece of every CTA, and
// the number of pieces.
struct Job {
  int n, cost, times;
};
struct Piece {
  int job, at, times;  // `times` jobs from the `at`-th of the run
  int from, to;        // tiles (all of them when times > 1)
};
int lay_out(const std::vector<Job>& jobs, int64_t share, int fixed, std::vector<Piece>* pieces,
            std::vector<int32_t>* begin) {
  int ctas = 1, count = 0;
  int64_t room = share;
  auto put = [&](const Piece& p) {
    ++count;
    if (pieces) pieces->push_back(p);
  };
  auto next_cta = [&] {
    ++ctas;
    if (begin) begin->push_back(count);
    room = share;
  };
  for (int k = 0; k < (int)jobs.size(); ++k) {
    const Job& j = jobs[k];
    const int64_t whole = fixed + (int64_t)j.n * j.cost;
    for (int at = 0; at < j.times;) {
      if (whole <= room) {
        const int take = (int)std::min<int64_t>(j.times - at, room / whole);
        put({k, at, take, 0, j.n});
        at += take;
        room -= take * whole;
        continue;
      }
      for (int from = 0; from < j.n;) {
        if (room < share && room < fixed + (int64_t)j.cost * std::min(j.n - from, 2)) next_cta();
        int take = (int)std::min<int64_t>(j.n - from, std::max<int64_t>(1, (room - fixed) / j.cost));
        if (j.n - from - take == 1) ++take;  // no sliver of one tile
        put({k, at, 1, from, from + take});
        from += take;
        room -= fixed + (int64_t)j.cost * take;
      }
      ++at;
    }
  }
  if (begin) begin->push_back(count);
  return ctas;
}
void cut_even(const std::vector<Job>& jobs, int ctas, int fixed, int least, std::vector<Piece>& pieces,
              std::vector<int32_t>& begin) {
  int64_t total = 0;
  int most = 1;
  for (const Job& j : jobs) {
    total += (fixed + (int64_t)j.n * j.cost) * j.times;
    most = std::max(most, j.cost);
  }
  // cut pieces add their fixed cost, and a share ends early or late by a few
  // tiles, so an exact share may need more CTAs: it grows in steps up to one
  // that cannot
  const int64_t slack = 2 * fixed + 4 * most;
  int64_t share = std::max<int64_t>(least, (total + ctas - 1) / ctas);
  for (int64_t step = std::max<int64_t>(1, slack / 4); lay_out(jobs, share, fixed, nullptr, nullptr) > ctas;)
    share += step;
  pieces.clear();
  begin.assign(1, 0);
  lay_out(jobs, share, fixed, &pieces, &begin);
}

struct ChunkPlan {
  std::vector<ChunkItem> items, kitems;
  std::vector<ChunkJoin> joins;
  std::vector<int32_t> begin, kbegin;
  int parts = 0;
  std::vector<WeightItem> witems;
  std::vector<WeightJoin> wjoins;
  std::vector<int32_t> wbegin;
  int wparts = 0;
};

// Attention: pairs of query tiles that follow each other (a key tile costs two
// products' time), and the last tiles alone, their key tiles split between the
// groups (one).  A piece's fixed cost is the time to load Q and to empty the
// pipeline, about three tiles: of 1, 2, 3, 4 and 6, three keeps each of ten calls
// (drafted tokens, many short chunks, prompts of 300 to 6007 tokens) within 6 % of
// its best; the others cost one of them 8 to 10 %.  The last tiles need a launch of their own, about
// 8 us; beside pairs, up to 12 key tiles of them a CTA (about 0.6 us each) go
// along as pairs without a second tile instead, at twice the cost (in one launch and
// in two: five ragged prompts, d = 64, 51 and 55 us; eight of about 500 tokens 57 and
// 66; one of 2000 62 and 71; 64 chunks of 40 to 100 tokens, more than 12 tiles a
// CTA, 115 and 137).
void plan_chunk(int n, const int32_t* cached, const int32_t* fresh, int Hkv, int G, int ctas, bool weights,
                ChunkPlan* p) {
  const int tok = 128 / G;
  std::vector<Job> jobs;
  std::vector<ChunkItem> of;
  std::vector<Piece> pieces;
  int64_t odd = 0;  // key tiles of the last tiles alone
  bool pairs = false;
  for (int r = 0; r < n; ++r) {
    pairs |= fresh[r] > tok;
    if ((fresh[r] + tok - 1) / tok % 2) odd += (int64_t)Hkv * ((cached[r] + fresh[r] + 127) / 128);
  }
  const bool along = pairs && odd <= 12ll * ctas;
  for (int r = 0; r < n; ++r)
    for (int h = 0; h < Hkv; ++h)
      for (int t = 0; t < fresh[r]; t += 2 * tok) {
        const bool alone = t + tok >= fresh[r];
        if (alone && !along) continue;
        jobs.push_back({(cached[r] + std::min(t + 2 * tok, fresh[r]) + 127) / 128, 2, 1});
        of.push_back({r, h, t, alone, 0, 0, -1, -1});
      }
  if (!jobs.empty()) cut_even(jobs, ctas, 3, 6, pieces, p->begin);
  for (size_t k = 0, e; k < pieces.size(); k = e) {
    for (e = k; e < pieces.size() && pieces[e].job == pieces[k].job;) ++e;
    const ChunkItem& job = of[pieces[k].job];
    const int count = (int)(e - k), first = p->parts;
    for (size_t i = k; i < e; ++i) {
      ChunkItem it = job;
      it.kb = pieces[i].from;
      it.ke = pieces[i].to;
      if (count > 1) {
        it.part_a = first + (int)(i - k);
        if (!job.alone) it.part_b = first + count + (int)(i - k);
      }
      p->items.push_back(it);
    }
    if (count > 1) {
      p->joins.push_back({job.r, job.h, job.t0, first, count, {}});
      if (!job.alone) p->joins.push_back({job.r, job.h, job.t0 + tok, first + count, count, {}});
      p->parts += job.alone ? count : 2 * count;
    }
  }
  // last tiles alone
  jobs.clear();
  of.clear();
  pieces.clear();
  for (int r = 0; r < n; ++r) {
    const int tiles = (fresh[r] + tok - 1) / tok;
    if (tiles % 2 == 0 || along) continue;
    for (int h = 0; h < Hkv; ++h) {
      jobs.push_back({(cached[r] + fresh[r] + 127) / 128, 1, 1});
      of.push_back({r, h, (tiles - 1) * tok, 0, 0, 0, -1, -1});
    }
  }
  if (!jobs.empty()) cut_even(jobs, ctas, 3, 6, pieces, p->kbegin);
  for (size_t k = 0, e; k < pieces.size(); k = e) {
    int parts = 0;
    for (e = k; e < pieces.size() && pieces[e].job == pieces[k].job; ++e) parts += pieces[e].to - pieces[e].from > 1 ? 2 : 1;
    const ChunkItem& job = of[pieces[k].job];
    int part = p->parts;
    for (size_t i = k; i < e; ++i) {
      ChunkItem it = job;
      it.kb = pieces[i].from;
      it.ke = pieces[i].to;
      if (parts > 1) {
        it.part_a = part++;
        if (it.ke - it.kb > 1) it.part_b = part++;
      }
      p->kitems.push_back(it);
    }
    if (parts > 1) {
      p->joins.push_back({job.r, job.h, job.t0, p->parts, parts, {}});
      p->parts += parts;
    }
  }
  if (!weights) return;
  // Weights: a page against the query tiles that see it; loading the page
  // costs about three query tiles' products (278, 273, 268, 266 and 269 us at 1, 2, 3,
  // 4 and 6 for the 6007 tokens, 28.0, 27.1, 27.4, 27.5 and 29.9 for ragged prompts;
  // of the ten calls three keeps each within 8 % of its best).  The pages that every token sees are alike.
  jobs.clear();
  std::vector<WeightItem> wof;
  for (int r = 0; r < n; ++r) {
    const int tiles = (fresh[r] + tok - 1) / tok, pages = (cached[r] + fresh[r] + kPage - 1) / kPage;
    if (fresh[r] == 0) continue;
    const int seen = std::min(pages, (cached[r] + tok - 1) / kPage + 1);  // pages that the first query tile sees some of
    for (int h = 0; h < Hkv; ++h) {
      jobs.push_back({tiles, 1, seen});
      wof.push_back({r, h, 0, 0, 0, tiles, -1, 0});
      for (int pg = seen; pg < pages; ++pg) {
        const int q0 = (pg * kPage - cached[r]) / tok;
        jobs.push_back({tiles - q0, 1, 1});
        wof.push_back({r, h, pg, 0, q0, tiles, -1, 0});
      }
    }
  }
  pieces.clear();
  cut_even(jobs, ctas, 3, 6, pieces, p->wbegin);
  for (size_t k = 0; k < pieces.size(); ++k) {
    const Piece& pc = pieces[k];
    WeightItem it = wof[pc.job];
    it.page += pc.at;
    it.pages = pc.times;
    if (pc.to - pc.from < jobs[pc.job].n) {  // a part of a page's query tiles
      if (pc.from == 0) p->wjoins.push_back({it.r, it.h, it.page, p->wparts, 0, {}});
      ++p->wjoins.back().n;
      it.part = p->wparts++;
    }
    it.qe = it.qb + pc.to;
    it.qb += pc.from;
    p->witems.push_back(it);
  }
}

// ---- work of the CUDA-core chunk kernels ------------------------------------------

struct TilePlan {
  std::vector<ChunkTile> tiles, wtiles;
  std::vector<ChunkTileJoin> joins, wjoins;
  int parts = 0, wparts = 0;
};

// Query tiles (weights: key tiles), those with most work first, each cut into
// equal items of at most `most` key tiles (query tiles).  Two CTAs fit on an SM;
// `most` is between a half and a whole of what a place of these has to do, where
// the rounds over all places cost least, an item counting 1.5 tiles more for its
// start and end.  Two requests of about 500 tokens, two KV heads, d = 64, fp32:
// attention 110 us and weights 66 us uncut, 42 and 23 us cut.
void plan_tiles(int n, const int32_t* cached, const int32_t* fresh, int Hkv, int G, int sms, bool weights, TilePlan* p) {
  const int tok = CHUNK_ROWS / G;
  std::vector<ChunkTile> whole;
  auto cut = [&](std::vector<ChunkTile>& tiles, std::vector<ChunkTileJoin>& joins, int& parts) {
    int64_t total = 0;
    for (const ChunkTile& t : whole) total += t.to - t.from;
    const int64_t places = 2 * (int64_t)sms;
    int most = 0;
    double least = 0.;
    const int64_t half = std::max<int64_t>(1, (total + 2 * places - 1) / (2 * places));
    const int64_t full = std::max<int64_t>(1, (total + places - 1) / places);
    for (int64_t m = half; m <= full; m += std::max<int64_t>(1, (full - half) / 12)) {  // some thirteen tries
      int64_t items = 0;
      for (const ChunkTile& t : whole) items += (t.to - t.from + m - 1) / m;
      const double cost = (double)((items + places - 1) / places) * (m + 1.5);
      if (most == 0 || cost < least) {
        most = (int)m;
        least = cost;
      }
    }
    for (ChunkTile t : whole) {
      const int from = t.from, len = t.to - t.from, count = (len + most - 1) / most;
      if (count > 1) joins.push_back({t.r, t.h, t.first, parts, count, {}});
      for (int i = 0; i < count; ++i) {
        t.from = from + (int)((int64_t)len * i / count);
        t.to = from + (int)((int64_t)len * (i + 1) / count);
        t.part = count > 1 ? parts++ : -1;
        tiles.push_back(t);
      }
    }
  };
  for (int r = 0; r < n; ++r)
    for (int t = (fresh[r] - 1) / tok * tok; fresh[r] > 0 && t >= 0; t -= tok)
      for (int h = 0; h < Hkv; ++h)
        whole.push_back({r, h, t, 0, (cached[r] + std::min(t + tok, fresh[r]) + CHUNK_KEYS - 1) / CHUNK_KEYS, -1, {}});
  cut(p->tiles, p->joins, p->parts);
  if (!weights) return;
  whole.clear();
  for (int r = 0; r < n; ++r)
    for (int s = 0; fresh[r] > 0 && s < cached[r] + fresh[r]; s += CHUNK_KEYS)
      for (int h = 0; h < Hkv; ++h)
        whole.push_back({r, h, s, std::max(0, s - cached[r]) / tok, (fresh[r] + tok - 1) / tok, -1, {}});
  cut(p->wtiles, p->wjoins, p->wparts);
}

}  // namespace

gp_status gp_append_tokens(gp_ctx* c, int32_t layer, int32_t n, const gp_request* reqs, const int32_t* num_cached,
                           const int32_t* num_new, const void* q_dev, const void* k_dev, const void* v_dev,
                           void* q_rot_dev, float* weights_dev) try {
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
  if (misaligned(weights_dev, 4)) return fail(c, GP_ERR_INVALID, "the weights must be 4-byte aligned");
  if (q_dev && q_rot_dev != q_dev &&
      overlap(q_dev, q_rot_dev, (size_t)rows * g.num_q_heads * g.head_dim * elt_bytes(g.q_dtype)))
    return fail(c, GP_ERR_INVALID, "q_rot overlaps q without being it");
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
  if ((st = wait_pending(c, n, reqs)) != GP_OK) return st;
  AppendArgs a{};
  AppendReq* hr = a.few;
  int32_t* hb = a.few_bt;
  const bool few = live <= AppendArgs::FEW_REQS && pages <= AppendArgs::FEW_PAGES;
  Layout lay;
  StagingSlot* slot = nullptr;
  if (!few) {
    const size_t at_req = lay.take(sizeof(AppendReq) * (size_t)live), at_bt = lay.take(sizeof(int32_t) * (size_t)pages);
    if ((st = staging_take(c, lay.bytes, &slot)) != GP_OK) return st;
    char *host = static_cast<char*>(slot->pinned), *dev = static_cast<char*>(slot->dev.p);
    hr = reinterpret_cast<AppendReq*>(host + at_req);
    hb = reinterpret_cast<int32_t*>(host + at_bt);
    a.reqs = reinterpret_cast<const AppendReq*>(dev + at_req);
    a.bt = reinterpret_cast<const int32_t*>(dev + at_bt);
  }
  int64_t row = 0;
  int at = 0, k = 0;
  for (int r = 0; r < n; ++r) {
    if (num_new[r] == 0) continue;
    hr[k++] = {reqs[r].pos, row, num_cached[r], num_new[r], reqs[r].slot, at};
    row += num_new[r];
    for (int j = num_cached[r] / kPage; j <= (num_cached[r] + num_new[r] - 1) / kPage; ++j)
      hb[at++] = reqs[r].block_table[j];
  }
  if (!few && (st = staging_upload(c, *slot, lay.bytes)) != GP_OK) return st;
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
} catch (const std::exception&) {
  return no_memory(c);
}

gp_status gp_chunk_attention(gp_ctx* c, int32_t layer, int32_t n, const gp_request* reqs, const int32_t* num_cached,
                             const int32_t* num_new, const void* q_dev, void* out_dev, float* weights_dev) try {
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
  if (misaligned(weights_dev, 4)) return fail(c, GP_ERR_INVALID, "the weights must be 4-byte aligned");
  if (overlap(q_dev, out_dev, (size_t)rows * g.num_q_heads * g.head_dim * elt_bytes(g.q_dtype)))
    return fail(c, GP_ERR_INVALID, "the outputs overlap the queries");
  if ((st = ready_call(c)) != GP_OK) return st;
  // The tensor-core kernels take bf16 caches and queries (AUTO and
  // TENSOR_CORE), the CUDA-core ones everything.
  const bool tc = c->attn_tc_ok && c->scan_kernel != GP_SCAN_CUDA_CORE && g.q_dtype == GP_DTYPE_BF16 &&
                  chunk_tc_shape(g.head_dim, G) && rows < (1ll << 31) - 256;
  if (c->scan_kernel == GP_SCAN_TENSOR_CORE && !tc)
    return fail(c, GP_ERR_UNSUPPORTED, "the tensor-core chunk kernels cannot take this cache, shape or query type");
  if ((st = wait_pending(c, n, reqs)) != GP_OK) return st;
  const int maxp = g.max_pages_per_req;
  ChunkPlan plan;
  TilePlan tiles;
  if (tc) plan_chunk(n, num_cached, num_new, Hkv, G, c->sms, weights_dev != nullptr, &plan);
  else plan_tiles(n, num_cached, num_new, Hkv, G, c->sms, weights_dev != nullptr, &tiles);
  Layout lay, scratch;
  const size_t at_req = lay.take(sizeof(ChunkReq) * (size_t)n), at_bt = lay.take(sizeof(int32_t) * (size_t)n * maxp);
  std::vector<std::pair<size_t, std::pair<const void*, size_t>>> tables;
  auto table = [&](const auto& v) {
    const size_t bytes = sizeof(v[0]) * v.size(), at = lay.take(bytes);
    tables.push_back({at, {v.data(), bytes}});
    return at;
  };
  const size_t at_tiles = table(tiles.tiles), at_wtiles = table(tiles.wtiles);
  const size_t at_tjoins = table(tiles.joins), at_twjoins = table(tiles.wjoins);
  const size_t at_items = table(plan.items), at_begin = table(plan.begin), at_joins = table(plan.joins);
  const size_t at_kitems = table(plan.kitems), at_kbegin = table(plan.kbegin);
  const size_t at_witems = table(plan.witems), at_wbegin = table(plan.wbegin), at_wjoins = table(plan.wjoins);
  const size_t at_part = scratch.take(sizeof(float) * chunk_part_floats(g.head_dim) * (size_t)plan.parts);
  const size_t at_wpart = scratch.take(sizeof(float) * kPage * (size_t)plan.wparts);
  const size_t at_tpart = scratch.take(sizeof(float) * chunk_tile_part_floats(g.head_dim) * (size_t)tiles.parts);
  const size_t at_twpart = scratch.take(sizeof(float) * CHUNK_KEYS * (size_t)tiles.wparts);
  if (weights_dev && (st = ensure(c, c->wstat, sizeof(float2) * (size_t)rows * g.num_q_heads)) != GP_OK) return st;
  if ((st = ensure(c, c->chunk, scratch.bytes)) != GP_OK) return st;
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
  for (const auto& t : tables)
    if (t.second.second) std::memcpy(host + t.first, t.second.first, t.second.second);
  if ((st = staging_upload(c, *slot, lay.bytes)) != GP_OK) return st;
  const char* dev = static_cast<char*>(slot->dev.p);
  const ChunkReq* dreqs = reinterpret_cast<const ChunkReq*>(dev + at_req);
  const int32_t* dbt = reinterpret_cast<const int32_t*>(dev + at_bt);
  float2* stat = weights_dev ? static_cast<float2*>(c->wstat.p) : nullptr;
  if (tc) {
    ChunkTcArgs a{};
    a.kmap = c->kmap;
    a.vmap = c->vmap;
    const cuuint64_t dims[3] = {(cuuint64_t)g.head_dim, (cuuint64_t)g.num_q_heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)g.head_dim * 2, (cuuint64_t)g.head_dim * 2 * g.num_q_heads};
    const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(128 / G)};
    if (!encode_bf16_map(&a.qmap, 3, q_dev, dims, strides, box))
      return fail(c, GP_ERR_CUDA, "no tensor map for the queries");
    a.num_pages_total = g.num_pages;
    a.layer = layer;
    a.Hq = g.num_q_heads;
    a.Hkv = Hkv;
    a.D = g.head_dim;
    a.G = G;
    a.M = g.max_slots;
    a.cap = (int64_t)maxp * kPage;
    a.reqs = dreqs;
    a.bt = dbt;
    a.items = reinterpret_cast<const ChunkItem*>(dev + at_items);
    a.begin = reinterpret_cast<const int32_t*>(dev + at_begin);
    a.grid = std::max(0, (int)plan.begin.size() - 1);
    a.kitems = reinterpret_cast<const ChunkItem*>(dev + at_kitems);
    a.kbegin = reinterpret_cast<const int32_t*>(dev + at_kbegin);
    a.kgrid = std::max(0, (int)plan.kbegin.size() - 1);
    a.joins = reinterpret_cast<const ChunkJoin*>(dev + at_joins);
    a.n_joins = (int)plan.joins.size();
    a.witems = reinterpret_cast<const WeightItem*>(dev + at_witems);
    a.wbegin = reinterpret_cast<const int32_t*>(dev + at_wbegin);
    a.wgrid = (int)plan.wbegin.size() - 1;
    a.wjoins = reinterpret_cast<const WeightJoin*>(dev + at_wjoins);
    a.n_wjoins = (int)plan.wjoins.size();
    a.out = out_dev;
    a.lse = reinterpret_cast<float*>(stat);
    a.weights = weights_dev;
    a.part = reinterpret_cast<float*>(static_cast<char*>(c->chunk.p) + at_part);
    a.wpart = reinterpret_cast<float*>(static_cast<char*>(c->chunk.p) + at_wpart);
    a.err = c->err_dev;
    a.wait_limit = c->wait_limit_chunk;
    st = timed_launch(c, GP_KERNEL_CHUNK, "chunk_attention", [&] { return launch_chunk_tc(a, c->stream); });
    if (st != GP_OK || !weights_dev) return st;
    a.wait_limit = c->wait_limit_weights;
    return timed_launch(c, GP_KERNEL_WEIGHTS, "chunk_weights", [&] { return launch_chunk_weights_tc(a, c->stream); });
  }
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
  a.reqs = dreqs;
  a.n = n;
  a.bt = dbt;
  a.tiles = reinterpret_cast<const ChunkTile*>(dev + at_tiles);
  a.n_tiles = (int)tiles.tiles.size();
  a.joins = reinterpret_cast<const ChunkTileJoin*>(dev + at_tjoins);
  a.n_joins = (int)tiles.joins.size();
  a.wtiles = reinterpret_cast<const ChunkTile*>(dev + at_wtiles);
  a.n_wtiles = (int)tiles.wtiles.size();
  a.wjoins = reinterpret_cast<const ChunkTileJoin*>(dev + at_twjoins);
  a.n_wjoins = (int)tiles.wjoins.size();
  a.part = reinterpret_cast<float*>(static_cast<char*>(c->chunk.p) + at_tpart);
  a.wpart = reinterpret_cast<float*>(static_cast<char*>(c->chunk.p) + at_twpart);
  a.q = q_dev;
  a.out = out_dev;
  a.stat = stat;
  a.weights = weights_dev;
  a.err = c->err_dev;
  st = timed_launch(c, GP_KERNEL_CHUNK, "chunk_attention", [&] { return launch_chunk(a, c->stream); });
  if (st != GP_OK || !weights_dev) return st;
  return timed_launch(c, GP_KERNEL_WEIGHTS, "chunk_weights", [&] { return launch_chunk_weights(a, c->stream); });
} catch (const std::exception&) {
  return no_memory(c);
}

gp_status gp_evict_weighted(gp_ctx* c, int32_t n, gp_request* reqs, const int32_t* num_tokens,
                            const int32_t* keep_tokens, float* weights_dev) try {
  if (!c) return GP_ERR_INVALID;
  gp_status st;
  const gp_config& g = c->cfg;
  if (n < 0 || n > g.max_slots) return fail(c, GP_ERR_INVALID, "n = %d outside [0, max_slots]", n);
  if (n == 0) return ready_call(c);
  if (!reqs || !num_tokens || !keep_tokens || !weights_dev) return fail(c, GP_ERR_INVALID, "null argument");
  if (misaligned(c->k_cache) || misaligned(c->v_cache) || misaligned(weights_dev, 4))
    return fail(c, GP_ERR_INVALID, "the caches must be 16-byte aligned, the weights 4-byte");
  const int units = units_of(c), maxp = g.max_pages_per_req;
  const int row_bytes = g.head_dim * elt_bytes(g.kv_dtype), R = evict_rows(row_bytes);
  std::vector<uint8_t> bound(g.max_slots, 0);
  size_t cow = 0;
  int longest = 0;
  int64_t idx_count = 0, items = 0, pre_count = 0;
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
    e.idx_off = idx_count;
    e.item0 = items;
    e.pre_off = pre_count;
    if (T <= keep) continue;  // nothing to evict: its tables and rows stay as they are, and no list is made
    e.idx_pitch = (keep + 7) / 8 * 8;
    e.items = (keep + R - 1) / R;
    idx_count += (int64_t)units * e.idx_pitch;
    items += (int64_t)units * e.items;
    pre_count += (int64_t)units * (e.items + 1);
    longest = std::max(longest, T);
    for (int j = 0; j < reqs[r].num_pages; ++j) cow += c->refcnt[reqs[r].block_table[j]] > 1;
  }
  // a page has a reference for every request that evicts from it: one with a single
  // reference is compacted in place, a shared one loses a reference to each copy
  begin_page_check(c);
  std::vector<int32_t> shared;
  for (int r = 0; r < n; ++r)
    for (int j = 0; er[r].items && j < reqs[r].num_pages; ++j) {
      const int32_t pg = reqs[r].block_table[j];
      if (c->refcnt[pg] > 1) shared.push_back(pg);
      else if (std::exchange(c->page_seen[pg], c->check) == c->check)
        return fail(c, GP_ERR_INVALID, "page %d is in two requests and has one reference", pg);
    }
  std::sort(shared.begin(), shared.end());
  for (size_t i = 0, e; i < shared.size(); i = e) {
    for (e = i; e < shared.size() && shared[e] == shared[i];) ++e;
    if ((int64_t)(e - i) > c->refcnt[shared[i]])
      return fail(c, GP_ERR_INVALID, "page %d is in %zu requests and has %d references", shared[i], e - i, c->refcnt[shared[i]]);
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
  c->last_compress.clear();  // its lists may be in the scratch
  if ((st = ensure(c, c->evict, scratch.bytes)) != GP_OK) return st;
  StagingSlot* slot = nullptr;
  if ((st = staging_take(c, lay.bytes, &slot)) != GP_OK) return st;
  char* host = static_cast<char*>(slot->pinned);
  std::memcpy(host + at_req, er.data(), sizeof(EvictReq) * (size_t)n);
  int32_t* old_bt = reinterpret_cast<int32_t*>(host + at_old);
  int32_t* new_bt = reinterpret_cast<int32_t*>(host + at_new);
  // everything that the call leaves behind is allocated before it changes anything
  std::vector<CompressRec> records(n);
  for (int r = 0; r < n; ++r) {
    CompressRec& rec = records[r];
    rec.num_pages = reqs[r].num_pages;
    rec.evict = true;
    rec.tokens = er[r].T;
    rec.kept = er[r].items ? er[r].keep : 0;
    rec.pitch = er[r].idx_pitch;
    rec.mask_off = er[r].idx_off;  // c->evict starts with the kept slots
  }
  std::unordered_set<int32_t> pages, slots;  // of a compaction on the side stream
  if (c->cstream) {
    size_t most = cow;
    for (int r = 0; r < n; ++r) most += reqs[r].num_pages;
    pages.reserve(most);
    for (int r = 0; r < n; ++r) {
      slots.insert(reqs[r].slot);
      pages.insert(reqs[r].block_table, reqs[r].block_table + reqs[r].num_pages);
    }
    auto it = c->free_pages.begin();  // those that the copies take
    for (size_t i = 0; i < cow; ++i) pages.insert(*it++);
  }
  std::vector<std::set<int32_t>::node_type> taken;  // free pages, as nodes that the released ones go back by
  taken.reserve(cow);
  // copy-on-write targets as in Compress & Hold (cannot fail now): lowest id first, ascending logical order
  for (int r = 0; r < n; ++r)
    for (int j = 0; j < reqs[r].num_pages; ++j) {
      const int32_t pg = reqs[r].block_table[j];
      int32_t to = pg;
      if (er[r].items && c->refcnt[pg] > 1) {
        taken.push_back(c->free_pages.extract(c->free_pages.begin()));
        to = taken.back().value();
        c->refcnt[to] = 1;
      }
      old_bt[(size_t)r * maxp + j] = pg;
      new_bt[(size_t)r * maxp + j] = to;
    }
  auto roll_back = [&](gp_status why) {
    for (auto& node : taken) {
      c->refcnt[node.value()] = 0;
      c->free_pages.insert(std::move(node));
    }
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
  a.idx = reinterpret_cast<uint16_t*>(scr + at_idx);
  a.pre = reinterpret_cast<int32_t*>(scr + at_pre);
  a.flags = reinterpret_cast<unsigned*>(scr + at_flags);
  a.ticket = reinterpret_cast<unsigned long long*>(scr + at_ticket);
  a.items = items;
  a.longest = longest;
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
    c->pending_pages.swap(pages);
    c->pending_slots.swap(slots);
  }
  c->last_compress.swap(records);
  for (int r = 0; r < n; ++r) {
    for (int j = 0; j < reqs[r].num_pages; ++j) {
      const int32_t from = old_bt[(size_t)r * maxp + j], to = new_bt[(size_t)r * maxp + j];
      if (to == from) continue;
      reqs[r].block_table[j] = to;
      if (--c->refcnt[from] == 0) {  // no more of these than pages taken
        taken.back().value() = from;
        c->free_pages.insert(std::move(taken.back()));
        taken.pop_back();
      }
      ++c->stats.cow_pages;
    }
    if (er[r].items) ++c->slot_gen[reqs[r].slot];
  }
  return GP_OK;
} catch (const std::exception&) {
  return no_memory(c);
}
