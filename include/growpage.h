/*
 * growpage.h -- C ABI of a GB300-native (sm_103a) capacity-boundary engine
 * for GrowPage ("GrowPage: On-Demand KV Budgeting for Efficient LLM
 * Reasoning Serving", arXiv 2609.03494) over a paged KV cache.
 *
 * What the engine computes (paper sections in brackets):
 *   - every decode step: the dual-timescale query summaries      [Sec. 3.2 Eq. 6, App. E.1]
 *   - at a capacity boundary: calibration + RoPE of both summaries,
 *     scores against every cached key through the block table,
 *     softmax, GQA mean and the p-coverage demand D_p per
 *     (layer, KV head), and the request-level trend Delta          [Sec. 3.2 Eqs. 7-8, App. E.1 Eq. 12]
 *   - the decision Grow by One Page vs Compress & Hold             [Sec. 3.2, Sec. 4.2]
 *   - Grow: append a fresh page to the block table                 [Sec. 3.3, Sec. 4.2]
 *   - Compress & Hold: importance max(a^S, a^L), protected recent
 *     window, block-local + global top-k, and copy-on-write
 *     compaction of the retained K/V into (P-1) b slots            [Sec. 3.3 Eqs. 9-10, App. E.2]
 *   - a refcounted page pool and a slot pool for the summaries    [Sec. 4.2, App. E.1 Eq. 11, App. E.2]
 *
 * Conventions
 *   - Every call returns gp_status; nothing throws across the ABI.  The
 *     text of the last failure is available from gp_last_error().
 *   - Device pointers ("_dev") are CUDA device addresses owned by the caller
 *     (for example PyTorch tensors); host pointers are plain memory owned by
 *     the caller.  The engine owns the summary pool, its scratch buffers, the
 *     page refcounts, the free-page list and the slot list.
 *   - All device work is issued on the stream given to gp_create, in call
 *     order.  gp_boundary_demand synchronises that stream before returning
 *     (the decision is a host decision, Sec. 4.2); the other hot-path calls
 *     are asynchronous.
 *   - Allocation failures (GP_ERR_NO_PAGES, GP_ERR_NO_SLOTS) leave every
 *     piece of state unchanged.
 *   - A context is not thread-safe; use one per host thread.
 *
 * Layouts
 *   K and V caches: [L][num_pages][Hkv][page_size][head_dim] of kv_dtype,
 *     so one (layer, page, KV head) tile is page_size * head_dim contiguous
 *     elements (64 KiB for bf16, d = 128, page_size = 256).
 *   Query summaries (engine-owned, fp64): [L][max_slots][2][Hq][head_dim],
 *     index 0 = short (beta_s), 1 = long (beta_l)  (App. E.1 Eq. 11).  fp64
 *     because the long summary's 1 - beta_l = 0.001 increments and the
 *     large logits of concentrated heads need more than fp32's 24 bits to
 *     keep importance scores within 1e-5 relative.
 *   Queries: [L][n][Hq][head_dim] of q_dtype, normalised and pre-RoPE.
 *   Query head j belongs to KV head j / (Hq / Hkv).
 *
 * EMA convention (fixed here because the paper's pages disagree): the stored
 * beta is the decay, the weight on the previous summary:
 *   qbar <- beta * qbar + (1 - beta) * q,  beta_s = 0.9 < beta_l = 0.999.
 */
#ifndef GROWPAGE_H
#define GROWPAGE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  GP_OK = 0,
  GP_ERR_INVALID = 1,     /* bad argument; nothing changed */
  GP_ERR_NO_PAGES = 2,    /* the free pool cannot supply the pages; nothing changed */
  GP_ERR_NO_SLOTS = 3,    /* no free summary slot; nothing changed */
  GP_ERR_CUDA = 4,        /* a CUDA runtime call failed, or host memory ran out (text in gp_last_error) */
  GP_ERR_TIMEOUT = 5,     /* a bounded device-side wait gave up (about one second of SM
                             clock); the kernel drained its copies and returned, so the
                             context stays usable, but that launch's outputs are
                             unspecified */
  GP_ERR_STATE = 6,       /* call out of order (e.g. compress without a fresh demand) */
  GP_ERR_UNSUPPORTED = 7  /* shape outside what the kernels were built for */
} gp_status;

typedef enum { GP_DTYPE_BF16 = 0, GP_DTYPE_F32 = 1 } gp_dtype;
/* Capacity-control policies (GrowPage Sec. 3.2; the alternatives of App. H.1):
 * GROWPAGE  Grow iff Delta > tau, else Compress & Hold;
 * FIXED     never Grow (GrowPage-Fixed);
 * RANDOM    Compress & Hold with probability random_compress, else Grow,
 *           whatever Delta (GrowPage-Random); the draw of the engine's k-th
 *           decision (k = 0, 1, ... since gp_create) is
 *           u_k = (splitmix64(random_seed * 2^32 + k) >> 11) * 2^-53;
 * INVERSE   Grow iff Delta <= tau, else Compress & Hold (GrowPage-Inverse);
 * SHRINK    Eq. 13: Shrink iff Delta < shrink_threshold, Grow iff Delta > tau,
 *           else Compress & Hold; Shrink only while the request holds more
 *           than shrink_floor_pages pages (App. H.1: 1024 tokens), else
 *           Compress & Hold. */
typedef enum {
  GP_POLICY_GROWPAGE = 0,
  GP_POLICY_FIXED = 1,
  GP_POLICY_RANDOM = 2,
  GP_POLICY_INVERSE = 3,
  GP_POLICY_SHRINK = 4
} gp_policy;
typedef enum { GP_ACT_GROW = 0, GP_ACT_COMPRESS = 1, GP_ACT_SHRINK = 2 } gp_action_kind;
/* Working-set metric of the demand estimation.
 *   TOP_P:   K^x = D_p(a^x) over C_t (Eq. 2, Eq. 7), the method's metric.
 *   ENTROPY: the ablation of Sec. 5.3 (Table 2) that puts attention entropy
 *            in its place.  The pages give no formula; the engine takes the
 *            entropy's effective support size E^x = exp(H(a^x)),
 *            H(a) = -sum_i a_i ln a_i over C_t (1 for a point mass, |C_t| for
 *            the uniform distribution), and uses it where K^x stands in
 *            Eq. 8.  D_p is still computed and reported. */
typedef enum { GP_METRIC_TOP_P = 0, GP_METRIC_ENTROPY = 1 } gp_metric;

/* Engine configuration.  Defaults (gp_config_default) follow the paper:
 * page_size 256, recent_window 16, k_loc 64, beta_s 0.9, beta_l 0.999,
 * p 0.99, tau 0, max_slots 512 (Sec. 3.2, Sec. 5.1, App. D, App. E.1). */
typedef struct gp_config {
  int32_t num_layers;        /* L */
  int32_t num_q_heads;       /* Hq */
  int32_t num_kv_heads;      /* Hkv; Hq / Hkv in {1, 2, 4, 8} */
  int32_t head_dim;          /* d: 64 or 128 */
  int32_t page_size;         /* b: 256 (the only size the kernels support) */
  int32_t kv_dtype;          /* gp_dtype of the K/V caches */
  int32_t q_dtype;           /* gp_dtype of the query inputs */
  int32_t max_slots;         /* M: rows of the summary pool */
  int32_t num_pages;         /* physical pages in the K/V caches */
  int32_t max_pages_per_req; /* block-table capacity; at most 256 */
  int32_t recent_window;     /* R: always-kept recent tokens, 0 <= R < b */
  int32_t k_loc;             /* Eq. 10 per-block quota */
  int32_t reserve_pages;     /* Grow only while free pages > reserve (Sec. 4.2) */
  int32_t policy;            /* gp_policy */
  double beta_s;             /* short-summary decay */
  double beta_l;             /* long-summary decay */
  double p;                  /* coverage target of D_p, 0 < p < 1 */
  double tau;                /* decision threshold on Delta */
  double rope_theta;         /* rotate-half RoPE base */
  /* policy variants (App. H.1); defaults 0.7, -0.005, 4 pages, 0 */
  double random_compress;    /* RANDOM: probability of Compress & Hold */
  double shrink_threshold;   /* SHRINK: Shrink iff Delta < this */
  int32_t shrink_floor_pages;/* SHRINK: no Shrink at or below this many pages */
  uint32_t random_seed;      /* RANDOM: seed of the counter-based draws */
  int32_t demand_metric;     /* gp_metric; default TOP_P */
} gp_config;

/* One request as the caller's scheduler sees it.  block_table is a HOST
 * array owned by the caller, capacity max_pages_per_req, holding num_pages
 * physical page ids in logical order.  gp_grow_page and gp_compress_hold
 * rewrite it in place.  pos is the current decode position (tokens
 * generated so far, evicted ones included); RoPE of the summaries uses it. */
typedef struct gp_request {
  int32_t slot;
  int32_t num_pages;
  int32_t* block_table;
  int64_t pos;
} gp_request;

/* Result of the demand estimation for one request (Eqs. 7-8):
 * sum_k_short = sum over (layer, KV head) of K^S, likewise sum_k_long;
 * num_candidates = |C_t| = (P - 1) * b; num_units = L * Hkv;
 * delta = (sum_k_short - sum_k_long) / (num_candidates * num_units).
 * Under GP_METRIC_ENTROPY, eff_short / eff_long = sums over the units of
 * exp(H(a^S)) / exp(H(a^L)) (in unit order), and
 * delta = (eff_short - eff_long) / (num_candidates * num_units); under
 * TOP_P both are 0. */
typedef struct gp_demand {
  int64_t sum_k_short;
  int64_t sum_k_long;
  int32_t num_candidates;
  int32_t num_units;
  double delta;
  double eff_short;
  double eff_long;
} gp_demand;

typedef struct gp_action {
  int32_t kind;      /* gp_action_kind */
  int32_t fallback;  /* 1: Delta asked for Grow but the pool could not grant it */
  int32_t forced;    /* 1: P == 1, nothing to compress, Grow forced */
} gp_action;

typedef struct gp_stats_t {
  int64_t demand_calls;
  int64_t demand_requests;
  int64_t grow;
  int64_t compress;
  int64_t fallback;
  int64_t forced_grow;
  int64_t cow_pages;       /* shared pages replaced by copy-on-write */
  int64_t moved_rows;      /* (layer, head, token) rows moved by compaction */
  int64_t shrink;          /* Shrink decisions (policy SHRINK) */
} gp_stats_t;

typedef struct gp_ctx gp_ctx;

/* ---- lifecycle --------------------------------------------------------- */

/* Fill *cfg with the paper's defaults (shape fields zero). */
gp_status gp_config_default(gp_config* cfg);

/* Create an engine.  k_cache / v_cache: device base addresses of the caller's
 * caches (layout above), which must stay alive and unmoved for the engine's
 * lifetime.  stream: a cudaStream_t (NULL = legacy default stream).
 * If k_cache and v_cache are both NULL the context is host-only: pages,
 * refcounts, slots and decisions work, no CUDA call is made, and the device
 * calls return GP_ERR_STATE.  On success *out owns the engine. */
gp_status gp_create(const gp_config* cfg, void* k_cache, void* v_cache,
                    void* stream, gp_ctx** out);
gp_status gp_destroy(gp_ctx* ctx);
const char* gp_last_error(const gp_ctx* ctx);
const char* gp_status_string(gp_status st);

/* ---- page pool with refcounts (Sec. 4.2, App. E.2) -----------------------
 * Pages index the caller's caches.  Allocation is deterministic: the lowest
 * free id.  gp_page_ref shares a page (prefix caching); gp_page_unref drops
 * one reference and frees the page at zero; an unref of a free page is
 * GP_ERR_INVALID. */
gp_status gp_page_alloc(gp_ctx* ctx, int32_t* page);
gp_status gp_page_ref(gp_ctx* ctx, int32_t page);
gp_status gp_page_unref(gp_ctx* ctx, int32_t page);
gp_status gp_page_refcount(const gp_ctx* ctx, int32_t page, int32_t* rc);
gp_status gp_free_page_count(const gp_ctx* ctx, int32_t* n);

/* ---- summary slots (App. E.1) --------------------------------------------
 * A slot is bound to a running request; its first gp_update_summaries must
 * pass first = 1, which overwrites stale values (no clearing needed). */
gp_status gp_slot_acquire(gp_ctx* ctx, int32_t* slot);
gp_status gp_slot_release(gp_ctx* ctx, int32_t slot);

/* ---- hot path -------------------------------------------------------------
 * gp_update_summaries: Sec. 3.2 Eq. 6 with the App. E.1 initialisation, for
 * n requests of one decode step.  slots_dev: int32[n] device; q_dev:
 * [L][n][Hq][d] q_dtype device; first_dev: uint8[n] device (1 = slot's first
 * step).  Asynchronous.  Slot ids out of range are skipped and reported as
 * GP_ERR_INVALID by the next synchronising call. */
gp_status gp_update_summaries(gp_ctx* ctx, int32_t n, const int32_t* slots_dev,
                              const void* q_dev, const uint8_t* first_dev);

/* gp_boundary_demand: for n requests at a capacity boundary (each holding
 * num_pages full pages), App. E.1 Eq. 12 calibration against q_cur, RoPE at
 * pos, scores of both summaries against every key of the request through
 * its block table, softmax over C_t = [0, (P-1) b) and D_p per (layer, KV
 * head) (Eqs. 2 and 7), and Delta (Eq. 8).  q_cur_dev: [L][n][Hq][d] q_dtype
 * device (the same q_t just passed to gp_update_summaries).  out: host
 * gp_demand[n].  It also caches, per (layer, KV head), the importance
 * max(a^S, a^L) of Eq. 9 over [0, P b - R) for a following
 * gp_compress_hold.  Synchronises the stream. */
gp_status gp_boundary_demand(gp_ctx* ctx, int32_t n, const gp_request* reqs,
                             const void* q_cur_dev, gp_demand* out);

/* gp_boundary_demand_noalloc: the same demand estimation as
 * gp_boundary_demand (same kernels, same results) for callers that must not
 * allocate memory -- for example a serving process that reserves all of its
 * GPU memory at start-up so that no request can fail later on an
 * out-of-memory error and no cudaMalloc/cudaFree synchronises the device
 * mid-flight.  The paper has no counterpart to this call.
 * It calls no cudaMalloc, cudaFree or other allocating routine: every
 * temporary (request descriptors, block tables, calibrated summaries and
 * their tensor-core operands, importance values, a-values, arrival tickets,
 * per-unit D_p and their sums) lives in one file-scope device array of
 * 64 MiB that every GPU loading the library holds until the process exits.
 * A call needing more is rejected with GP_ERR_INVALID and a message naming
 * the size; n is at most 512.  The need: per request, its importance values
 * and a-values, L * Hkv * (4 (P b - R) + 8 (P - 1) b) bytes (about
 * 12 L Hkv P b; each region rounded up to 256 bytes), plus per (layer, KV
 * head) of every request 16 * 8 * 26 bytes of partial softmax statistics,
 * 8 G d bytes of calibrated summaries, (d / 64) * 128 * ceil(6 G / 16) * 16
 * bytes of tensor-core operand and 16 bytes of counters -- about 15.3 KiB at
 * d = 128, G = 4 -- plus small descriptor arrays.  On the first call on a device, with that device current, the
 * array's address is looked up once (cudaGetSymbolAddress); make that first
 * call before any stream capture.  All calls share the array and its host
 * staging, which keep the last call's contents: calls that overlap on the
 * GPU, or run on several host threads at once, race.  Inputs and outputs
 * are the caller's: out is host gp_demand[n]; k_units, if not NULL, is host
 * int32[n][L * Hkv][2] receiving K^S, K^L per (layer, KV head).  It does not
 * prepare a following gp_compress_hold: the demand records that an earlier
 * gp_boundary_demand left for these slots are dropped, so a
 * gp_compress_hold of them returns GP_ERR_STATE until the next
 * gp_boundary_demand.  Device-side errors are reported as by gp_synchronize.
 * Contexts with demand_metric GP_METRIC_ENTROPY are refused
 * (GP_ERR_UNSUPPORTED); eff_short and eff_long are 0.
 * Synchronises the stream. */
gp_status gp_boundary_demand_noalloc(gp_ctx* ctx, int32_t n, const gp_request* reqs,
                                     const void* q_cur_dev, gp_demand* out,
                                     int32_t* k_units);

/* gp_decide: per the configured policy (gp_policy above; GROWPAGE: Grow iff
 * Delta > tau, else Compress & Hold, Sec. 3.2).  Delta is compared as
 * delta = (sum_k_short - sum_k_long) / (num_candidates * num_units) in
 * double (for tau == 0 the Grow test is the exact integer one); under
 * GP_METRIC_ENTROPY as (eff_short - eff_long) / (num_candidates *
 * num_units), compared with tau in double.  P == 1
 * forces Grow; a Grow that would leave the pool at or below reserve_pages
 * (counting earlier grants of this call) becomes a fallback Compress
 * (Sec. 4.2, App. H.2).  Host only. */
gp_status gp_decide(gp_ctx* ctx, int32_t n, const gp_request* reqs,
                    const gp_demand* demand, gp_action* out);

/* gp_grow_page: Grow by One Page -- take the lowest free page (refcount 1)
 * and append it to req->block_table (num_pages + 1).  GP_ERR_NO_PAGES or a
 * full block table leave the request unchanged.  Host only. */
gp_status gp_grow_page(gp_ctx* ctx, gp_request* req);

/* Device-side errors of the asynchronous calls below (a failed check inside a
 * kernel, or a bounded wait that gave up) are reported by the next call that
 * synchronises with the engine -- gp_synchronize, gp_boundary_demand or an
 * inspection call -- as GP_ERR_INVALID or GP_ERR_TIMEOUT.  The host-side state
 * of the failed call (block tables, refcounts, the pool) was committed when it
 * returned GP_OK; the K/V rows of the units it was compacting are then
 * unspecified.  Errors found before the launch (arguments, GP_ERR_NO_PAGES, a
 * launch that fails) change nothing.
 *
 * gp_compress_hold: Compress & Hold for n requests, each of which must have
 * been passed to the last gp_boundary_demand with the same slot, pages and
 * block table (else GP_ERR_STATE).  Per (layer, KV head): importance
 * (Eq. 9), the recent R tokens always kept, block-local top-k_loc' with
 * k_loc' = min(k_loc, |B_j|, floor(K_t / P)) plus global top-(K_t - |S_loc|)
 * (Eq. 10, K_t = (P-1) b - R, equal scores: lower slot first), then stable
 * compaction: the k-th kept slot moves to logical slot k.  Copy-on-write
 * (App. E.2): every page with refcount > 1 is first replaced in the block
 * table by a fresh page (lowest id first, ascending logical order) and the
 * request's reference to the shared page is dropped after the copy.
 * num_pages is unchanged; logical slots [(P-1) b, P b) become free.
 * GP_ERR_NO_PAGES (not enough fresh pages for copy-on-write) changes
 * nothing.  Asynchronous on the stream. */
gp_status gp_compress_hold(gp_ctx* ctx, int32_t n, gp_request* reqs);

/* gp_shrink: Shrink (App. H.1, Eq. 13) for n requests prepared like those of
 * gp_compress_hold (a gp_boundary_demand on the same slot, pages and block
 * table): the same selection and copy-on-write as Compress & Hold, but with
 * K_t = (P-2) b - R, so two pages' worth of history is compacted into
 * logical slots [0, (P-2) b); the last page of the (new) block table is
 * then returned to the pool (its reference dropped) and num_pages becomes
 * P - 1, which leaves one page of free slots [(P-2) b, (P-1) b).  Needs
 * P >= 3 (else GP_ERR_INVALID).  GP_ERR_NO_PAGES (copy-on-write) changes
 * nothing.  Asynchronous on the stream. */
gp_status gp_shrink(gp_ctx* ctx, int32_t n, gp_request* reqs);

/* gp_compress_fill: Compress & Hold with hole-fill compaction -- NOT the
 * paper's compaction, an order-destroying variant that moves far fewer
 * bytes.  Selection and copy-on-write as gp_compress_hold (same keep
 * masks), but the kept slots of the first P-1 logical pages stay where they
 * are and the kept slots of the last page fill the holes (dropped slots of
 * the first P-1 pages): the k-th kept slot of the last page (ascending) goes
 * to the k-th hole (ascending).  Logical order and block locality are not
 * preserved; num_pages is unchanged and logical slots [(P-1) b, P b) become
 * free.  At most one page of rows moves per (layer, KV head).
 * Asynchronous on the stream. */
gp_status gp_compress_fill(gp_ctx* ctx, int32_t n, gp_request* reqs);

/* gp_compact_kv: the compaction step of Compress & Hold for a caller-given
 * index set (App. E.2), with the same copy-on-write handling.
 * keep_masks_dev: device uint32, per request [L][Hkv][ceil(P b / 32)] bit
 * masks (bit i%32 of word i/32 = keep slot i), requests concatenated in
 * order; each (layer, KV head) must keep exactly (P-1) b slots (else the
 * masks are rejected with GP_ERR_INVALID at the next synchronising call and
 * that unit is not moved).  Asynchronous. */
gp_status gp_compact_kv(gp_ctx* ctx, int32_t n, gp_request* reqs,
                        const uint32_t* keep_masks_dev);

/* gp_decode_attention: one layer of a decode step -- attention over each
 * request's paged cache with the summary update fused in, where the paper
 * integrates it (Sec. 4.1: the decode attention kernel updates the query
 * summaries in passing).  For request r and query head g (KV head g / G):
 *   the summaries of (layer, slot, g) are updated from the PRE-RoPE query q
 *   exactly as gp_update_summaries does (first_dev[r]: both set to q);
 *   z_i = RoPE_pos(q) . k_i / sqrt(d) over the first num_tokens[r] logical
 *   slots (keys are stored rotated, rotate-half at rope_theta), a =
 *   softmax(z), out[r][g] = sum_i a_i v_i.
 * q_dev: device [n][Hq][d] in q_dtype; first_dev: device uint8 [n];
 * num_tokens: HOST int32 [n], 0 <= num_tokens[r] <= num_pages * 256 (0 gives
 * a zero output); the cache slots past num_tokens[r] may hold any bits, NaN
 * and inf included: they do not reach the output.  out_dev: device fp32
 * [n][Hq][d], 4-byte aligned.  Requests need not be at a boundary.  bf16
 * caches with d = 128 and 2 or 4 query heads per KV head run on the
 * tensor-core kernel, everything else (or everything, under
 * gp_set_scan_kernel(CUDA_CORE)) on the CUDA-core one; both give the same
 * results within fp32 tolerances.  With a compaction pending on the side stream (see
 * gp_set_compaction_stream), the call makes the engine stream wait for it
 * only if one of its requests holds a page that compaction reads or writes;
 * otherwise the attention runs concurrently with it (App. E.3).  out_dev must
 * not overlap q_dev.  Asynchronous on the engine stream, which must not be
 * capturing a graph (GP_ERR_UNSUPPORTED, as below). */
gp_status gp_decode_attention(gp_ctx* ctx, int32_t layer, int32_t n, const gp_request* reqs,
                              const int32_t* num_tokens, const void* q_dev, const uint8_t* first_dev,
                              float* out_dev);

/* ---- eviction by accumulated attention weight ---------------------------------
 * The common alternative to the demand estimate: keep the tokens that received
 * the most attention so far, and a recent window.  Four calls carry it from
 * the prompt on: gp_append_tokens writes new tokens, gp_chunk_attention (a
 * prompt, or a few drafted tokens) and gp_decode_attention_weighted (one token)
 * attend and add the weights they give, gp_evict_weighted evicts by them.
 *
 * Accumulated weights ("weights_dev"): device fp32
 * [L][max_slots][Hkv][max_pages_per_req * 256], owned by the caller, 4-byte
 * aligned, indexed by request slot and logical token -- not by page, so
 * requests that share prefix pages gather weights of their own.  Entry i of
 * (layer, slot, h) is the sum over the queries so far of the softmax weights
 * of token i, summed over the query heads of KV head h.  gp_append_tokens
 * clears the entries of the tokens it writes, so the array needs no clearing
 * of its own; entries past a request's tokens are never read or written.
 * The sums are fp32, each entry has one writer per call and a fixed order:
 * the same calls give the same bits.
 *
 * The calls share these rules.  Requests need a bound slot, listed once per
 * call.  Arguments are checked before anything happens (GP_ERR_INVALID,
 * nothing changed).  The device current at gp_create must be current
 * (GP_ERR_INVALID), and neither the engine stream nor the compaction stream may
 * be capturing a graph (GP_ERR_UNSUPPORTED: a replay would not see a later call's tables and
 * lengths).  They run on the engine stream, asynchronously, and wait there
 * for a pending side-stream compaction only if a request holds one of its
 * pages or a slot whose weights it moves.  Two contexts share no scratch and may run at the same time.
 *
 * gp_append_tokens: new tokens of one layer into the cache.  Request r appends
 * num_new[r] >= 0 tokens after its num_cached[r] >= 0 cached ones; the rows of
 * q, k and v are packed, request after request.  Token t goes to logical slot
 * num_cached[r] + t of the request's pages with its key rotated (rotate-half
 * RoPE at position reqs[r].pos + t, rope_theta; angles in fp64, one rounding
 * to kv_dtype) and its value copied; q_rot gets the rotated queries, rounded
 * to q_dtype, as gp_chunk_attention takes them.  q_dev, q_rot_dev: device
 * [rows][Hq][d] q_dtype, both or neither NULL, the same buffer or disjoint ones;
 * k_dev, v_dev: device [rows][Hkv][d] kv_dtype, apart from q_rot; weights_dev
 * may be NULL.
 * All but weights_dev 16-byte aligned, as the caches.  num_cached and num_new:
 * HOST int32 [n]; the tokens must fit the request's pages, and a page written
 * must have one reference and be written by one request of the call
 * (GP_ERR_INVALID: copy a shared page first).  A gp_boundary_demand result of
 * the slots is stale afterwards (GP_ERR_STATE in gp_compress_hold). */
gp_status gp_append_tokens(gp_ctx* ctx, int32_t layer, int32_t n, const gp_request* reqs,
                           const int32_t* num_cached, const int32_t* num_new, const void* q_dev,
                           const void* k_dev, const void* v_dev, void* q_rot_dev, float* weights_dev);

/* gp_decode_attention_weighted: gp_decode_attention (same arguments, same
 * outputs) that also adds its softmax weights: entry i
 * < num_tokens[r] of (layer, slot, h) grows by the sum over the G query heads
 * of a_i.  first_dev may be NULL: the summaries are then left as they are. */
gp_status gp_decode_attention_weighted(gp_ctx* ctx, int32_t layer, int32_t n, const gp_request* reqs,
                                       const int32_t* num_tokens, const void* q_dev, const uint8_t* first_dev,
                                       float* out_dev, float* weights_dev);

/* gp_chunk_attention: causal attention of one layer for num_new[r] >= 0 tokens
 * of each request that are already in the cache behind num_cached[r] others
 * (gp_append_tokens): token t attends to the logical slots
 * [0, num_cached[r] + t + 1), z = q . k / sqrt(d), a = softmax(z),
 * out = sum a v.  q_dev: device [rows][Hq][d] q_dtype, ROTATED, packed as in
 * gp_append_tokens; out_dev: the same shape and type; both 16-byte aligned.
 * With weights_dev, the weights of every token are added; NULL leaves that
 * out.  Nothing takes added weights back: for drafted tokens that may yet be
 * rejected, call with NULL, and once they are settled again with weights_dev and
 * the accepted count of each request as num_new (their rows of q packed anew).
 * The rows of K and V of the attended tokens must be finite; cache slots
 * past num_cached[r] + num_new[r] may hold any bits.  out_dev must not overlap
 * q_dev.  bf16 caches and queries run on the tensor-core kernels, which hold
 * the softmax weights to 2^-15 of themselves for the product with V (out is
 * bf16; the accumulated weights are not rounded); the rest, or everything under
 * gp_set_scan_kernel(CUDA_CORE), on CUDA-core ones in fp32. */
gp_status gp_chunk_attention(gp_ctx* ctx, int32_t layer, int32_t n, const gp_request* reqs,
                             const int32_t* num_cached, const int32_t* num_new, const void* q_dev,
                             void* out_dev, float* weights_dev);

/* gp_evict_weighted: evict request r's num_tokens[r] tokens down to
 * keep_tokens[r] >= 1, per (layer, KV head): the min(recent_window, keep)
 * most recent tokens stay, and of the others the keep - that many of largest
 * accumulated weight (equal weights: the lower slot; NaN counts as larger
 * than any number). K, V and the weights of the kept tokens move, in order,
 * to the logical slots [0, keep); num_pages is unchanged and the slots from
 * keep on become free, their contents unspecified. A request with num_tokens
 * <= keep_tokens is left as it is. Copy-on-write as in gp_compress_hold for
 * the requests that evict (GP_ERR_NO_PAGES: nothing changed); a page of
 * several of them must have a reference for each (GP_ERR_INVALID). Shared
 * pages past keep are replaced too, as they hold the next tokens. A caller
 * that wants the emptied pages back, [ceil(keep / 256), num_pages), unrefs
 * each and lowers num_pages, at once also with a side stream: an append to
 * such a page waits for the eviction that still reads it. num_tokens and
 * keep_tokens: HOST int32 [n]. Runs on the compaction stream if one is set,
 * with gp_compress_hold's rules, which hold for the weights of the evicted
 * requests as for their K/V; a gp_boundary_demand result of the slots is
 * stale afterwards. gp_debug_keep_mask gives the kept sets. */
gp_status gp_evict_weighted(gp_ctx* ctx, int32_t n, gp_request* reqs, const int32_t* num_tokens,
                            const int32_t* keep_tokens, float* weights_dev);

/* ---- a step over device arrays, and attention over selected blocks ---------------
 * The alternative to eviction: every token stays cached, and a query reads only
 * the blocks of keys that a cheap score selects for it.  Five calls carry a step:
 * gp_build_tables lays out its rows, gp_append_mapped writes their keys and
 * values, gp_block_bounds bounds the keys of the blocks they fall into,
 * gp_select_blocks lists the blocks of each row, gp_sparse_attention attends to
 * them.  gp_build_tables is called once a step, the others once a layer.
 *
 * They take lengths and block tables from DEVICE arrays (gp_step), which the
 * host never sees: lengths that only the GPU knows (accepted drafts) need no
 * way back, and the calls CAN be captured into a CUDA graph and replayed over
 * other contents of the same arrays.  They use no scratch of the engine: graphs
 * share nothing but the caller's buffers.
 *
 * They share these rules.  Addresses, sizes and options are checked before
 * anything happens (GP_ERR_INVALID, nothing changed); the device current at
 * gp_create must be current (GP_ERR_INVALID).  What the device arrays hold is
 * checked by the kernels.  A row whose request, slot or place is outside the
 * engine's sizes is left out: its outputs stay as they were, the other rows of its
 * request take part.  To gp_append_mapped that is a slot_map outside the pool; to the
 * last three calls a row takes part if row_req names its request and row0 agrees,
 * row0[r] <= row < row0[r + 1], and if its own token has a place in the table.  A page
 * of a table that is outside the pool counts for nothing (to gp_select_blocks: for any
 * page).  Both are reported by the next synchronising call as GP_ERR_INVALID.  Rows
 * whose row_req (slot_map) is -1 and those behind the step's last one, from row0[n] on, are
 * left as they were without a report.  row0 must ascend; where it does not, which
 * rows take part is not defined.  Block sizes are 16, 32, 64, 128 or 256 tokens.
 * max_rows times the KV heads is below 2^27 (GP_ERR_UNSUPPORTED).  gp_set_timing does not time captured launches.
 * All run on the engine stream, asynchronously.  Those that read or write K/V
 * (gp_append_mapped, gp_block_bounds, gp_sparse_attention) wait there for a
 * compaction pending on the side stream, whatever its pages; a call that is
 * being captured is refused while one is (GP_ERR_STATE), and a graph's launches
 * do not wait: gp_wait_compaction on the launching stream comes first.
 *
 * gp_step: the arrays of one step, device memory of the caller, 4-byte (64-bit
 * ones 8-byte) aligned and apart from one another.  The first four are inputs of
 * gp_build_tables; tables is read and extended by it; the last four are what it
 * writes.  gp_append_mapped reads slot_map and positions, the other three calls slots,
 * num_cached, tables, row0 and row_req.  A caller may fill them by other means.
 *   n          requests, at most max_slots and 4096
 *   max_rows   rows that the step's buffers have room for (new tokens of all
 *              requests together).  The host knows no other count: launches are
 *              sized by it, and gp_select_blocks (above 8 rows a request) and
 *              gp_sparse_attention (above 16 Hkv / Hq) take the kernels for prompts
 *              by it.  A step of single tokens is faster with room for its rows alone:
 *              a gp_step of its own, over the same arrays
 *   slots      int32 [n], the requests' slots (gp_slot_acquire), listed once
 *   num_cached int32 [n], tokens in the cache before the step
 *   num_new    int32 [n], tokens of the step
 *   pos        int64 [n], rotary position of the first new token
 *   tables     int32 [max_slots][max_pages_per_req], block tables by slot
 *   row0       int32 [n + 1], first row of each request, and the rows in all
 *   row_req    int32 [max_rows], a row's request (index below n), -1: none
 *   slot_map   int64 [max_rows], page * 256 + place in the page, -1: none
 *   positions  int64 [max_rows], rotary position */
typedef struct gp_step {
  int32_t n;
  int32_t max_rows;
  const int32_t* slots;
  const int32_t* num_cached;
  const int32_t* num_new;
  const int64_t* pos;
  int32_t* tables;
  int32_t* row0;
  int32_t* row_req;
  int64_t* slot_map;
  int64_t* positions;
} gp_step;

/* What became of a request in gp_build_tables. */
typedef enum {
  GP_STEP_GIVEN = 0,    /* its rows are in the step */
  GP_STEP_NO_PAGES = 1, /* the free list has too few pages */
  GP_STEP_NO_ROWS = 2,  /* its rows do not fit behind those that the valid requests before it ask for */
  GP_STEP_INVALID = 3   /* slot out of range or listed twice, a negative length, more tokens
                           than max_pages_per_req pages, or cached ones without a page */
} gp_step_state;

/* gp_build_tables: rows, block tables, slot map and positions of a step.
 * Request i with slot s holds held[s] pages; it needs ceil((num_cached[i] +
 * num_new[i]) / 256) and takes the ones missing from free_dev, behind those taken
 * by the requests before it.  A request whose rows or pages do not fit
 * has no row in this step, takes no page and keeps its table.  Both are given in
 * order, and none is passed over.  Rows: the new tokens of all valid requests are added
 * up, those of refused ones among them, and from where the sum passes max_rows no
 * request with new tokens has a row.  Pages: from where the missing ones of the requests
 * whose rows fit pass the list, no request takes any; later ones that need none still
 * have their rows.  free_dev: int32 [num_free], pages that the caller took with
 * gp_page_alloc, each listed once, of which the first taken_in[0] (NULL: none) are
 * used up; taken_dev: int32 [1] gets the count after the call, and may be
 * taken_in.  held_dev: int32 [max_slots]; num_pages_dev: int32 [max_slots] gets the
 * pages of the listed slots after the call, and may be held_dev: a call repeated
 * over the same lengths then takes nothing.  state_dev: int32 [n], gp_step_state,
 * apart from the inputs.
 * Which pages a request was given, only its row of tables tells.  When it ends, or
 * before a call that takes a host table (Compress & Hold, an eviction), the caller copies
 * that row back, num_pages_dev[slot] entries of it: one gp_page_unref each, or the
 * gp_request's block_table, whose row on the device is written again after a call that
 * changes it. */
gp_status gp_build_tables(gp_ctx* ctx, const gp_step* step, const int32_t* held_dev, int32_t* num_pages_dev,
                          const int32_t* free_dev, int32_t num_free, const int32_t* taken_in_dev, int32_t* taken_dev,
                          int32_t* state_dev);

/* Rotary forms.  Pairs of a head's first rotary_dim dimensions are rotated by
 * position * f_i, the other dimensions copied: (i, i + rotary_dim / 2) in the HALF
 * layout, (2 i, 2 i + 1) in the INTERLEAVED one.  Before scaling
 * f_i = theta^(-2 i / rotary_dim).  Scaling for contexts longer than
 * original_length, by `factor` >= 1:
 *   LINEAR  f_i / factor
 *   BANDS   with t_i = original_length f_i / (2 pi), the turns of pair i over the
 *           original length: f_i / factor where t_i <= low_turns, f_i where
 *           t_i >= high_turns, between them k f_i + (1 - k) f_i / factor,
 *           k = (t_i - low_turns) / (high_turns - low_turns)
 *   RAMP    the same blend by the pair's index: with
 *           p(t) = rotary_dim ln(original_length / (2 pi t)) / (2 ln theta), a =
 *           max(0, floor(p(high_turns))), b = min(rotary_dim - 1, ceil(p(low_turns))),
 *           the part of f_i / factor is (i - a) / (b - a) held to [0, 1] (b - a
 *           at least 0.001)
 * Sine and cosine are multiplied by `amplitude`; 0 stands for 0.1 ln(factor) + 1
 * under RAMP and for 1 otherwise. */
typedef enum { GP_ROPE_HALF = 0, GP_ROPE_INTERLEAVED = 1 } gp_rope_layout;
typedef enum { GP_ROPE_NONE = 0, GP_ROPE_LINEAR = 1, GP_ROPE_BANDS = 2, GP_ROPE_RAMP = 3 } gp_rope_scaling;
typedef struct gp_rope {
  int32_t layout;          /* gp_rope_layout */
  int32_t rotary_dim;      /* a multiple of 16 up to head_dim; 0: no rotation */
  int32_t scaling;         /* gp_rope_scaling */
  int32_t original_length; /* BANDS, RAMP: at least 1 */
  double theta;            /* above 1 */
  double factor;
  double low_turns;        /* below high_turns, above 0 */
  double high_turns;
  double amplitude;        /* 0: by the rule above */
} gp_rope;

/* Fill *rope with: HALF, rotary_dim 0, NONE, original_length 8192, theta 10000, factor
 * 1, low_turns 1, high_turns 0 (which stands for 4 under BANDS and 32 under RAMP),
 * amplitude 0. */
gp_status gp_rope_default(gp_rope* rope);

/* gp_append_mapped: the step's new tokens of one layer into the cache, as
 * gp_append_tokens, but by slot_map and positions and in any of the rotary forms.
 * q_dev, k_dev, v_dev: device [max_rows] rows of [Hq][d] q_dtype and [Hkv][d]
 * kv_dtype, whose starts lie q_stride, k_stride and v_stride elements apart (at
 * least the row, so that all three may be columns of one projection's output);
 * q_rot_dev: [max_rows][Hq][d], packed, apart from the inputs, or q_dev itself if
 * that is packed.  q and q_rot both or neither NULL.  All 16-byte aligned, strides
 * too.  A page written must be the request's alone: the engine does not see the
 * tables and cannot check.  Accumulated weights are not cleared (an
 * append that feeds them is gp_append_tokens).  gp_boundary_demand results of all slots
 * are stale afterwards; a graph's launches do not mark them so: after one, the next
 * gp_compress_hold needs a new gp_boundary_demand all the same. */
gp_status gp_append_mapped(gp_ctx* ctx, int32_t layer, const gp_step* step, const gp_rope* rope, const void* q_dev,
                           int64_t q_stride, const void* k_dev, int64_t k_stride, const void* v_dev, int64_t v_stride,
                           void* q_rot_dev);

/* gp_block_bounds: bounds of the keys of each block that a row of the step falls
 * into, over all tokens of the block up to the request's last (older ones are read
 * again).  bounds_dev: int8 [L][num_pages][Hkv][256 / block][2][d], 16-byte aligned,
 * scales_dev: fp32 [L][num_pages][Hkv][256 / block]; the caller's, by page, so
 * that requests share those of a shared prefix.  Per (block, KV head): e is the
 * least whole number >= -100 with max |k| <= 127 * 2^e (at most 100), the scale is
 * 2^e, and dimension i has [0][i] = floor(min k_i / 2^e) and [1][i] = ceil(max k_i /
 * 2^e), held to [-127, 127].  NaN keys are left out (a dimension with no other
 * counts as 0).  A call that moves keys (Compress & Hold, an eviction) leaves the
 * bounds of its pages stale: a step with num_cached = 0 and num_new = the tokens
 * left forms them again (its rows need no queries). */
gp_status gp_block_bounds(gp_ctx* ctx, int32_t layer, const gp_step* step, int32_t block, int8_t* bounds_dev,
                          float* scales_dev);

/* gp_select_blocks: the blocks that each row attends to, per KV head.  With the
 * group's queries as whole numbers Q_g = round(q_g / 2^e) in [-127, 127] (e as above,
 * of all of the group), a block's score is the sum over g and i of the larger of
 * Q_gi lo_i and Q_gi hi_i, times its scale: what the group's logits can reach in it.
 * A row in block b attends to blocks of [0, b]: all of them if they are `top` or
 * fewer, else the first `sink`, the last `recent` >= 1, and of the others those of
 * largest score (equal scores: the lower block), `top` >= sink + recent in all.
 * The arithmetic is exact; a NaN in a query counts as 0.  q_rot_dev: [max_rows][Hq][d] q_dtype, 16-byte aligned,
 * as gp_append_mapped gives it; blocks_dev: int32 [max_rows][Hkv][top], ascending,
 * then -1. */
gp_status gp_select_blocks(gp_ctx* ctx, int32_t layer, const gp_step* step, int32_t block, int32_t top, int32_t sink,
                           int32_t recent, const void* q_rot_dev, const int8_t* bounds_dev, const float* scales_dev,
                           int32_t* blocks_dev);

/* gp_sparse_attention: attention of each row over the tokens, up to its own, of
 * the blocks listed for it: z = q . k / sqrt(d), a = softmax(z), out = sum a v.
 * blocks_dev: int32 [max_rows][Hkv][top]; a list is ascending and ends at the first
 * entry that is negative, not above the one before it, or past the row's own
 * block; an empty one gives 0, a query with NaN or an infinite logit NaN.  q_rot_dev, out_dev: [max_rows][Hq][d] q_dtype,
 * 16-byte aligned, apart.  Keys and values of the listed blocks, up to the
 * request's last token of the step, must be finite; other cache slots may hold any
 * bits. */
gp_status gp_sparse_attention(gp_ctx* ctx, int32_t layer, const gp_step* step, int32_t block, int32_t top,
                              const void* q_rot_dev, const int32_t* blocks_dev, void* out_dev);

/* ---- asynchronous compaction (App. E.3: compaction overlapped with decoding)
 * gp_set_compaction_stream: from now on the compaction of gp_compress_hold,
 * gp_shrink, gp_compress_fill, gp_compact_kv and gp_evict_weighted runs on `stream` (a caller
 * CUDA stream; NULL: the engine stream again).  Each such call makes the
 * side stream wait for the work the engine stream holds at that point, then
 * returns without waiting for the compaction; the block tables and the page
 * pool are updated on the host as before.  While it runs, gp_update_summaries
 * (which touches no K/V), gp_decode_attention of requests that share no page
 * with it, and the caller's work on other streams may overlap it; every
 * later engine call that reads K/V or the engine's scratch (demand,
 * compaction, inspection, gp_stats, gp_synchronize, gp_destroy) first waits
 * for it on the host.  Before reading the compacted requests' K/V, the
 * caller makes its own stream wait with gp_wait_compaction.  The pages such
 * a call releases (shared pages replaced by copy-on-write, the page Shrink
 * returns) are back in the pool when it returns, while the side stream may
 * still read them: a caller that writes into a page the pool hands out
 * (gp_page_alloc, gp_grow_page) makes the writing stream wait with
 * gp_wait_compaction first.  Waits for a pending compaction first. */
gp_status gp_set_compaction_stream(gp_ctx* ctx, void* stream);
/* gp_wait_compaction: `stream` (NULL: the engine stream) waits for the last
 * compaction launched on the side stream (no-op if none ever was).  It
 * enqueues the wait and returns at once. */
gp_status gp_wait_compaction(gp_ctx* ctx, void* stream);

/* ---- inspection (tests, benchmarks) ---------------------------------------
 * All of these synchronise the stream.  req_idx indexes the request list of
 * the last gp_boundary_demand (k, probabilities, scores) or of the last
 * gp_compress_hold or gp_evict_weighted (keep masks). */

/* K^S, K^L per unit: k_out host int32[L * Hkv * 2] ([unit][x]). */
gp_status gp_debug_demand_k(gp_ctx* ctx, int32_t req_idx, int32_t* k_out);
/* Importance log2 max(a^S, a^L) over [0, P b - R): host float[L*Hkv][P b - R]. */
gp_status gp_debug_scores(gp_ctx* ctx, int32_t req_idx, float* out);
/* Demand distributions a^S, a^L over C_t: host float[L*Hkv][2][(P-1) b]
 * (the kernels keep them for the D_p select of every demand call). */
gp_status gp_debug_probs(gp_ctx* ctx, int32_t req_idx, float* out);
/* Keep masks of the last gp_compress_hold: host uint32[L*Hkv][ceil(P b/32)]. */
gp_status gp_debug_keep_mask(gp_ctx* ctx, int32_t req_idx, uint32_t* out);
/* Effective support sizes exp(H(a^S)), exp(H(a^L)) per unit of the last
 * demand call: host double[L * Hkv * 2] ([unit][x]).  GP_ERR_STATE unless
 * the context's demand_metric is GP_METRIC_ENTROPY. */
gp_status gp_debug_entropy(gp_ctx* ctx, int32_t req_idx, double* out);
/* Summaries of one slot: host double[L][2][Hq][d]. */
gp_status gp_read_summaries(gp_ctx* ctx, int32_t slot, double* out);

/* gp_synchronize: waits for every piece of engine work (the engine stream,
 * the speculative selection, a side-stream compaction) and reports the
 * device-side errors of earlier asynchronous calls: GP_ERR_TIMEOUT if only
 * bounded waits gave up, GP_ERR_INVALID if a device-side check failed (the
 * text names the error bits), GP_OK otherwise.  The error word is cleared. */
gp_status gp_synchronize(gp_ctx* ctx);

/* gp_debug_attention_plan: the work split gp_decode_attention gives the
 * tensor-core attention kernel for n requests attending to num_tokens[r]
 * tokens on a device of `sms` SMs, computed on the host without launching
 * anything (also on a host-only context).  Every (request, KV head) pair's
 * attended pages are laid end to end and cut into one even range per SM;
 * each range's pieces are one CTA's items.  items_out: host int32
 * [max_items][8], per item (request, KV head, piece, pieces of the pair,
 * first page, tiles of 128 keys, first item of the pair, CTA), items of a
 * CTA consecutive and CTAs in order.  *n_items, *n_ctas: the counts (set
 * also when max_items is too small, which returns GP_ERR_INVALID).  Host
 * only. */
gp_status gp_debug_attention_plan(gp_ctx* ctx, int32_t n, const int32_t* num_tokens, int32_t sms,
                                  int32_t max_items, int32_t* items_out, int32_t* n_items, int32_t* n_ctas);

/* ---- test hooks -------------------------------------------------------------
 * gp_debug_set_wait_limit: the limit, in SM clock cycles, of the bounded copy
 * waits of later launches of `kernel` (GP_KERNEL_COMPRESS: the compaction;
 * GP_KERNEL_SELECT: the speculative selection; GP_KERNEL_EVICT: the eviction's
 * waits for rows still to be read; GP_KERNEL_CHUNK, GP_KERNEL_WEIGHTS,
 * GP_KERNEL_SPARSE: the waits inside the tensor-core chunk attention, its weights and
 * the tensor-core kernels of gp_sparse_attention); 0 makes each
 * such wait give up at once (of the last three, those for a free buffer), a
 * negative value restores the default of 2^31 (about one second).  A wait that gives up makes its CTA wait for the copies it already
 * issued (always with the default limit), record a timeout and return;
 * gp_synchronize then reports GP_ERR_TIMEOUT.  (gp_sparse_attention leaves a row and head
 * whose blocks were not all attended to as it was.)  Other kernels:
 * GP_ERR_UNSUPPORTED.  Host only; for tests of the timeout path.
 * gp_debug_fail_next_launch: the next launch of `kernel` (GP_KERNEL_*) fails
 * without running, as a failed launch would (GP_ERR_CUDA); -1 clears it.
 * Host only; for tests of the rollback paths. */
gp_status gp_debug_set_wait_limit(gp_ctx* ctx, int32_t kernel, int64_t cycles);
gp_status gp_debug_fail_next_launch(gp_ctx* ctx, int32_t kernel);

/* Which kernels do the cache-wide contractions: the scan of
 * gp_boundary_demand and the scores and weighted values of
 * gp_decode_attention(_weighted), gp_chunk_attention and gp_sparse_attention (which
 * two take bf16 queries and caches on the tensor cores).  AUTO (default): the tensor-core (tcgen05) kernels
 * where they apply -- the scan for bf16 caches (every request length up to
 * the 256-page block-table limit), attention for bf16 caches with d = 128
 * and 2 or 4 query heads per KV head -- and the CUDA-core (fp32 FMA)
 * kernels otherwise: fp32 caches, other attention shapes, or a K or V cache
 * no tensor map can describe (base not 16-byte aligned, or 2^31 or more key
 * rows).  CUDA_CORE forces the latter everywhere; TENSOR_CORE makes calls the
 * tensor-core kernels cannot serve fail with GP_ERR_UNSUPPORTED.  Both give
 * the same results within the tolerances of fp32 arithmetic.  Host only. */
#define GP_SCAN_AUTO 0
#define GP_SCAN_CUDA_CORE 1
#define GP_SCAN_TENSOR_CORE 2
gp_status gp_set_scan_kernel(gp_ctx* ctx, int32_t kind);

/* Where Compress & Hold's Eq. 10 selection runs (Sec. 3.3).  SPECULATIVE:
 * after every gp_boundary_demand, on an engine-owned stream, while the host
 * reads the sums and decides, so that a following Compress & Hold (or hole
 * fill) only moves rows.  IN_COMPACTION: at the head of each (layer, KV
 * head) unit's compaction CTA, where the copies of the other units' CTAs
 * keep HBM busy.  AUTO (default): speculative for demand calls of at most
 * 4 x (SM count) units that Compress & Hold could take, in the compaction
 * above that.  The keep masks are the same either way.  Host only. */
#define GP_SELECT_AUTO 0
#define GP_SELECT_SPECULATIVE 1
#define GP_SELECT_IN_COMPACTION 2
gp_status gp_set_selection_mode(gp_ctx* ctx, int32_t mode);

/* Per-kernel device time: when enabled, every kernel launch is bracketed by
 * CUDA events on the engine stream.  names: GP_KERNEL_* below.  The query
 * synchronises and returns the summed milliseconds and launch count since
 * the last reset. */
#define GP_KERNEL_EMA 0
#define GP_KERNEL_PREP 1
#define GP_KERNEL_DEMAND 2
#define GP_KERNEL_COMPRESS 3
#define GP_KERNEL_ATTENTION 4
#define GP_KERNEL_SELECT 5
#define GP_KERNEL_ENTROPY 6
#define GP_KERNEL_APPEND 7
#define GP_KERNEL_CHUNK 8
#define GP_KERNEL_WEIGHTS 9        /* the weights of a decode step or a chunk */
#define GP_KERNEL_EVICT_SELECT 10
#define GP_KERNEL_EVICT 11
#define GP_KERNEL_TABLES 12
#define GP_KERNEL_MAPPED 13        /* gp_append_mapped */
#define GP_KERNEL_BOUNDS 14
#define GP_KERNEL_BLOCK_SELECT 15
#define GP_KERNEL_SPARSE 16
#define GP_KERNEL_COUNT 17
gp_status gp_set_timing(gp_ctx* ctx, int32_t enabled);
gp_status gp_kernel_time(gp_ctx* ctx, int32_t kernel, double* ms, int64_t* launches);
gp_status gp_reset_timing(gp_ctx* ctx);

gp_status gp_stats(const gp_ctx* ctx, gp_stats_t* out);

#ifdef __cplusplus
}
#endif

#endif /* GROWPAGE_H */
