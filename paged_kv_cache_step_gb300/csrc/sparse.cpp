// Host side of the calls over a step's device arrays: tables, rotary forms
// through the slot map, block bounds, block selection and attention over the
// listed blocks.  Checks addresses, sizes and options and launches; what the
// arrays hold is checked by the kernels.  Nothing here reads device data or uses
// engine scratch, so the calls can be captured into a graph.
#include "growpage.h"

#include <cuda_runtime.h>

#include <cmath>
#include <cstring>
#include <initializer_list>

#include "engine.h"
#include "sparse_kernels.h"

using namespace gp;

namespace {

struct Span {
  const void* p;
  size_t bytes;
};
bool apart(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return !a.p || !b.p || x >= y + b.bytes || y >= x + a.bytes;
}
bool off(const void* p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

gp_status check_step(gp_ctx* c, const gp_step* s) {
  const gp_config& g = c->cfg;
  if (!s) return fail(c, GP_ERR_INVALID, "null step");
  if (s->n < 0 || s->n > g.max_slots || s->n > kStepMaxRequests)
    return fail(c, GP_ERR_INVALID, "n = %d outside [0, max_slots] or above %d", s->n, kStepMaxRequests);
  if (s->max_rows < 0) return fail(c, GP_ERR_INVALID, "max_rows = %d", s->max_rows);
  // a piece of rows, a KV head and a split each are a block of a launch
  if ((int64_t)s->max_rows * g.num_kv_heads >= (1 << 27)) return fail(c, GP_ERR_UNSUPPORTED, "%d rows in one step", s->max_rows);
  if (!s->row0 || !s->tables || (s->n > 0 && (!s->slots || !s->num_cached || !s->num_new || !s->pos)) ||
      (s->max_rows > 0 && (!s->row_req || !s->slot_map || !s->positions)))
    return fail(c, GP_ERR_INVALID, "null array in the step");
  if (off(s->slots, 4) || off(s->num_cached, 4) || off(s->num_new, 4) || off(s->pos, 8) || off(s->tables, 4) || off(s->row0, 4) ||
      off(s->row_req, 4) || off(s->slot_map, 8) || off(s->positions, 8))
    return fail(c, GP_ERR_INVALID, "misaligned array in the step");
  return GP_OK;
}

gp_status check_layer(gp_ctx* c, int32_t layer, int32_t block) {
  if (layer < 0 || layer >= c->cfg.num_layers) return fail(c, GP_ERR_INVALID, "layer %d", layer);
  if (block != 16 && block != 32 && block != 64 && block != 128 && block != 256)
    return fail(c, GP_ERR_INVALID, "blocks of %d tokens: 16, 32, 64, 128 or 256", block);
  return GP_OK;
}

// A device, the engine's, and for calls that touch K/V no compaction ahead of them.
// *capturing: the engine stream is.
gp_status ready_step(gp_ctx* c, bool touches_kv, bool* capturing) {
  gp_status st = need_device(c);
  if (st != GP_OK) return st;
  int dev = -1;
  GP_CUDA(c, cudaGetDevice(&dev));
  if (dev != c->device)
    return fail(c, GP_ERR_INVALID, "device %d is current, the engine was created on device %d", dev, c->device);
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  GP_CUDA(c, cudaStreamIsCapturing(c->stream, &cap));
  *capturing = cap != cudaStreamCaptureStatusNone;
  if (!touches_kv || !c->compaction_pending) return GP_OK;
  if (*capturing) return fail(c, GP_ERR_STATE, "a compaction is pending on the side stream: gp_synchronize before the capture");
  GP_CUDA(c, cudaStreamWaitEvent(c->stream, c->ev_done, 0));
  return GP_OK;
}

template <typename F>
gp_status launch_step(gp_ctx* c, bool capturing, int kernel, const char* name, F&& launch) {
  if (!capturing || c->inject_fail == kernel) return timed_launch(c, kernel, name, std::forward<F>(launch));
  const cudaError_t e = launch();  // a captured launch has no time of its own
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(c, GP_ERR_CUDA, "%s launch failed: %s", name, cudaGetErrorString(e));
  }
  return GP_OK;
}

StepArgs step_args(gp_ctx* c, const gp_step* s) {
  StepArgs a{};
  a.n = s->n;
  a.max_rows = s->max_rows;
  a.slots = s->slots;
  a.cached = s->num_cached;
  a.row0 = s->row0;
  a.row_req = s->row_req;
  a.tables = s->tables;
  a.M = c->cfg.max_slots;
  a.maxp = c->cfg.max_pages_per_req;
  a.num_pages_total = c->cfg.num_pages;
  a.err = c->err_dev;
  return a;
}

// The caches in boxes of a block's rows (64 of a larger block's).
bool block_maps(gp_ctx* c, int block, SparseMaps* maps) {
  const gp_config& g = c->cfg;
  const int i = block == 16 ? 0 : block == 32 ? 1 : 2;
  if (!c->block_maps_ok[i]) {
    const cuuint64_t dims[2] = {(cuuint64_t)g.head_dim, (cuuint64_t)g.num_layers * g.num_pages * g.num_kv_heads * kPage};
    const cuuint64_t strides[1] = {(cuuint64_t)g.head_dim * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)std::min(block, 64)};
    if (!encode_bf16_map(&c->block_maps[i][0], 2, c->k_cache, dims, strides, box) ||
        !encode_bf16_map(&c->block_maps[i][1], 2, c->v_cache, dims, strides, box))
      return false;
    c->block_maps_ok[i] = true;
  }
  maps->k = c->block_maps[i][0];
  maps->v = c->block_maps[i][1];
  return true;
}

// The scaled inverse frequencies of a rotary form (header), fp64.
void frequencies(const gp_rope& r, double* inv, float* amplitude) {
  const double two_pi = 6.283185307179586476925, rd = r.rotary_dim, L = r.original_length;
  const double high = r.high_turns != 0. ? r.high_turns : r.scaling == GP_ROPE_RAMP ? 32. : 4.;
  double from = 0., to = 0.;
  if (r.scaling == GP_ROPE_RAMP) {
    auto pair = [&](double turns) { return rd * std::log(L / (two_pi * turns)) / (2. * std::log(r.theta)); };
    from = std::fmax(0., std::floor(pair(high)));
    to = std::fmin(rd - 1., std::ceil(pair(r.low_turns)));
  }
  for (int i = 0; i < r.rotary_dim / 2; ++i) {
    const double f = std::pow(r.theta, -2. * i / rd);
    double part = 0.;  // of f / factor
    if (r.scaling == GP_ROPE_LINEAR) part = 1.;
    if (r.scaling == GP_ROPE_BANDS) part = 1. - std::fmin(1., std::fmax(0., (L * f / two_pi - r.low_turns) / (high - r.low_turns)));
    if (r.scaling == GP_ROPE_RAMP) part = std::fmin(1., std::fmax(0., (i - from) / std::fmax(to - from, 0.001)));
    inv[i] = part > 0. ? f * (1. - part) + f / r.factor * part : f;  // (the factor counts for nothing under NONE)
  }
  *amplitude = (float)(r.amplitude != 0. ? r.amplitude : r.scaling == GP_ROPE_RAMP ? 0.1 * std::log(r.factor) + 1. : 1.);
}

gp_status check_rope(gp_ctx* c, const gp_rope* r) {
  if (!r) return fail(c, GP_ERR_INVALID, "null rotary form");
  if (r->layout != GP_ROPE_HALF && r->layout != GP_ROPE_INTERLEAVED) return fail(c, GP_ERR_INVALID, "rotary layout %d", r->layout);
  if (r->rotary_dim < 0 || r->rotary_dim > c->cfg.head_dim || r->rotary_dim % 16)
    return fail(c, GP_ERR_INVALID, "rotary_dim %d: a multiple of 16 up to %d", r->rotary_dim, c->cfg.head_dim);
  if (r->scaling < GP_ROPE_NONE || r->scaling > GP_ROPE_RAMP) return fail(c, GP_ERR_INVALID, "rotary scaling %d", r->scaling);
  if (!(r->theta > 1.) || !std::isfinite(r->theta) || !std::isfinite(r->amplitude))
    return fail(c, GP_ERR_INVALID, "rotary theta %g, amplitude %g", r->theta, r->amplitude);
  if (r->scaling == GP_ROPE_NONE) return GP_OK;
  if (!(r->factor >= 1.) || !std::isfinite(r->factor)) return fail(c, GP_ERR_INVALID, "rotary factor %g", r->factor);
  if (r->scaling == GP_ROPE_LINEAR) return GP_OK;
  const double high = r->high_turns != 0. ? r->high_turns : r->scaling == GP_ROPE_RAMP ? 32. : 4.;
  if (r->original_length < 1 || !(r->low_turns > 0.) || !(high > r->low_turns) || !std::isfinite(high))
    return fail(c, GP_ERR_INVALID, "rotary original_length %d, turns %g to %g", r->original_length, r->low_turns, high);
  return GP_OK;
}

}  // namespace

gp_status gp_build_tables(gp_ctx* c, const gp_step* s, const int32_t* held_dev, int32_t* num_pages_dev, const int32_t* free_dev,
                          int32_t num_free, const int32_t* taken_in_dev, int32_t* taken_dev, int32_t* state_dev) try {
  if (!c) return GP_ERR_INVALID;
  gp_status st;
  const gp_config& g = c->cfg;
  if ((st = check_step(c, s)) != GP_OK) return st;
  if (g.max_slots > kStepMaxSlots) return fail(c, GP_ERR_UNSUPPORTED, "max_slots %d above %d", g.max_slots, kStepMaxSlots);
  if (num_free < 0 || (num_free > 0 && !free_dev)) return fail(c, GP_ERR_INVALID, "%d free pages, or no list of them", num_free);
  if (!held_dev || !num_pages_dev || !taken_dev || (s->n > 0 && !state_dev)) return fail(c, GP_ERR_INVALID, "null argument");
  for (const void* p : {(const void*)held_dev, (const void*)num_pages_dev, (const void*)free_dev, (const void*)taken_in_dev,
                        (const void*)taken_dev, (const void*)state_dev})
    if (off(p, 4)) return fail(c, GP_ERR_INVALID, "misaligned array");
  // what is written while others are read, or by other threads
  const size_t n = s->n, rows = s->max_rows, slots = g.max_slots;
  const Span in[] = {{s->slots, 4 * n},  {s->num_cached, 4 * n}, {s->num_new, 4 * n},         {s->pos, 8 * n},
                     {held_dev, 4 * slots}, {free_dev, 4 * (size_t)num_free}, {taken_in_dev, 4}};
  const Span out[] = {{s->tables, 4 * slots * g.max_pages_per_req}, {s->row0, 4 * (n + 1)}, {s->row_req, 4 * rows},
                      {s->slot_map, 8 * rows}, {s->positions, 8 * rows}, {state_dev, 4 * n},
                      {num_pages_dev, 4 * slots}, {taken_dev, 4}};
  for (const Span& o : out) {
    for (const Span& i : in)
      if (!apart(o, i) && !(o.p == i.p && ((o.p == num_pages_dev && i.p == held_dev) || (o.p == taken_dev && i.p == taken_in_dev))))
        return fail(c, GP_ERR_INVALID, "an output overlaps an input");
    for (const Span& p : out)
      if (&p != &o && !apart(o, p)) return fail(c, GP_ERR_INVALID, "two outputs overlap");
  }
  bool capturing = false;
  if ((st = ready_step(c, false, &capturing)) != GP_OK) return st;
  TablesArgs a{};
  a.n = s->n;
  a.max_rows = s->max_rows;
  a.num_free = num_free;
  a.M = g.max_slots;
  a.maxp = g.max_pages_per_req;
  a.num_pages_total = g.num_pages;
  a.slots = s->slots;
  a.cached = s->num_cached;
  a.fresh = s->num_new;
  a.pos = s->pos;
  a.held = held_dev;
  a.free_pages = free_dev;
  a.taken_in = taken_in_dev;
  a.tables = s->tables;
  a.num_pages = num_pages_dev;
  a.row0 = s->row0;
  a.row_req = s->row_req;
  a.state = state_dev;
  a.taken = taken_dev;
  a.slot_map = s->slot_map;
  a.positions = s->positions;
  a.err = c->err_dev;
  a.apart = num_pages_dev != held_dev && taken_dev != taken_in_dev;
  return launch_step(c, capturing, GP_KERNEL_TABLES, "build_tables", [&] { return launch_tables(a, c->stream); });
} catch (const std::exception&) {
  return no_memory(c);
}

gp_status gp_rope_default(gp_rope* r) {
  if (!r) return GP_ERR_INVALID;
  *r = gp_rope{};
  r->layout = GP_ROPE_HALF;
  r->scaling = GP_ROPE_NONE;
  r->original_length = 8192;
  r->theta = 10000.;
  r->factor = 1.;
  r->low_turns = 1.;
  return GP_OK;
}

gp_status gp_append_mapped(gp_ctx* c, int32_t layer, const gp_step* s, const gp_rope* rope, const void* q_dev, int64_t q_stride,
                           const void* k_dev, int64_t k_stride, const void* v_dev, int64_t v_stride, void* q_rot_dev) try {
  if (!c) return GP_ERR_INVALID;
  gp_status st;
  const gp_config& g = c->cfg;
  if ((st = check_step(c, s)) != GP_OK || (st = check_layer(c, layer, 16)) != GP_OK || (st = check_rope(c, rope)) != GP_OK) return st;
  bool capturing = false;
  if (s->max_rows == 0) return ready_step(c, false, &capturing);
  if (!k_dev || !v_dev || (q_dev == nullptr) != (q_rot_dev == nullptr))
    return fail(c, GP_ERR_INVALID, "null keys or values, or only one of q and q_rot");
  const int64_t qe = elt_bytes(g.q_dtype), ke = elt_bytes(g.kv_dtype), rows = s->max_rows;
  const int64_t q_row = (int64_t)g.num_q_heads * g.head_dim, kv_row = (int64_t)g.num_kv_heads * g.head_dim;
  auto bad = [&](int64_t stride, int64_t row, int64_t e) { return stride < row || stride > (1ll << 40) || stride * e % 16 != 0; };
  if ((q_dev && bad(q_stride, q_row, qe)) || bad(k_stride, kv_row, ke) || bad(v_stride, kv_row, ke))
    return fail(c, GP_ERR_INVALID, "row strides %lld, %lld, %lld: at least a row, whole 16 bytes", (long long)q_stride,
                (long long)k_stride, (long long)v_stride);
  for (const void* p : {q_dev, k_dev, v_dev, (const void*)q_rot_dev, (const void*)c->k_cache, (const void*)c->v_cache})
    if (off(p, 16)) return fail(c, GP_ERR_INVALID, "queries, keys, values and caches must be 16-byte aligned");
  const Span rot{q_rot_dev, (size_t)(rows * q_row * qe)};
  const Span q{q_dev, (size_t)(((rows - 1) * q_stride + q_row) * qe)}, k{k_dev, (size_t)(((rows - 1) * k_stride + kv_row) * ke)},
      v{v_dev, (size_t)(((rows - 1) * v_stride + kv_row) * ke)};
  if (!apart(rot, k) || !apart(rot, v) || (!apart(rot, q) && !(q_dev == q_rot_dev && q_stride == q_row)))
    return fail(c, GP_ERR_INVALID, "q_rot overlaps an input without being a packed q");
  if ((st = ready_step(c, true, &capturing)) != GP_OK) return st;
  MappedArgs a{};
  a.rows = s->max_rows;
  a.slot_map = s->slot_map;
  a.positions = s->positions;
  a.k_cache = c->k_cache;
  a.v_cache = c->v_cache;
  a.kv_f32 = g.kv_dtype == GP_DTYPE_F32;
  a.q_f32 = g.q_dtype == GP_DTYPE_F32;
  a.num_pages_total = g.num_pages;
  a.layer = layer;
  a.Hq = g.num_q_heads;
  a.Hkv = g.num_kv_heads;
  a.D = g.head_dim;
  a.q = q_dev;
  a.k = k_dev;
  a.v = v_dev;
  a.q_row = q_stride;
  a.k_row = k_stride;
  a.v_row = v_stride;
  a.q_rot = q_rot_dev;
  a.rotary_dim = rope->rotary_dim;
  a.interleaved = rope->layout == GP_ROPE_INTERLEAVED;
  a.err = c->err_dev;
  if (c->rope.theta == 0. || std::memcmp(&c->rope, rope, sizeof(gp_rope)) != 0) {  // (theta is above 1)
    frequencies(*rope, c->rope_inv, &c->rope_amplitude);
    c->rope = *rope;
  }
  std::memcpy(a.inv_freq, c->rope_inv, sizeof(a.inv_freq));
  a.amplitude = c->rope_amplitude;
  st = launch_step(c, capturing, GP_KERNEL_MAPPED, "append_mapped", [&] { return launch_mapped(a, c->stream); });
  if (st != GP_OK) return st;
  for (auto& gen : c->slot_gen) ++gen;  // demand results over the old rows are stale; whose, only the device knows
  return GP_OK;
} catch (const std::exception&) {
  return no_memory(c);
}

gp_status gp_block_bounds(gp_ctx* c, int32_t layer, const gp_step* s, int32_t block, int8_t* bounds_dev, float* scales_dev) try {
  if (!c) return GP_ERR_INVALID;
  gp_status st;
  if ((st = check_step(c, s)) != GP_OK || (st = check_layer(c, layer, block)) != GP_OK) return st;
  bool capturing = false;
  if (s->max_rows == 0 || s->n == 0) return ready_step(c, false, &capturing);
  if (!bounds_dev || !scales_dev) return fail(c, GP_ERR_INVALID, "null argument");
  if (off(bounds_dev, 16) || off(scales_dev, 4) || off(c->k_cache, 16))
    return fail(c, GP_ERR_INVALID, "bounds and keys must be 16-byte aligned, scales 4-byte");
  if ((st = ready_step(c, true, &capturing)) != GP_OK) return st;
  BoundsArgs a{};
  a.s = step_args(c, s);
  a.k_cache = c->k_cache;
  a.kv_f32 = c->cfg.kv_dtype == GP_DTYPE_F32;
  a.layer = layer;
  a.Hkv = c->cfg.num_kv_heads;
  a.D = c->cfg.head_dim;
  a.block = block;
  a.bounds = bounds_dev;
  a.scales = scales_dev;
  return launch_step(c, capturing, GP_KERNEL_BOUNDS, "block_bounds", [&] { return launch_bounds(a, c->stream); });
} catch (const std::exception&) {
  return no_memory(c);
}

gp_status gp_select_blocks(gp_ctx* c, int32_t layer, const gp_step* s, int32_t block, int32_t top, int32_t sink, int32_t recent,
                           const void* q_rot_dev, const int8_t* bounds_dev, const float* scales_dev, int32_t* blocks_dev) try {
  if (!c) return GP_ERR_INVALID;
  gp_status st;
  const gp_config& g = c->cfg;
  if ((st = check_step(c, s)) != GP_OK || (st = check_layer(c, layer, block)) != GP_OK) return st;
  if (sink < 0 || recent < 1 || top > (1 << 16) || (int64_t)sink + recent > top)
    return fail(c, GP_ERR_INVALID, "%d blocks, %d first and %d last: 0 <= sink, 1 <= recent, sink + recent <= top <= 65536", top, sink,
                recent);
  bool capturing = false;
  if (s->max_rows == 0 || s->n == 0) return ready_step(c, false, &capturing);
  if (!q_rot_dev || !bounds_dev || !scales_dev || !blocks_dev) return fail(c, GP_ERR_INVALID, "null argument");
  if (off(q_rot_dev, 16) || off(bounds_dev, 16) || off(scales_dev, 4) || off(blocks_dev, 4))
    return fail(c, GP_ERR_INVALID, "queries and bounds must be 16-byte aligned, scales and blocks 4-byte");
  if ((st = ready_step(c, false, &capturing)) != GP_OK) return st;
  SelectBlocksArgs a{};
  a.s = step_args(c, s);
  a.layer = layer;
  a.Hq = g.num_q_heads;
  a.Hkv = g.num_kv_heads;
  a.D = g.head_dim;
  a.q_f32 = g.q_dtype == GP_DTYPE_F32;
  a.block = block;
  a.top = top;
  a.sink = sink;
  a.recent = recent;
  a.q = q_rot_dev;
  a.bounds = bounds_dev;
  a.scales = scales_dev;
  a.blocks = blocks_dev;
  const int blocks = g.max_pages_per_req * (kPage / block);
  a.rows = s->max_rows > 8 * (int64_t)s->n && 16 * 4 * blocks <= kSelectShared ? 16 : 8;
  const int64_t tiles = std::min<int64_t>(sparse_pieces(a.s, a.rows), s->max_rows) * g.num_kv_heads;
  a.splits = 1;
  // Clusters share the blocks of tiles of 8 rows while all of their CTAs find a place at once
  // (four an SM: scores of up to 1600 blocks a row; of 4096, 256 pages in blocks of 16, one)
  // and each has 64 blocks.  Decode steps of 4, 16, 32 and 64 requests of up to 125
  // pages: 11.5, 12.4, 13.0 and 14.5 us without, 8.7, 9.5, 11.3 and 17.8 us shared by 4, 4, 2 and 2.
  // Tiles of 16 rows have work enough for a CTA: 300 rows 10.8 us, shared by two 13.8.
  while (a.rows == 8 && a.splits < 8 && (a.splits + 1) * tiles <= 4 * c->sms && blocks >= 64 * (a.splits + 1)) ++a.splits;
  return launch_step(c, capturing, GP_KERNEL_BLOCK_SELECT, "select_blocks", [&] { return launch_select_blocks(a, c->stream); });
} catch (const std::exception&) {
  return no_memory(c);
}

gp_status gp_sparse_attention(gp_ctx* c, int32_t layer, const gp_step* s, int32_t block, int32_t top, const void* q_rot_dev,
                              const int32_t* blocks_dev, void* out_dev) try {
  if (!c) return GP_ERR_INVALID;
  gp_status st;
  const gp_config& g = c->cfg;
  if ((st = check_step(c, s)) != GP_OK || (st = check_layer(c, layer, block)) != GP_OK) return st;
  if (top < 1 || top > (1 << 16)) return fail(c, GP_ERR_INVALID, "%d blocks: 1 to 65536", top);
  bool capturing = false;
  if (s->max_rows == 0 || s->n == 0) return ready_step(c, false, &capturing);
  if (!q_rot_dev || !blocks_dev || !out_dev) return fail(c, GP_ERR_INVALID, "null argument");
  if (off(q_rot_dev, 16) || off(out_dev, 16) || off(blocks_dev, 4) || off(c->k_cache, 16) || off(c->v_cache, 16))
    return fail(c, GP_ERR_INVALID, "queries, outputs and caches must be 16-byte aligned, blocks 4-byte");
  const size_t bytes = (size_t)s->max_rows * g.num_q_heads * g.head_dim * elt_bytes(g.q_dtype);
  if (!apart({q_rot_dev, bytes}, {out_dev, bytes}) || !apart({blocks_dev, 4 * (size_t)s->max_rows * g.num_kv_heads * top}, {out_dev, bytes}))
    return fail(c, GP_ERR_INVALID, "the outputs overlap an input");
  if ((st = ready_step(c, true, &capturing)) != GP_OK) return st;
  SparseArgs a{};
  a.s = step_args(c, s);
  a.k_cache = c->k_cache;
  a.v_cache = c->v_cache;
  a.kv_f32 = g.kv_dtype == GP_DTYPE_F32;
  a.q_f32 = g.q_dtype == GP_DTYPE_F32;
  a.layer = layer;
  a.Hq = g.num_q_heads;
  a.Hkv = g.num_kv_heads;
  a.D = g.head_dim;
  a.block = block;
  a.top = top;
  a.q = q_rot_dev;
  a.blocks = blocks_dev;
  a.out = out_dev;
  a.wait_limit = c->wait_limit_sparse;
  const bool tc = c->attn_tc_ok && c->scan_kernel != GP_SCAN_CUDA_CORE && g.q_dtype == GP_DTYPE_BF16;
  if (c->scan_kernel == GP_SCAN_TENSOR_CORE && !tc)
    return fail(c, GP_ERR_UNSUPPORTED, "the tensor-core kernels cannot take this cache or query type");
  // Clusters share the blocks of a piece while all of their CTAs find a place at once
  // (two an SM: shared memory has room for two of up to 115 KB, bitmaps and lists by
  // max_pages_per_req among them; above that, d = 128 with blocks of 16 or 32 and long
  // tables, one) and a share keeps 64 tokens.  One long request, 64 blocks of 64: 46, 28, 19 and
  // 14.7 us at 1, 2, 4 and 8; 16 requests 31, 29, 37 and 52; 64 requests 90, 104, 120 and 175.
  const int64_t tokens = (int64_t)std::min(top, g.max_pages_per_req * (kPage / block)) * block;
  auto share = [&](int64_t pieces, int most) {
    pieces = std::min<int64_t>(pieces, s->max_rows);
    a.splits = 1;
    while (a.splits < most && (a.splits + 1) * pieces * g.num_kv_heads <= 2 * c->sms && tokens >= 64 * (a.splits + 1)) ++a.splits;
  };
  if (!tc) {
    share(s->max_rows, 8);
    return launch_step(c, capturing, GP_KERNEL_SPARSE, "sparse_attention", [&] { return launch_sparse(a, c->stream); });
  }
  SparseMaps maps;
  if (!block_maps(c, block, &maps)) return fail(c, GP_ERR_CUDA, "no tensor map of the caches");
  // A row or two of each request at a time, or pieces of 128 / G rows: those from
  // where a request has more rows than the small pieces take in one (4 rows of one, 8
  // and 64 requests with G = 4: 15.2 us on either, 31 and 47, 125 on either; 8 rows: 31 instead
  // of 47 and 137 instead of 177; 4001 rows: 320 instead of 1094).
  const int G = g.num_q_heads / g.num_kv_heads;
  const bool many = s->max_rows > (int64_t)s->n * kSparseMmaRows / G;
  share(sparse_pieces(a.s, (many ? kSparseTcRows : kSparseMmaRows) / G), many ? 8 : 16);
  CUtensorMap qmap;
  if (many) {
    const cuuint64_t row = (cuuint64_t)g.head_dim * 2;
    const cuuint64_t dims[3] = {(cuuint64_t)g.head_dim, (cuuint64_t)g.num_q_heads, (cuuint64_t)s->max_rows};
    const cuuint64_t strides[2] = {row, row * g.num_q_heads};
    const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(kSparseTcRows / G)};
    if (!encode_bf16_map(&qmap, 3, q_rot_dev, dims, strides, box)) return fail(c, GP_ERR_CUDA, "no tensor map of the queries");
  }
  return launch_step(c, capturing, GP_KERNEL_SPARSE, "sparse_attention",
                     [&] { return many ? launch_sparse_tc(a, maps, qmap, c->stream) : launch_sparse_mma(a, maps, c->stream); });
} catch (const std::exception&) {
  return no_memory(c);
}
