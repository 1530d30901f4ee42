// The engine context and what every translation unit of the host side needs
// of it: status texts, growing buffers, event-timed launches, the waits for
// work on other streams, and the validation of requests.  growpage.cpp holds
// the boundary engine, weighted.cpp the attention that accumulates weights and
// the eviction by them.
#pragma once

#include "growpage.h"

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <exception>
#include <set>
#include <string>
#include <unordered_set>
#include <utility>
#include <vector>

#include "gp_kernels.h"
#include "gp_internal.h"

namespace gp {

constexpr int kPage = 256;
constexpr int kMaxPagesPerReq = 256;

struct DevBuf {
  void* p = nullptr;
  size_t cap = 0;
};

struct DemandRec {
  int32_t slot = -1;
  int32_t num_pages = 0;
  std::vector<int32_t> pages;
  uint64_t gen = 0;
  int64_t score_off = 0;
  int64_t aval_off = 0;
  int64_t spec_off = -1;  // word offset of its speculative keep masks, -1 if none
};

struct CompressRec {
  bool spec = false;      // masks in the speculative buffer (at mask_off), else in `masks`
  int32_t num_pages = 0;
  int64_t mask_off = 0;
  // gp_evict_weighted: lists of kept slots instead of masks, at mask_off
  bool evict = false;
  int32_t tokens = 0, kept = 0, pitch = 0;  // kept 0: all of the tokens
};

// A call's descriptors on their way to the device: pinned memory, its device
// mirror (pieces of the engine's), and the event after which both may be written
// again.
struct StagingSlot {
  void* pinned = nullptr;
  DevBuf dev;
  cudaEvent_t free = nullptr;
};
constexpr int kStagingSlots = 8;

struct TimedEvent {
  int kernel;
  cudaEvent_t start, stop;
};


}  // namespace gp

struct gp_ctx {
  gp_config cfg{};
  bool host_only = true;
  void* k_cache = nullptr;
  void* v_cache = nullptr;
  cudaStream_t stream = nullptr;
  std::string err;

  // page pool (Sec. 4.2, App. E.2)
  std::vector<int32_t> refcnt;
  std::vector<uint32_t> page_seen;  // per page: the last block table check that met it
  uint32_t check = 0;               // number of that check
  std::set<int32_t> free_pages;
  // summary slots (App. E.1)
  std::vector<uint8_t> slot_bound;
  std::vector<uint64_t> slot_gen;
  std::set<int32_t> free_slots;

  // device state
  double* pool = nullptr;          // [L][M][2][Hq][D]
  int* err_dev = nullptr;          // kernel error bits
  unsigned long long* moved_dev = nullptr;
  gp::DevBuf upload, bt2, qt, bq, scores, aval, tickets, kout, ksum, masks, xstat, attn, spec_masks, ent;
  // decode attention and the accumulated-weight operators: descriptor staging
  // (calls in turn, so that a call waits on the host only for the one
  // kStagingSlots before it, and none disturbs a compaction's) and scratch
  gp::StagingSlot staging[gp::kStagingSlots];
  int staging_next = 0;
  void* staging_pinned = nullptr;  // of all slots
  gp::DevBuf staging_dev;
  size_t staging_cap = 0;          // bytes of a slot
  gp::DevBuf logits, wstat, evict, chunk;
  int device = 0;                  // the device current at gp_create
  // speculative selection: the Eq. 10 keep masks of every request of the last
  // demand call, computed on an engine-owned stream while the host decides
  cudaStream_t sel_stream = nullptr;
  cudaEvent_t ev_dem = nullptr, ev_sel = nullptr;
  bool sel_pending = false;
  double* inv_freq = nullptr;      // [D/2] theta^(-2i/D) for RoPE
  CUtensorMap kmap;                // K cache as a 2-D bf16 tensor (tensor-core scan and attention)
  CUtensorMap vmap;                // V cache the same way (tensor-core attention)
  bool tc_ok = false;              // kmap is valid
  bool attn_tc_ok = false;         // kmap and vmap are valid
  int sms = 152;                   // SMs of the device
  int scan_kernel = GP_SCAN_AUTO;
  int select_mode = GP_SELECT_AUTO;
  int64_t spec_units_max = 4 * 152;  // AUTO: speculative selection up to this many units per call
  void* pinned = nullptr;
  size_t pinned_cap = 0;
  cudaEvent_t pinned_free = nullptr;  // recorded after the last async use of `pinned`
  void* readback = nullptr;           // pinned: a demand call's sums and error word
  size_t readback_cap = 0;
  // asynchronous compaction: a side stream, the event the side stream waits
  // for (engine stream state), and the event of the last compaction there
  cudaStream_t cstream = nullptr;
  cudaEvent_t ev_ready = nullptr, ev_done = nullptr;
  bool compaction_pending = false;
  std::unordered_set<int32_t> pending_pages;  // old and new pages of the pending compaction
  std::unordered_set<int32_t> pending_slots;  // slots whose accumulated weights it moves

  std::vector<gp::DemandRec> last_demand;
  std::vector<gp::CompressRec> last_compress;

  gp_stats_t stats{};
  int64_t decisions = 0;           // decisions taken so far (index of the RANDOM policy's draws)
  bool timing = false;
  std::vector<gp::TimedEvent> timed;
  std::vector<cudaEvent_t> event_pool;
  double t_ms[GP_KERNEL_COUNT] = {};
  int64_t t_count[GP_KERNEL_COUNT] = {};
  // test hooks: the copy-wait limit of the selection / compaction launches,
  // and a launch to fail without running (-1: none)
  long long wait_limit_select = gp::kDefaultWaitLimit;
  long long wait_limit_compress = gp::kDefaultWaitLimit;
  long long wait_limit_evict = gp::kDefaultWaitLimit;
  long long wait_limit_chunk = gp::kDefaultWaitLimit;
  long long wait_limit_weights = gp::kDefaultWaitLimit;
  int inject_fail = -1;
};

namespace gp {

inline gp_status fail(gp_ctx* c, gp_status st, const char* fmt, ...) {
  if (c) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    c->err = buf;
  }
  return st;
}

// What an entry point returns for an exception, none of which leaves it: the only
// ones are of allocations, all of which come before the call changes anything.
inline gp_status no_memory(gp_ctx* c) {
  try {
    return fail(c, GP_ERR_CUDA, "out of host memory");
  } catch (const std::exception&) {
    if (c) c->err.clear();
    return GP_ERR_CUDA;
  }
}

#define GP_CUDA(ctx, call)                                                              \
  do {                                                                                  \
    cudaError_t e_ = (call);                                                            \
    if (e_ != cudaSuccess) {                                                            \
      cudaGetLastError(); /* else the next launch's check would meet it again */        \
      return fail((ctx), GP_ERR_CUDA, "%s failed: %s", #call, cudaGetErrorString(e_)); \
    }                                                                                   \
  } while (0)

inline int elt_bytes(int dtype) { return dtype == GP_DTYPE_F32 ? 4 : 2; }

inline gp_status ensure(gp_ctx* c, DevBuf& b, size_t bytes) {
  if (bytes <= b.cap) return GP_OK;
  size_t cap = std::max(bytes, b.cap + b.cap / 2);
  cap = (cap + 255) & ~size_t(255);
  if (b.p) GP_CUDA(c, cudaFree(b.p));
  b.p = nullptr;
  b.cap = 0;
  GP_CUDA(c, cudaMalloc(&b.p, cap));
  b.cap = cap;
  return GP_OK;
}

inline gp_status ensure_pinned(gp_ctx* c, size_t bytes) {
  if (c->pinned_free) GP_CUDA(c, cudaEventSynchronize(c->pinned_free));
  if (bytes <= c->pinned_cap) return GP_OK;
  size_t cap = std::max(bytes, c->pinned_cap * 2);
  cap = (cap + 4095) & ~size_t(4095);
  if (c->pinned) GP_CUDA(c, cudaFreeHost(c->pinned));
  c->pinned = nullptr;
  c->pinned_cap = 0;
  GP_CUDA(c, cudaHostAlloc(&c->pinned, cap, cudaHostAllocDefault));
  c->pinned_cap = cap;
  return GP_OK;
}

// The pinned readback buffer; a demand call reads it only after
// synchronising the stream, so no copy into it is still in flight here.
inline gp_status ensure_readback(gp_ctx* c, size_t bytes) {
  if (bytes <= c->readback_cap) return GP_OK;
  size_t cap = std::max<size_t>(std::max(bytes, c->readback_cap * 2), 4096);
  cap = (cap + 4095) & ~size_t(4095);
  if (c->readback) GP_CUDA(c, cudaFreeHost(c->readback));
  c->readback = nullptr;
  c->readback_cap = 0;
  GP_CUDA(c, cudaHostAlloc(&c->readback, cap, cudaHostAllocDefault));
  c->readback_cap = cap;
  return GP_OK;
}

inline cudaEvent_t take_event(gp_ctx* c) {
  if (!c->event_pool.empty()) {
    cudaEvent_t e = c->event_pool.back();
    c->event_pool.pop_back();
    return e;
  }
  cudaEvent_t e = nullptr;
  cudaEventCreate(&e);
  return e;
}

// Launch wrapper: brackets the launch with events when timing is on.
template <typename F>
gp_status timed_launch_on(gp_ctx* c, cudaStream_t s, int kernel, const char* name, F&& launch) {
  if (c->inject_fail == kernel) {  // test hook: fail as a launch failure would, without running
    c->inject_fail = -1;
    return fail(c, GP_ERR_CUDA, "%s launch failed: injected failure (test hook)", name);
  }
  cudaEvent_t a = nullptr, b = nullptr;
  if (c->timing) {
    if (c->timed.size() == c->timed.capacity()) c->timed.reserve(2 * c->timed.size() + 16);
    a = take_event(c);
    b = take_event(c);
    cudaEventRecord(a, s);
  }
  cudaError_t e = launch();
  if (e != cudaSuccess) return fail(c, GP_ERR_CUDA, "%s launch failed: %s", name, cudaGetErrorString(e));
  if (c->timing) {
    cudaEventRecord(b, s);
    c->timed.push_back({kernel, a, b});  // (room made above)
  }
  return GP_OK;
}

template <typename F>
gp_status timed_launch(gp_ctx* c, int kernel, const char* name, F&& launch) {
  return timed_launch_on(c, c->stream, kernel, name, std::forward<F>(launch));
}

// Waits (host) for a speculative selection still running: it reads the
// importance cache and writes the speculative masks, which the next demand
// call rewrites.
inline gp_status join_select(gp_ctx* c) {
  if (c->sel_pending) {
    GP_CUDA(c, cudaEventSynchronize(c->ev_sel));
    c->sel_pending = false;
  }
  return GP_OK;
}

// Waits (host) for a compaction still running on the side stream: its K/V
// writes, its reads of the engine's scratch (tables, importance, masks) and
// its statistics must be done before the engine reuses, regrows or reads
// any of them.
inline gp_status join_compaction(gp_ctx* c) {
  if (c->compaction_pending) {
    GP_CUDA(c, cudaEventSynchronize(c->ev_done));
    c->compaction_pending = false;
    c->pending_pages.clear();
    c->pending_slots.clear();
  }
  return GP_OK;
}

inline gp_status need_device(gp_ctx* c) {
  if (!c) return GP_ERR_INVALID;
  if (c->host_only) return fail(c, GP_ERR_STATE, "host-only context has no device caches");
  return GP_OK;
}

// Refuses a call while a stream of the engine is being captured: its descriptors
// are host data of the call, and a replay would copy whatever their memory holds by
// then.
inline gp_status refuse_capture(gp_ctx* c) {
  for (cudaStream_t s : {c->stream, c->cstream ? c->cstream : c->stream}) {
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    GP_CUDA(c, cudaStreamIsCapturing(s, &cap));
    if (cap != cudaStreamCaptureStatusNone)
      return fail(c, GP_ERR_UNSUPPORTED, "a stream of the engine is being captured: the call reads host data at every launch");
  }
  return GP_OK;
}

// What the accumulated-weight operators check first: that, and that their launches
// go to the engine's device.
inline gp_status ready_call(gp_ctx* c) {
  gp_status st = need_device(c);
  if (st != GP_OK) return st;
  int dev = -1;
  GP_CUDA(c, cudaGetDevice(&dev));
  if (dev != c->device)
    return fail(c, GP_ERR_INVALID, "device %d is current, the engine was created on device %d", dev, c->device);
  return refuse_capture(c);
}

// A staging slot of at least `bytes`, free to be written.  The slots are pieces
// of one allocation, made at the first call and again when a call needs more than
// any before it: a call that is not the largest so far allocates nothing.
inline gp_status staging_take(gp_ctx* c, size_t bytes, StagingSlot** out) {
  if (bytes > c->staging_cap) {
    for (StagingSlot& s : c->staging) {
      if (!s.free) GP_CUDA(c, cudaEventCreateWithFlags(&s.free, cudaEventDisableTiming));
      GP_CUDA(c, cudaEventSynchronize(s.free));  // its copy has read the pinned memory
    }
    const size_t cap = (std::max(bytes, 2 * c->staging_cap) + 65535) & ~size_t(65535);
    c->staging_cap = 0;
    if (c->staging_pinned) {
      void* old = std::exchange(c->staging_pinned, nullptr);
      GP_CUDA(c, cudaFreeHost(old));
    }
    GP_CUDA(c, cudaHostAlloc(&c->staging_pinned, kStagingSlots * cap, cudaHostAllocDefault));
    const gp_status st = ensure(c, c->staging_dev, kStagingSlots * cap);  // (a cudaFree waits for the kernels that read it)
    if (st != GP_OK) return st;
    for (int i = 0; i < kStagingSlots; ++i) {
      c->staging[i].pinned = static_cast<char*>(c->staging_pinned) + i * cap;
      c->staging[i].dev.p = static_cast<char*>(c->staging_dev.p) + i * cap;
    }
    c->staging_cap = cap;
  }
  StagingSlot& s = c->staging[c->staging_next];
  GP_CUDA(c, cudaEventSynchronize(s.free));
  c->staging_next = (c->staging_next + 1) % kStagingSlots;
  *out = &s;
  return GP_OK;
}

inline gp_status staging_upload(gp_ctx* c, StagingSlot& s, size_t bytes) {
  GP_CUDA(c, cudaMemcpyAsync(s.dev.p, s.pinned, bytes, cudaMemcpyHostToDevice, c->stream));
  GP_CUDA(c, cudaEventRecord(s.free, c->stream));
  return GP_OK;
}

// The engine stream waits for a compaction pending on the side stream if a
// request holds a page it reads or writes (App. E.3), or a slot whose weights it
// moves: the slot of a finished request may be another's by now, on other pages.
inline gp_status wait_pending(gp_ctx* c, int n, const gp_request* reqs) {
  if (!c->compaction_pending) return GP_OK;
  bool shared = false;
  for (int r = 0; r < n && !shared; ++r) {
    shared = c->pending_slots.count(reqs[r].slot) != 0;
    for (int j = 0; j < reqs[r].num_pages && !shared; ++j) shared = c->pending_pages.count(reqs[r].block_table[j]) != 0;
  }
  if (shared) GP_CUDA(c, cudaStreamWaitEvent(c->stream, c->ev_done, 0));
  return GP_OK;
}

// Read and clear the kernels' error word (synchronises the stream).  A word
// holding only ERR_TIMEOUT (bounded waits gave up) is GP_ERR_TIMEOUT; any
// failed device-side check makes it GP_ERR_INVALID.
inline gp_status kernel_error_status(gp_ctx* c, int e);

inline gp_status check_kernel_errors(gp_ctx* c) {
  int e = 0;
  GP_CUDA(c, cudaMemcpyAsync(&e, c->err_dev, sizeof(int), cudaMemcpyDeviceToHost, c->stream));
  GP_CUDA(c, cudaStreamSynchronize(c->stream));
  return kernel_error_status(c, e);
}

// The status of an error word already read (the stream synchronised); a
// non-zero word is cleared on the device.
inline gp_status kernel_error_status(gp_ctx* c, int e) {
  if (e) {
    GP_CUDA(c, cudaMemsetAsync(c->err_dev, 0, sizeof(int), c->stream));
    GP_CUDA(c, cudaStreamSynchronize(c->stream));
    return fail(c, gp::status_of_kernel_error(e),
                "device-side error (bits 0x%x: 1 slot, 2 page, 4 keep mask count, 8 selection, 16 wait timed out)",
                e);
  }
  return GP_OK;
}

// Starts a check that marks pages as it meets them (page_seen == check).
inline void begin_page_check(gp_ctx* c) {
  if (c->page_seen.size() != c->refcnt.size() || ++c->check == 0) {
    c->page_seen.assign(c->refcnt.size(), 0);
    c->check = 1;
  }
}

inline gp_status validate_request(gp_ctx* c, const gp_request& r, int idx, bool need_slot) {
  const gp_config& g = c->cfg;
  if (need_slot && (r.slot < 0 || r.slot >= g.max_slots || !c->slot_bound[r.slot]))
    return fail(c, GP_ERR_INVALID, "request %d: slot %d is not bound", idx, r.slot);
  if (r.num_pages < 1 || r.num_pages > g.max_pages_per_req)
    return fail(c, GP_ERR_INVALID, "request %d: num_pages %d outside [1, %d]", idx, r.num_pages,
                g.max_pages_per_req);
  if (!r.block_table) return fail(c, GP_ERR_INVALID, "request %d: null block table", idx);
  if (r.pos < 0) return fail(c, GP_ERR_INVALID, "request %d: negative position", idx);
  // a page is marked with the number of the check that meets it: no set to build
  begin_page_check(c);
  for (int j = 0; j < r.num_pages; ++j) {
    const int32_t pg = r.block_table[j];
    if (pg < 0 || pg >= g.num_pages || c->refcnt[pg] <= 0)
      return fail(c, GP_ERR_INVALID, "request %d: block %d holds page %d that is not allocated", idx, j, pg);
    if (std::exchange(c->page_seen[pg], c->check) == c->check)
      return fail(c, GP_ERR_INVALID, "request %d: page %d appears twice in the block table", idx, pg);
  }
  return GP_OK;
}

// A tiled bf16 tensor map with the 128-byte swizzle; false if it cannot be made.
inline bool encode_bf16_map(CUtensorMap* map, uint32_t rank, const void* base, const cuuint64_t* dims,
                            const cuuint64_t* strides, const cuuint32_t* box) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q{};
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
                        cudaSuccess && q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn) : nullptr;
  }();
  const cuuint32_t ones[3] = {1, 1, 1};
  return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box,
                          ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int units_of(const gp_ctx* c) { return c->cfg.num_layers * c->cfg.num_kv_heads; }

}  // namespace gp
