// A CUDA runtime without a device, for tests of the host side on the CPU: device
// memory is host memory, a copy happens at once, streams and events do nothing,
// kernels are counted and not run.  The named call fails when a test asks for it.
// Linked with the library's own host objects in place of the runtime and kernels.
#include <cuda_runtime.h>

#include <cstdlib>
#include <cstring>
#include <map>
#include <new>
#include <string>
#include <utility>

#include "attn_kernels.h"
#include "gp_internal.h"
#include "gp_kernels.h"
#include "weighted_kernels.h"

namespace {
std::map<std::string, long> calls, fail_at;
std::map<void*, size_t> sizes;
int skip_select = 0;
long news = 0, news_until_failure = -1;  // -1: none fails
// counts the call; an error when it is the one that is to fail
cudaError_t called(const char* name) {
  const struct Own {  // the runtime's own allocations do not fail
    long held = std::exchange(news_until_failure, -1);
    ~Own() { news_until_failure = held; }
  } own;
  const long n = ++calls[name];
  const auto it = fail_at.find(name);
  return it != fail_at.end() && it->second == n ? cudaErrorMemoryAllocation : cudaSuccess;
}
cudaError_t take(const char* name, void** p, size_t n) {
  if (called(name) != cudaSuccess) return cudaErrorMemoryAllocation;
  *p = std::malloc(n ? n : 1);
  std::memset(*p, 0xff, n);  // what a kernel leaves unwritten is recognised
  const long held = std::exchange(news_until_failure, -1);
  sizes[*p] = n;
  news_until_failure = held;
  return cudaSuccess;
}
cudaError_t give(const char* name, void* p) {  // the block stays, so that a late use of it does not end the process
  if (called(name) != cudaSuccess) return cudaErrorMemoryAllocation;
  if (p) std::memset(p, 0xff, sizes[p]);
  return cudaSuccess;
}
}  // namespace

extern "C" {
long fake_calls(const char* name) { return calls[name]; }
void fake_fail(const char* name, long after) { fail_at[name] = calls[name] + after; }  // the after-th call from now
void fake_reset() {
  calls.clear();
  fail_at.clear();
  skip_select = 0;
  news_until_failure = -1;
}
void fake_fail_new(long after) { news_until_failure = after; }  // the after-th allocation from now, -1: none
void fake_skip_select(int yes) { skip_select = yes; }

cudaError_t cudaMalloc(void** p, size_t n) { return take("cudaMalloc", p, n); }
cudaError_t cudaHostAlloc(void** p, size_t n, unsigned) { return take("cudaHostAlloc", p, n); }
cudaError_t cudaFree(void* p) { return give("cudaFree", p); }
cudaError_t cudaFreeHost(void* p) { return give("cudaFreeHost", p); }
cudaError_t cudaMemcpyAsync(void* to, const void* from, size_t n, cudaMemcpyKind, cudaStream_t) {
  if (called("cudaMemcpyAsync") != cudaSuccess) return cudaErrorMemoryAllocation;
  std::memcpy(to, from, n);
  return cudaSuccess;
}
cudaError_t cudaMemcpy2DAsync(void* to, size_t tp, const void* from, size_t fp, size_t w, size_t h, cudaMemcpyKind, cudaStream_t) {
  for (size_t i = 0; i < h; ++i) std::memcpy(static_cast<char*>(to) + i * tp, static_cast<const char*>(from) + i * fp, w);
  return called("cudaMemcpy2DAsync");
}
cudaError_t cudaMemsetAsync(void* p, int v, size_t n, cudaStream_t) {
  std::memset(p, v, n);
  return called("cudaMemsetAsync");
}
cudaError_t cudaEventCreate(cudaEvent_t* e) { return cudaEventCreateWithFlags(e, 0); }
cudaError_t cudaEventCreateWithFlags(cudaEvent_t* e, unsigned) {
  *e = reinterpret_cast<cudaEvent_t>(16);
  return called("cudaEventCreate");
}
cudaError_t cudaEventDestroy(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return called("cudaEventRecord"); }
cudaError_t cudaEventSynchronize(cudaEvent_t) { return called("cudaEventSynchronize"); }
cudaError_t cudaEventElapsedTime(float* ms, cudaEvent_t, cudaEvent_t) {
  *ms = 0.f;
  return cudaSuccess;
}
cudaError_t cudaStreamCreateWithFlags(cudaStream_t* s, unsigned) {
  *s = reinterpret_cast<cudaStream_t>(16);
  return cudaSuccess;
}
cudaError_t cudaStreamDestroy(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return called("cudaStreamSynchronize"); }
cudaError_t cudaStreamWaitEvent(cudaStream_t, cudaEvent_t, unsigned) { return called("cudaStreamWaitEvent"); }
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus* s) {
  *s = cudaStreamCaptureStatusNone;
  return cudaSuccess;
}
cudaError_t cudaGetDevice(int* d) {
  *d = 0;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) {
  *v = 152;
  return cudaSuccess;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return "a failure that the test asked for"; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void**, unsigned, unsigned long long, cudaDriverEntryPointQueryResult*) {
  return cudaErrorNotSupported;  // no tensor maps: the CUDA-core kernels are chosen
}
gp_status gp_boundary_demand_noalloc(gp_ctx*, int32_t, const gp_request*, const void*, gp_demand*, int32_t*) {
  return GP_ERR_UNSUPPORTED;
}
}

// The library's own allocations (linked with -Bsymbolic).
void* operator new(size_t n) {
  ++news;
  if (news_until_failure > 0 && --news_until_failure == 0) {
    news_until_failure = -1;
    throw std::bad_alloc();
  }
  if (void* p = std::malloc(n ? n : 1)) return p;
  throw std::bad_alloc();
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, size_t) noexcept { std::free(p); }

namespace gp {
#define FAKE_LAUNCH(name, args) \
  cudaError_t name(const args&, cudaStream_t) { return called(#name); }
FAKE_LAUNCH(launch_append, AppendArgs)
FAKE_LAUNCH(launch_chunk, ChunkArgs)
FAKE_LAUNCH(launch_chunk_tc, ChunkTcArgs)
FAKE_LAUNCH(launch_chunk_weights, ChunkArgs)
FAKE_LAUNCH(launch_chunk_weights_tc, ChunkTcArgs)
FAKE_LAUNCH(launch_compress, CompressArgs)
FAKE_LAUNCH(launch_decode_attention, AttnArgs)
FAKE_LAUNCH(launch_decode_weights, WeightArgs)
FAKE_LAUNCH(launch_demand_ffma, DemandArgs)
FAKE_LAUNCH(launch_demand_tc, DemandArgs)
FAKE_LAUNCH(launch_ema, EmaArgs)
FAKE_LAUNCH(launch_entropy, EntropyArgs)
FAKE_LAUNCH(launch_evict_move, EvictArgs)
FAKE_LAUNCH(launch_prep, PrepArgs)
// keeps the first slots of every unit
cudaError_t launch_evict_select(const EvictArgs& a, cudaStream_t) {
  if (called("launch_evict_select") != cudaSuccess) return cudaErrorMemoryAllocation;
  for (int r = 0; r < a.n && !skip_select; ++r)
    for (int u = 0; u < a.L * a.Hkv && a.reqs[r].items; ++u)
      for (int i = 0; i < a.reqs[r].keep; ++i) a.idx[a.reqs[r].idx_off + (size_t)u * a.reqs[r].idx_pitch + i] = (uint16_t)i;
  return cudaSuccess;
}
}  // namespace gp
