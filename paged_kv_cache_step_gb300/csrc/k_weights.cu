// The accumulated weights of one decode step: for KV head h of request r and
// token i,
//   W_i += sum over the group's heads g of 2^(z_gi - m_g) / l_g,
// z the base-2 logits that the attention kernel kept, m_g and l_g the
// maximum and sum of its softmax, final only once every piece of the pair is
// joined; hence a pass of its own.  It reads G fp32 logits a token (most of
// them still in L2) where K and V cost 4 d bytes in bf16, so it adds about
// (4 G + 4 G + 8) / 4 d = 8 % of the traffic at d = 128, G = 4.  Forming the
// logits again from K would add 50 %.
//
// 64 requests of 1.05 M tokens in all, 32 query and 8 KV heads: 28 us beside 679 of
// attention, whose logits of 134 MB are partly still in L2.
//
// A thread owns four tokens, a warp half a page of one KV head: every weight has
// one writer, so the sums do not depend on any order.
#include <cstdint>

#include "chained.cuh"
#include "math2.cuh"
#include "weighted_kernels.h"

namespace gp {
namespace {

constexpr int PAGE = 256;

constexpr int NT = 256;
constexpr int SPAN = 128;  // tokens of a warp

template <int G>
__global__ void __launch_bounds__(NT) k_decode_weights(const __grid_constant__ WeightArgs a) {
  const int lane = threadIdx.x & 31;
  // the warp's half page: pages of all requests, then KV heads, then halves
  const int64_t id = (int64_t)blockIdx.x * (NT / 32) + (threadIdx.x >> 5);
  const int half = (int)(id & 1), h = (int)((id >> 1) % a.Hkv);
  const int64_t page = (id >> 1) / a.Hkv;
  wait_for_previous();
  if (page >= a.pages) return;
  int lo = 0, hi = a.n;  // reqs[lo].page0 <= page < reqs[hi].page0, empty requests never found
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.reqs[mid].page0 <= page) lo = mid;
    else hi = mid;
  }
  const WeightReq rq = a.reqs[lo];
  const int i0 = ((int)page - rq.page0) * PAGE + half * SPAN + lane;
  if (rq.slot < 0 || rq.slot >= a.M) return;
  const size_t held = (size_t)((rq.ntok + PAGE - 1) / PAGE) * PAGE;  // tokens of a head's logits
  const float* z = a.logits + rq.logit_off + ((size_t)h * held + i0) * G;
  float* dst = a.weights + (((size_t)a.layer * a.M + rq.slot) * a.Hkv + h) * a.cap + i0;
  float v[4][G], w[4], m[G], inv[G];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bool in = i0 + 32 * j < rq.ntok;
    if constexpr (G == 4) {
      const float4 x = in ? __ldcs(reinterpret_cast<const float4*>(z) + 32 * j) : make_float4(0.f, 0.f, 0.f, 0.f);
      v[j][0] = x.x; v[j][1] = x.y; v[j][2] = x.z; v[j][3] = x.w;
    } else {
      const float2 x = in ? __ldcs(reinterpret_cast<const float2*>(z) + 32 * j) : make_float2(0.f, 0.f);
      v[j][0] = x.x; v[j][1] = x.y;
    }
    w[j] = in ? dst[32 * j] : 0.f;
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const float2 st = a.stat[(size_t)lo * a.Hq + h * G + g];
    m[g] = st.x;
    inv[g] = st.y;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float sum = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) sum = fmaf(ex2f(v[j][g] - m[g]), inv[g], sum);
    if (i0 + 32 * j < rq.ntok) dst[32 * j] = w[j] + sum;
  }
}

}  // namespace

cudaError_t launch_decode_weights(const WeightArgs& a, cudaStream_t s) {
  if (a.pages == 0) return cudaSuccess;
  const int64_t warps = 2ll * a.pages * a.Hkv, blocks = (warps + NT / 32 - 1) / (NT / 32);
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)blocks);
  if (a.G == 4) return launch_chained(k_decode_weights<4>, grid, NT, 0, s, a);
  if (a.G == 2) return launch_chained(k_decode_weights<2>, grid, NT, 0, s, a);
  return cudaErrorInvalidValue;
}

}  // namespace gp
