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
// A thread owns a token, a block a page of one KV head: every weight has one
// writer, so the sums do not depend on any order.
#include <cstdint>

#include "weighted_kernels.h"

namespace gp {
namespace {

constexpr int PAGE = 256;

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int G>
__global__ void __launch_bounds__(PAGE) k_decode_weights(const __grid_constant__ WeightArgs a) {
  int lo = 0, hi = a.n;  // reqs[lo].page0 <= blockIdx.x < reqs[hi].page0, empty requests never found
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.reqs[mid].page0 <= (int)blockIdx.x) lo = mid;
    else hi = mid;
  }
  const WeightReq rq = a.reqs[lo];
  const int h = blockIdx.y;
  const int i = ((int)blockIdx.x - rq.page0) * PAGE + (int)threadIdx.x;
  if (rq.slot < 0 || rq.slot >= a.M || i >= rq.ntok) return;
  const size_t held = (size_t)((rq.ntok + PAGE - 1) / PAGE) * PAGE;  // tokens of a head's logits
  const float* z = a.logits + rq.logit_off + ((size_t)h * held + i) * G;
  float v[G];
  if constexpr (G == 4) {
    const float4 x = __ldcs(reinterpret_cast<const float4*>(z));
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  } else {
    const float2 x = __ldcs(reinterpret_cast<const float2*>(z));
    v[0] = x.x; v[1] = x.y;
  }
  float w = 0.f;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const float2 st = a.stat[(size_t)lo * a.Hq + h * G + g];
    w = fmaf(ex2f(v[g] - st.x), st.y, w);
  }
  float* dst = a.weights + (((size_t)a.layer * a.M + rq.slot) * a.Hkv + h) * a.cap + i;
  *dst += w;
}

}  // namespace

cudaError_t launch_decode_weights(const WeightArgs& a, cudaStream_t s) {
  if (a.pages == 0) return cudaSuccess;
  const dim3 grid((unsigned)a.pages, (unsigned)a.Hkv);
  if (a.Hkv > 65535) return cudaErrorInvalidValue;
  if (a.G == 4) k_decode_weights<4><<<grid, PAGE, 0, s>>>(a);
  else if (a.G == 2) k_decode_weights<2><<<grid, PAGE, 0, s>>>(a);
  else return cudaErrorInvalidValue;
  return cudaGetLastError();
}

}  // namespace gp
