// Attention of each row over the blocks that are listed for it, on the CUDA cores:
// fp32 caches or queries, or when forced.
//
//   z_i = q . k_i / sqrt(d) over the tokens of the listed blocks up to the row's own,
//   a = softmax(z),  out = sum a v  (0 when the list is empty).
// A list is ascending; it ends at the first entry that is negative, not above the
// one before it or past the row's own block.
//
// A cluster of `splits` CTAs a (row, KV head); each takes an even share of the
// list, and the shares' maxima, sums and outputs are joined through distributed
// shared memory: no scratch, no second launch, one fixed order.
// In a CTA a key's row is read by D / 8 lanes, 8 dimensions each; every group of
// lanes keeps its own running maximum and sum (base 2) over its keys.  The logits of
// four keys are summed over the lanes by halves, so that a lane ends with one or two of
// them and weighs those alone (15 exchanges for 16 logits instead of 64).  All in fp32;
// one rounding to the query's type at the end.  Six requests of 3 to 5 rows, d = 64, fp32, 24 blocks
// of 16: 6.2 us in a graph.  64 requests of 2048 listed tokens,
// 32 + 8 heads, d = 128, fp32: 240 us, 66 % of the copy rate; with registers for one CTA an SM
// (147; of 128, G = 4 spills 24 bytes a thread) 402 us: the loads of two hide each other's sums.
#include <cuda_bf16.h>

#include <cstdint>

#include "math2.cuh"
#include "step.cuh"

namespace gp {
namespace {

constexpr int NT = 256;
constexpr int NW = NT / 32;
constexpr int ENTRIES = 64;  // of a share that are looked up at a time
constexpr float NEG = -1.0e30f;
constexpr float LAZY = 16.f;

// Dimension t of the 8 that lane c of a group owns (k_attention.cu's layout: the
// lanes of a quarter warp read 128 contiguous bytes).
template <int D, bool F32>
__device__ __forceinline__ int lane_dim(int c, int t) {
  if constexpr (F32) return t < 4 ? 4 * c + t : D / 2 + 4 * c + (t - 4);
  else return 8 * c + t;
}
template <int D, bool F32>
__device__ __forceinline__ void load_row(const unsigned char* row, int c, float (&f)[8]) {
  if constexpr (F32) {
    const float4 x = *reinterpret_cast<const float4*>(row + c * 16), y = *reinterpret_cast<const float4*>(row + (c + D / 8) * 16);
    f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
    f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(row + c * 16);
    const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

template <int D, int G, bool QF32, bool KF32>
__global__ void __launch_bounds__(NT, 2) k_sparse(const __grid_constant__ SparseArgs a) {
  constexpr int LN = D / 8;           // lanes of a group
  constexpr int GROUPS = NT / LN;
  constexpr int U = 4;                // keys of a group in flight
  constexpr int KB = KF32 ? 4 : 2;
  __shared__ int count_s;
  __shared__ int64_t at_s[ENTRIES];   // first cache row of an entry's block, -1: none
  __shared__ int tok_s[ENTRIES];      // its first logical slot
  __shared__ float acc_s[NW][G][D];
  __shared__ float m_s[NW][G], l_s[NW][G];
  __shared__ float part[G][D + 2];    // this CTA's outputs, maxima, sums
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = tid % LN, group = tid / LN;
  const int C = a.splits, rank = blockIdx.x % C;
  const int64_t unit = blockIdx.x / C;
  const int row = (int)(unit / a.Hkv), h = (int)(unit % a.Hkv);
  begin_step();
  const StepRow rw = find_row(a.s, row, tid == 0);
  if (!rw.live) return;  // (the whole cluster)
  const int lb = log2_of(a.block), lper = kStepPageLog - lb, own = rw.at >> lb;
  const int32_t* list = a.blocks + unit * a.top;
  if (tid == 0) count_s = a.top;
  __syncthreads();
  for (int k = tid; k < a.top; k += NT) {
    const int b = list[k], before = k ? list[k - 1] : -1;
    if (b < 0 || b <= before || b > own) atomicMin(&count_s, k);
  }
  float q[G][8];
  const float sc = 1.4426950408889634f / sqrtf((float)D);
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const size_t at = ((size_t)row * a.Hq + h * G + g) * D + lane_dim<D, KF32>(c, t);
      q[g][t] = sc * (QF32 ? static_cast<const float*>(a.q)[at] : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at]));
    }
  __syncthreads();
  const int count = count_s;
  const int from = (int)((int64_t)count * rank / C), to = (int)((int64_t)count * (rank + 1) / C);

  // The G U logits of a turn are summed over the lanes of the group by halves, after
  // which lane c holds OWN of them, those from FIRST(c) = g U + u on; it keeps the
  // maximum and its part of the sum of their head.
  constexpr int NV = G * U, OWN = NV > LN ? NV / LN : 1, TWINS = LN > NV ? LN / NV : 1;  // TWINS lanes hold the same
  const unsigned mates = ((1u << (LN - 1) << 1) - 1) << (lane / LN * LN);
  const int first = c / TWINS * OWN;
  float m_own = NEG, l_own = 0.f, acc[G][8];
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int t = 0; t < 8; ++t) acc[g][t] = 0.f;
  for (int e0 = from; e0 < to; e0 += ENTRIES) {
    const int n = min(ENTRIES, to - e0);
    __syncthreads();
    if (tid < n) {
      const int b = list[e0 + tid], page = step_page(a.s, rw.slot, b >> lper);
      at_s[tid] = page < 0 ? -1 : (((int64_t)a.layer * a.s.num_pages_total + page) * a.Hkv + h) * kStepPage + ((b << lb) & (kStepPage - 1));
      tok_s[tid] = b << lb;
    }
    __syncthreads();
    const int keys = n << lb;
    for (int k0 = group; k0 < keys; k0 += GROUPS * U) {
      float z[NV], v[U][8];
      unsigned seen = 0u;  // a bit a key
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * GROUPS, e = min(k >> lb, n - 1), o = k & (a.block - 1);
        const bool see = k < keys && at_s[e] >= 0 && tok_s[e] + o <= rw.at;
        float kk[8];
        if (see) {
          const size_t at = (size_t)(at_s[e] + o) * D * KB;
          load_row<D, KF32>(static_cast<const unsigned char*>(a.k_cache) + at, c, kk);
          load_row<D, KF32>(static_cast<const unsigned char*>(a.v_cache) + at, c, v[u]);
          seen |= 1u << u;
        } else {
#pragma unroll
          for (int t = 0; t < 8; ++t) kk[t] = v[u][t] = 0.f;
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          float x = 0.f;
#pragma unroll
          for (int t = 0; t < 8; ++t) x = fmaf(q[g][t], kk[t], x);
          z[g * U + u] = x;
        }
      }
      // (the lanes of a group take the same turns; groups of a warp may not)
      int have = NV;
#pragma unroll
      for (int d = LN / 2; d > 0; d /= 2) {
        if (have > 1) {
          have /= 2;
          const bool upper = (c & d) != 0;
#pragma unroll
          for (int i = 0; i < NV / 2; ++i)
            if (i < have) {
              const float keep = upper ? z[i + have] : z[i], send = upper ? z[i] : z[i + have];
              z[i] = keep + __shfl_xor_sync(mates, send, d);
            }
        } else {
          z[0] += __shfl_xor_sync(mates, z[0], d);
        }
      }
      float top = NEG;
#pragma unroll
      for (int i = 0; i < OWN; ++i) {
        if (!(seen >> ((first + i) % U) & 1u)) z[i] = __int_as_float(0xff800000);  // -inf
        top = fmaxf(top, z[i]);
      }
#pragma unroll
      for (int d = TWINS; d < U / OWN * TWINS; d *= 2) top = fmaxf(top, __shfl_xor_sync(mates, top, d));
      const bool grow = top > m_own + LAZY;
      if (__any_sync(mates, grow)) {  // a maximum is followed only when it grows by more than 16
        const float f = grow ? ex2f(m_own - top) : 1.f;
        if (grow) m_own = top;
        l_own *= f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float fg = __shfl_sync(mates, f, g * U / OWN * TWINS, LN);
#pragma unroll
          for (int t = 0; t < 8; ++t) acc[g][t] *= fg;
        }
      }
      float w[OWN];
#pragma unroll
      for (int i = 0; i < OWN; ++i) {
        w[i] = ex2f(z[i] - m_own);
        l_own += w[i];
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float x = __shfl_sync(mates, w[(g * U + u) % OWN], (g * U + u) / OWN * TWINS, LN);
#pragma unroll
          for (int t = 0; t < 8; ++t) acc[g][t] = fmaf(x, v[u][t], acc[g][t]);
        }
    }
  }
  __syncwarp();
#pragma unroll
  for (int d = TWINS; d < U / OWN * TWINS; d *= 2) l_own += __shfl_xor_sync(0xffffffffu, l_own, d);
  float m[G], l[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    m[g] = __shfl_sync(0xffffffffu, m_own, g * U / OWN * TWINS, LN);
    l[g] = __shfl_sync(0xffffffffu, l_own, g * U / OWN * TWINS, LN);
  }
  // the groups of a warp, the warps, the CTAs
#pragma unroll
  for (int d = LN; d < 32; d *= 2)
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float mo = __shfl_xor_sync(0xffffffffu, m[g], d), lo = __shfl_xor_sync(0xffffffffu, l[g], d);
      const float top = fmaxf(m[g], mo), f = ex2f(m[g] - top), fo = ex2f(mo - top);
      m[g] = top;
      l[g] = l[g] * f + lo * fo;
#pragma unroll
      for (int t = 0; t < 8; ++t) acc[g][t] = acc[g][t] * f + __shfl_xor_sync(0xffffffffu, acc[g][t], d) * fo;
    }
  if (lane < LN) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
      for (int t = 0; t < 8; ++t) acc_s[warp][g][lane_dim<D, KF32>(c, t)] = acc[g][t];
      if (lane == 0) {
        m_s[warp][g] = m[g];
        l_s[warp][g] = l[g];
      }
    }
  }
  __syncthreads();
  for (int x = tid; x < G * D; x += NT) {
    const int g = x / D, d = x % D;
    float top = NEG;
#pragma unroll
    for (int w = 0; w < NW; ++w) top = fmaxf(top, m_s[w][g]);
    float o = 0.f, sum = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = ex2f(m_s[w][g] - top);
      o = fmaf(acc_s[w][g][d], f, o);
      sum = fmaf(l_s[w][g], f, sum);
    }
    part[g][d] = o;
    if (d == 0) {
      part[g][D] = top;
      part[g][D + 1] = sum;
    }
  }
  auto meet = [&] {
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  };
  if (C > 1) meet();
  else __syncthreads();
  auto of = [&](int r, const float* p) {  // *p of CTA r of the cluster
    if (C == 1) return *p;
    uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(p)), there;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(r));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(there) : "memory");
    return v;
  };
  for (int x = rank * NT + tid; x < G * D; x += C * NT) {
    const int g = x / D, d = x % D;
    float top = NEG;
    for (int r = 0; r < C; ++r) top = fmaxf(top, of(r, &part[g][D]));
    float o = 0.f, sum = 0.f;
    for (int r = 0; r < C; ++r) {
      const float f = ex2f(of(r, &part[g][D]) - top);
      o = fmaf(of(r, &part[g][d]), f, o);
      sum = fmaf(of(r, &part[g][D + 1]), f, sum);
    }
    const float y = sum == 0.f ? 0.f : o / sum;  // (an empty list; NaN stays NaN)
    const size_t at = ((size_t)row * a.Hq + h * G + g) * D + d;
    if (QF32) static_cast<float*>(a.out)[at] = y;
    else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(y);
  }
  if (C > 1) meet();  // no CTA leaves while another reads it
}

template <int D, int G, bool QF32, bool KF32>
cudaError_t launch_t(const SparseArgs& a, cudaStream_t s) {
  return launch_step_kernel(k_sparse<D, G, QF32, KF32>, dim3((unsigned)(a.s.max_rows * a.Hkv * a.splits)), NT, 0, a.splits, s, a);
}
template <int D, int G>
cudaError_t launch_g(const SparseArgs& a, cudaStream_t s) {
  if (a.q_f32) return a.kv_f32 ? launch_t<D, G, true, true>(a, s) : launch_t<D, G, true, false>(a, s);
  return a.kv_f32 ? launch_t<D, G, false, true>(a, s) : launch_t<D, G, false, false>(a, s);
}
template <int D>
cudaError_t launch_d(const SparseArgs& a, cudaStream_t s) {
  switch (a.Hq / a.Hkv) {
    case 2: return launch_g<D, 2>(a, s);
    case 4: return launch_g<D, 4>(a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_sparse(const SparseArgs& a, cudaStream_t s) {
  if (a.s.n == 0 || a.s.max_rows == 0) return cudaSuccess;
  if (a.D == 128) return launch_d<128>(a, s);
  if (a.D == 64) return launch_d<64>(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace gp
