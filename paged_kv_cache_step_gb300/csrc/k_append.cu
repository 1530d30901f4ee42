// New tokens into the paged cache: row t of request r goes to logical slot
// cached + t, at RoPE position pos + t.
//
//   (x_i, x_{i+d/2}) -> (x_i cos - x_{i+d/2} sin, x_{i+d/2} cos + x_i sin),
//   angle (pos + t) theta^(-2i/d),
// for the G heads' queries (to q_rot) and the keys (to the page); the values
// are copied and the slot's accumulated weights cleared.
//
// The angle is formed and reduced to [-pi, pi] in fp64: an fp32 product at
// position 10^5 is off by 2^-24 x 10^5 = 0.006 rad.  One rounding, to the
// type of the query or cache, at the end.
//
// Bounded by HBM: every element is read and written once in 16-byte pieces,
// a pair's two halves by the same thread (so q_rot may be q).  One block a
// token: the d / 2 angles are shared by all its heads, and formed while the
// rows are on their way.  16 884 tokens of 32 + 8 heads, d = 128, bf16: 64 us,
// 96 % of the copy rate (76 us with the loads after the angles).
#include <cuda_bf16.h>

#include <cstdint>

#include "weighted_kernels.h"

namespace gp {
namespace {

constexpr int NT = 256;
constexpr int PAGE = 256;

template <bool F32>
struct Piece;  // 16 bytes
template <>
struct Piece<true> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(const uint4& u, float f[4]) {
    f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 put(const float f[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <>
struct Piece<false> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4& u, float f[8]) {
    const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 put(const float f[8]) {
    unsigned w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const unsigned*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// One piece of each half of a head's row, rotated.
template <bool F32>
__device__ __forceinline__ void rotate_piece(const uint4& lo, const uint4& hi, uint4* dst_lo, uint4* dst_hi, int piece,
                                             const float* cs, const float* sn) {
  using P = Piece<F32>;
  float a[P::N], b[P::N], x[P::N], y[P::N];
  P::get(lo, a);
  P::get(hi, b);
#pragma unroll
  for (int i = 0; i < P::N; ++i) {
    const float c = cs[piece * P::N + i], s = sn[piece * P::N + i];
    x[i] = fmaf(a[i], c, -b[i] * s);
    y[i] = fmaf(b[i], c, a[i] * s);
  }
  *dst_lo = P::put(x);
  *dst_hi = P::put(y);
}

template <int D, bool QF32, bool KF32>
__global__ void __launch_bounds__(NT) k_append(const __grid_constant__ AppendArgs a) {
  constexpr int QB = QF32 ? 4 * D : 2 * D, KB = KF32 ? 4 * D : 2 * D;  // bytes of a row
  constexpr int UQ = D / 2 / Piece<QF32>::N, UK = D / 2 / Piece<KF32>::N, UV = KB / 16;  // units of a head
  constexpr int AHEAD = 2;  // units a thread loads before the angles are known
  __shared__ __align__(16) float cs[D / 2];
  __shared__ __align__(16) float sn[D / 2];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  int lo = 0, hi = a.n;  // request lo: its row0 <= row < request hi's row0
  if (a.n == a.rows) {   // one token each
    lo = (int)row;
  } else {
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((a.reqs ? a.reqs[mid].row0 : a.few[mid].row0) <= row) lo = mid;
      else hi = mid;
    }
  }
  const AppendReq rq = a.reqs ? a.reqs[lo] : a.few[lo];
  const int t = (int)(row - rq.row0);
  const int tok = rq.cached + t;
  const int at = rq.bt_off + (tok / PAGE - rq.cached / PAGE);
  const int page = a.reqs ? a.bt[at] : a.few_bt[at];
  if (page < 0 || page >= a.num_pages_total || rq.slot < 0 || rq.slot >= a.M) {  // the host checked both
    if (tid == 0) atomicOr(a.err, ERR_BAD_PAGE);
    return;
  }
  const size_t head0 = ((size_t)a.layer * a.num_pages_total + page) * a.Hkv;  // (layer, page)'s first KV head
  const size_t in_page = (size_t)(tok % PAGE) * KB;
  const int nq = a.q ? a.Hq * UQ : 0, nk = nq + a.Hkv * UK, nv = nk + a.Hkv * UV;
  // unit u: a piece of each half of a query or key row, or a piece of a value row
  auto load = [&](int u, uint4& lo, uint4& hi) {
    if (u < nq) {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(a.q) + ((size_t)row * a.Hq + u / UQ) * QB);
      lo = src[u % UQ];
      hi = src[u % UQ + UQ];
    } else if (u < nk) {
      const int h = (u - nq) / UK, p = (u - nq) % UK;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(a.k) + ((size_t)row * a.Hkv + h) * KB);
      lo = src[p];
      hi = src[p + UK];
    } else if (u < nv) {
      const int h = (u - nk) / UV, p = (u - nk) % UV;
      lo = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(a.v) + ((size_t)row * a.Hkv + h) * KB)[p];
    }
  };
  auto store = [&](int u, const uint4& lo, const uint4& hi) {
    if (u < nq) {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<unsigned char*>(a.q_rot) + ((size_t)row * a.Hq + u / UQ) * QB) + u % UQ;
      rotate_piece<QF32>(lo, hi, dst, dst + UQ, u % UQ, cs, sn);
    } else if (u < nk) {
      const int h = (u - nq) / UK, p = (u - nq) % UK;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<unsigned char*>(a.k_cache) + (head0 + h) * (size_t)PAGE * KB + in_page) + p;
      rotate_piece<KF32>(lo, hi, dst, dst + UK, p, cs, sn);
    } else if (u < nv) {
      const int h = (u - nk) / UV, p = (u - nk) % UV;
      reinterpret_cast<uint4*>(static_cast<unsigned char*>(a.v_cache) + (head0 + h) * (size_t)PAGE * KB + in_page)[p] = lo;
    }
  };
  uint4 first[AHEAD], second[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) load(tid + i * NT, first[i], second[i]);
  if (tid < D / 2) {
    const double ang = (double)(rq.pos + t) * a.inv_freq[tid];
    const double k = rint(ang * 0.15915494309189535);  // 1 / (2 pi)
    double red = fma(-k, 6.283185307179586, ang);      // 2 pi in two parts
    red = fma(-k, 2.4492935982947064e-16, red);
    float s, c;
    sincosf((float)red, &s, &c);
    cs[tid] = c;
    sn[tid] = s;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) store(tid + i * NT, first[i], second[i]);
  for (int u = tid + AHEAD * NT; u < nv; u += NT) {
    load(u, first[0], second[0]);
    store(u, first[0], second[0]);
  }
  if (a.weights)
    for (int h = tid; h < a.Hkv; h += NT)
      a.weights[(((size_t)a.layer * a.M + rq.slot) * a.Hkv + h) * a.cap + tok] = 0.f;
}

template <int D, bool QF32, bool KF32>
cudaError_t launch_t(const AppendArgs& a, cudaStream_t s) {
  k_append<D, QF32, KF32><<<dim3((unsigned)a.rows), NT, 0, s>>>(a);
  return cudaGetLastError();
}
template <int D>
cudaError_t launch_d(const AppendArgs& a, cudaStream_t s) {
  if (a.q_f32) return a.kv_f32 ? launch_t<D, true, true>(a, s) : launch_t<D, true, false>(a, s);
  return a.kv_f32 ? launch_t<D, false, true>(a, s) : launch_t<D, false, false>(a, s);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  if (a.rows < 0 || a.n < 1) return cudaErrorInvalidValue;
  if (a.D == 128) return launch_d<128>(a, s);
  if (a.D == 64) return launch_d<64>(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace gp
