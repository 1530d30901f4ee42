// Rotary forms of new tokens, written where a step's slot map says.
//
//   (x_a, x_b) -> amplitude (x_a cos - x_b sin, x_b cos + x_a sin),
//   angle position f_i,  pairs (i, i + rd / 2) or (2 i, 2 i + 1), i < rd / 2,
// over the first rd = rotary_dim dimensions of a head, the others copied: the
// queries to q_rot, the keys to their page, the values copied there.  f_i are the
// scaled inverse frequencies, in fp64 with the launch (512 bytes: a captured
// launch carries its own).  The angle is formed and reduced to [-pi, pi] in fp64;
// one rounding, to the type of the query or cache, at the end.
//
// Bounded by HBM: every element is read and written once in 16-byte pieces.  A
// unit is two pieces of a head that belong together: of rotated halves the
// pieces p and p + rd / 2, else (interleaved pairs, copied dimensions) two
// neighbours; so a pair is in one thread and q_rot may be q.  A block a token;
// its rd / 2 angles serve all heads and are formed while the rows are on their way,
// which start before the row's place is looked up.  Small blocks keep
// more loads in flight beside the angles of others: 13 621 rows of 32 + 8 heads, d = 128,
// interleaved, 56 us with 64 threads, 59 with 192, 73 with 256 and 82 with 384, by
// themselves (a row of 16 + 8 heads, d = 64: 24 and 37 with 64 and 192); among others, their
// starts overlapped, 52 us, 95 % of the copy rate.
#include <cuda_bf16.h>

#include <cstdint>

#include "step.cuh"

namespace gp {
namespace {

constexpr int NT = 64;  // and at least half a head
constexpr int PAGE = 256;

template <bool F32>
__device__ __forceinline__ void unpack(const uint4& u, float* f) {
  const unsigned w[4] = {u.x, u.y, u.z, u.w};
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
template <bool F32>
__device__ __forceinline__ uint4 pack(const float* f) {
  unsigned w[4];
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const unsigned*>(&b);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Unit i of a head's row: its two pieces, and whether they are rotated.
struct Unit {
  int p0, p1;
  bool turned;
};
template <int N>  // elements of a piece
__device__ __forceinline__ Unit unit_of(const MappedArgs& a, int i) {
  const int ru = a.rotary_dim / (2 * N);
  if (i >= ru || a.interleaved) return {2 * i, 2 * i + 1, i < ru};
  return {i, i + ru, true};
}

template <bool F32, int N = F32 ? 4 : 8>
__device__ __forceinline__ void turn(const MappedArgs& a, int i, uint4& u0, uint4& u1, const float* cs, const float* sn) {
  float x[N], y[N];
  unpack<F32>(u0, x);
  unpack<F32>(u1, y);
  if (a.interleaved) {
#pragma unroll
    for (int k = 0; k < N; k += 2) {
      const int f = i * N + k / 2, g = f + N / 2;  // pairs of the first and of the second piece
      float p = x[k], q = x[k + 1];
      x[k] = fmaf(p, cs[f], -q * sn[f]);
      x[k + 1] = fmaf(q, cs[f], p * sn[f]);
      p = y[k], q = y[k + 1];
      y[k] = fmaf(p, cs[g], -q * sn[g]);
      y[k + 1] = fmaf(q, cs[g], p * sn[g]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float c = cs[i * N + k], s = sn[i * N + k], p = x[k], q = y[k];
      x[k] = fmaf(p, c, -q * s);
      y[k] = fmaf(q, c, p * s);
    }
  }
  u0 = pack<F32>(x);
  u1 = pack<F32>(y);
}

template <int D, bool QF32, bool KF32>
__global__ void __launch_bounds__(NT) k_mapped(const __grid_constant__ MappedArgs a) {
  constexpr int QE = QF32 ? 4 : 2, KE = KF32 ? 4 : 2, NQ = 16 / QE, NK = 16 / KE;  // bytes of an element, elements of a piece
  constexpr int UQ = D / (2 * NQ), UK = D / (2 * NK);                             // units of a head
  constexpr int AHEAD = 3;  // units a thread loads before the angles are known
  __shared__ float cs[D / 2];
  __shared__ float sn[D / 2];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const int nq = a.q ? a.Hq * UQ : 0, nk = nq + a.Hkv * UK, nv = nk + a.Hkv * UK;
  auto load = [&](int u, uint4& u0, uint4& u1) {
    if (u >= nv) return;
    const uint4* src;
    Unit w;
    if (u < nq) {
      src = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(a.q) + (row * a.q_row + u / UQ * D) * QE);
      w = unit_of<NQ>(a, u % UQ);
    } else {
      const bool key = u < nk;
      const int v = u - (key ? nq : nk);
      src = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(key ? a.k : a.v) +
                                           (row * (key ? a.k_row : a.v_row) + v / UK * D) * KE);
      w = unit_of<NK>(a, v % UK);
    }
    u0 = src[w.p0];
    u1 = src[w.p1];
  };
  begin_step();
  // the rows are on their way before their place is known
  uint4 u0[AHEAD], u1[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) load(tid + i * NT, u0[i], u1[i]);
  const int64_t to = a.slot_map[row];
  const double pos = (double)a.positions[row];
  if (to == -1) return;
  if (to < 0 || to >= (int64_t)a.num_pages_total * PAGE) {
    if (tid == 0) atomicOr(a.err, ERR_BAD_PAGE);
    return;
  }
  const size_t head0 = ((size_t)a.layer * a.num_pages_total + (size_t)(to / PAGE)) * a.Hkv;
  const size_t in_page = (size_t)(to % PAGE) * D * KE;
  auto store = [&](int u, uint4 u0, uint4 u1) {
    if (u >= nv) return;
    uint4* dst;
    Unit w;
    if (u < nq) {
      dst = reinterpret_cast<uint4*>(static_cast<unsigned char*>(a.q_rot) + ((size_t)row * a.Hq + u / UQ) * D * QE);
      w = unit_of<NQ>(a, u % UQ);
      if (w.turned) turn<QF32>(a, u % UQ, u0, u1, cs, sn);
    } else {
      const bool key = u < nk;
      const int v = u - (key ? nq : nk);
      dst = reinterpret_cast<uint4*>(static_cast<unsigned char*>(key ? a.k_cache : a.v_cache) +
                                     (head0 + v / UK) * (size_t)PAGE * D * KE + in_page);
      w = unit_of<NK>(a, v % UK);
      if (key && w.turned) turn<KF32>(a, v % UK, u0, u1, cs, sn);
    }
    dst[w.p0] = u0;
    dst[w.p1] = u1;
  };
  if (tid < a.rotary_dim / 2) {
    const double ang = pos * a.inv_freq[tid];
    const double k = rint(ang * 0.15915494309189535);  // 1 / (2 pi)
    double red = fma(-k, 6.283185307179586, ang);      // 2 pi in two parts
    red = fma(-k, 2.4492935982947064e-16, red);
    float s, c;
    sincosf((float)red, &s, &c);
    cs[tid] = c * a.amplitude;
    sn[tid] = s * a.amplitude;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) store(tid + i * NT, u0[i], u1[i]);
  for (int u = tid + AHEAD * NT; u < nv; u += NT) {
    load(u, u0[0], u1[0]);
    store(u, u0[0], u1[0]);
  }
}

template <int D>
cudaError_t launch_d(const MappedArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)a.rows);
  auto launch = [&](auto kernel) { return launch_step_kernel(kernel, grid, NT, 0, 1, s, a); };
  if (a.q_f32) return a.kv_f32 ? launch(k_mapped<D, true, true>) : launch(k_mapped<D, true, false>);
  return a.kv_f32 ? launch(k_mapped<D, false, true>) : launch(k_mapped<D, false, false>);
}

}  // namespace

cudaError_t launch_mapped(const MappedArgs& a, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  if (a.rows < 0) return cudaErrorInvalidValue;
  if (a.D == 128) return launch_d<128>(a, s);
  if (a.D == 64) return launch_d<64>(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace gp
