// Gated feed-forward product over feature rows and its backward pass.
//
//   g = x W0 + b0, u = x W1 + b1, out = act(g) u
//   dg = dh u act'(g), du = dh act(g)
//   dx = dg W0^T + du W1^T, dW = x^T [dg du], db = column sums of [dg du]
//
// Tiled products on the CUDA cores, fp32 accumulation.
#include <algorithm>

#include "smc_internal.h"
#include "smc_rows.cuh"

namespace smc {
namespace {

constexpr int kT = 64;   // tile edge
constexpr int kKs = 16;  // depth of a step
constexpr int kGatedThreads = 256;

__device__ __forceinline__ float act_value(float v, int act) {
  switch (act) {
    case SMC_ACT_RELU:
      return fmaxf(v, 0.f);
    case SMC_ACT_SILU:
      return v / (1.f + expf(-v));
    case SMC_ACT_GELU:
      return 0.5f * v * (1.f + erff(v * 0.7071067811865476f));
    default:
      return v;
  }
}
__device__ __forceinline__ float act_slope(float v, int act) {
  switch (act) {
    case SMC_ACT_RELU:
      return v > 0.f ? 1.f : 0.f;
    case SMC_ACT_SILU: {
      const float s = 1.f / (1.f + expf(-v));
      return s * (1.f + v * (1.f - s));
    }
    case SMC_ACT_GELU:
      return 0.5f * (1.f + erff(v * 0.7071067811865476f)) +
             v * expf(-0.5f * v * v) * 0.3989422804014327f;
    default:
      return 1.f;
  }
}

// D[m][n] = sum over k of A(m, k) B(k, n) for NB products that share A; each
// thread ends with 4 x 4 sums and passes them to the epilogue.
template <int NB, class LA, class LB, class Epi>
__device__ __forceinline__ void tile_product(int64_t m0, int64_t n0, int64_t M, int64_t N,
                                             int64_t k0, int64_t k1, LA la, LB lb, Epi epi) {
  __shared__ float sa[kKs][kT + 1], sb[NB][kKs][kT + 1];
  float acc[NB][4][4] = {};
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  for (int64_t kk = k0; kk < k1; kk += kKs) {
    for (int i = threadIdx.x; i < kT * kKs; i += kGatedThreads) {
      const int k = i % kKs, r = i / kKs;
      sa[k][r] = m0 + r < M && kk + k < k1 ? la(m0 + r, kk + k) : 0.f;
      for (int b = 0; b < NB; ++b)
        sb[b][k][r] = n0 + r < N && kk + k < k1 ? lb(b, kk + k, n0 + r) : 0.f;
    }
    __syncthreads();
    for (int k = 0; k < kKs; ++k)
      for (int i = 0; i < 4; ++i)
        for (int b = 0; b < NB; ++b)
          for (int j = 0; j < 4; ++j) acc[b][i][j] += sa[k][ty + 16 * i] * sb[b][k][tx + 16 * j];
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      float v[NB];
      for (int b = 0; b < NB; ++b) v[b] = acc[b][i][j];
      if (m < M && n < N) epi(m, n, v);
    }
}

template <class T>
struct Args {
  const T *x, *W, *bias, *dh;
  T *out, *dx, *dW, *dbias, *dgu;  // dgu: [n][2 hidden] = dg, du
  int64_t n;
  int cin, hidden, act;
};

// out (BWD: dg and du) of one 64 x 64 tile.
template <class T, bool BWD>
__global__ void __launch_bounds__(kGatedThreads) k_gated_pre(Args<T> a) {
  const int64_t C = a.cin, H = a.hidden;
  tile_product<2>(
      blockIdx.x * int64_t(kT), blockIdx.y * int64_t(kT), a.n, H, 0, C,
      [&](int64_t m, int64_t k) { return rows::to_float(a.x[m * C + k]); },
      [&](int b, int64_t k, int64_t j) { return rows::to_float(a.W[(b * C + k) * H + j]); },
      [&](int64_t m, int64_t j, const float* v) {
        const float g = v[0] + (a.bias ? rows::to_float(a.bias[j]) : 0.f);
        const float u = v[1] + (a.bias ? rows::to_float(a.bias[H + j]) : 0.f);
        if constexpr (BWD) {
          const float dh = rows::to_float(a.dh[m * H + j]);
          a.dgu[m * 2 * H + j] = rows::from_float<T>(dh * u * act_slope(g, a.act));
          a.dgu[m * 2 * H + H + j] = rows::from_float<T>(dh * act_value(g, a.act));
        } else {
          a.out[m * H + j] = rows::from_float<T>(act_value(g, a.act) * u);
        }
      });
}

template <class T>
__global__ void __launch_bounds__(kGatedThreads) k_gated_dx(Args<T> a) {
  const int64_t C = a.cin, H = a.hidden;
  tile_product<1>(
      blockIdx.x * int64_t(kT), blockIdx.y * int64_t(kT), a.n, C, 0, 2 * H,
      [&](int64_t m, int64_t k) { return rows::to_float(a.dgu[m * 2 * H + k]); },
      [&](int, int64_t k, int64_t j) {
        return rows::to_float(k < H ? a.W[j * H + k] : a.W[(C + j) * H + k - H]);
      },
      [&](int64_t m, int64_t j, const float* v) { a.dx[m * C + j] = rows::from_float<T>(v[0]); });
}

template <class T>
__global__ void __launch_bounds__(kGatedThreads) k_gated_dw(Args<T> a) {
  const int64_t C = a.cin, H = a.hidden;
  tile_product<1>(
      blockIdx.x * int64_t(kT), blockIdx.y * int64_t(kT), C, 2 * H, 0, a.n,
      [&](int64_t m, int64_t k) { return rows::to_float(a.x[k * C + m]); },
      [&](int, int64_t k, int64_t j) { return rows::to_float(a.dgu[k * 2 * H + j]); },
      [&](int64_t m, int64_t j, const float* v) {
        a.dW[((j < H ? 0 : C) + m) * H + (j < H ? j : j - H)] = rows::from_float<T>(v[0]);
      });
}

template <class T>
__global__ void __launch_bounds__(kGatedThreads) k_gated_db(Args<T> a) {
  __shared__ float part[8][33];
  const int64_t H2 = 2 * int64_t(a.hidden), j = blockIdx.x * int64_t(32) + threadIdx.x % 32;
  float s = 0.f;
  if (j < H2)
    for (int64_t r = threadIdx.x / 32; r < a.n; r += 8) s += rows::to_float(a.dgu[r * H2 + j]);
  part[threadIdx.x / 32][threadIdx.x % 32] = s;
  __syncthreads();
  if (threadIdx.x < 32 && j < H2) {
    for (int w = 1; w < 8; ++w) s += part[w][threadIdx.x];
    a.dbias[j] = rows::from_float<T>(s);
  }
}

unsigned tiles(int64_t m) { return unsigned((m + kT - 1) / kT); }

template <class T>
Args<T> args_of(const GatedCall& g) {
  Args<T> a = {};
  a.x = static_cast<const T*>(g.x);
  a.W = static_cast<const T*>(g.W);
  a.bias = static_cast<const T*>(g.bias);
  a.dgu = static_cast<T*>(g.workspace);
  a.n = g.n;
  a.cin = g.cin;
  a.hidden = g.hidden;
  a.act = g.act;
  return a;
}

}  // namespace

int64_t gated_workspace(int64_t n, int, int hidden, int dtype, bool backward) {
  return backward ? n * 2 * hidden * (dtype == SMC_F32 ? 4 : 2) : 0;
}

int gated_forward(const GatedCall& g, void* out, cudaStream_t s) {
  return rows::by_type(g.dtype, [&](auto tag) {
    using T = decltype(tag);
    Args<T> a = args_of<T>(g);
    a.out = static_cast<T*>(out);
    k_gated_pre<T, false><<<dim3(tiles(g.n), tiles(g.hidden)), kGatedThreads, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? SMC_OK : SMC_ERR_CUDA;
  });
}

int gated_backward(const GatedCall& g, const void* dh, void* dx, void* dW, void* dbias,
                   cudaStream_t s) {
  return rows::by_type(g.dtype, [&](auto tag) {
    using T = decltype(tag);
    Args<T> a = args_of<T>(g);
    a.dh = static_cast<const T*>(dh);
    a.dx = static_cast<T*>(dx);
    a.dW = static_cast<T*>(dW);
    a.dbias = static_cast<T*>(dbias);
    k_gated_pre<T, true><<<dim3(tiles(g.n), tiles(g.hidden)), kGatedThreads, 0, s>>>(a);
    if (dx) k_gated_dx<T><<<dim3(tiles(g.n), tiles(g.cin)), kGatedThreads, 0, s>>>(a);
    if (dW)
      k_gated_dw<T><<<dim3(tiles(g.cin), tiles(2 * int64_t(g.hidden))), kGatedThreads, 0, s>>>(a);
    if (dbias)
      k_gated_db<T><<<unsigned((2 * int64_t(g.hidden) + 31) / 32), kGatedThreads, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? SMC_OK : SMC_ERR_CUDA;
  });
}

}  // namespace smc
