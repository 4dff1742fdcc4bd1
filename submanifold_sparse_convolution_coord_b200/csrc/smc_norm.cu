// Layer norm over feature rows and its backward pass.
//
//   y = (x - mean) r gamma + beta, r = 1 / sqrt(var + eps)
//   dx = r (g - mean(g) - xhat mean(g xhat)), g = dy gamma, xhat = (x - mean) r
//   dgamma = sum over rows of dy xhat, dbeta = sum over rows of dy
//
// Both passes move each row once and do a few operations per element, so they
// are bound by memory.  The backward recomputes the statistics from x.
#include <algorithm>

#include "smc_internal.h"
#include "smc_rows.cuh"

namespace smc {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float block_sum(float v, float* smem) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();  // the previous sum has been read
  if (threadIdx.x % 32 == 0) smem[threadIdx.x / 32] = v;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) t += smem[w];
  return t;
}

// Mean and 1 / sqrt(var + eps) of a row, the variance about the mean found first.
template <class T>
__device__ __forceinline__ float2 row_stats(const T* x, int64_t c, float eps, float* smem) {
  float s = 0.f;
  for (int64_t j = threadIdx.x; j < c; j += kThreads) s += rows::to_float(x[j]);
  const float mean = block_sum(s, smem) / float(c);
  s = 0.f;
  for (int64_t j = threadIdx.x; j < c; j += kThreads) {
    const float d = rows::to_float(x[j]) - mean;
    s += d * d;
  }
  return make_float2(mean, rsqrtf(block_sum(s, smem) / float(c) + eps));
}

// One block per row, any channel count.
template <class T>
__global__ void __launch_bounds__(kThreads)
k_norm(const T* x, const float* gamma, const float* beta, T* out, int64_t c, float eps) {
  __shared__ float smem[kThreads / 32];
  x += blockIdx.x * c;
  out += blockIdx.x * c;
  const float2 st = row_stats(x, c, eps, smem);
  for (int64_t j = threadIdx.x; j < c; j += kThreads) {
    float v = (rows::to_float(x[j]) - st.x) * st.y;
    if (gamma) v *= gamma[j];
    if (beta) v += beta[j];
    out[j] = rows::from_float<T>(v);
  }
}

template <class T>
__global__ void __launch_bounds__(kThreads)
k_norm_bwd(const T* x, const float* gamma, const T* dy, T* dx, float2* stats, int64_t c,
           float eps) {
  __shared__ float smem[kThreads / 32];
  x += blockIdx.x * c;
  dy += blockIdx.x * c;
  dx += blockIdx.x * c;
  const float2 st = row_stats(x, c, eps, smem);
  if (threadIdx.x == 0) stats[blockIdx.x] = st;
  float s1 = 0.f, s2 = 0.f;
  for (int64_t j = threadIdx.x; j < c; j += kThreads) {
    const float g = rows::to_float(dy[j]) * (gamma ? gamma[j] : 1.f);
    s1 += g;
    s2 += g * ((rows::to_float(x[j]) - st.x) * st.y);
  }
  s1 = block_sum(s1, smem) / float(c);
  s2 = block_sum(s2, smem) / float(c);
  for (int64_t j = threadIdx.x; j < c; j += kThreads) {
    const float g = rows::to_float(dy[j]) * (gamma ? gamma[j] : 1.f);
    const float xh = (rows::to_float(x[j]) - st.x) * st.y;
    dx[j] = rows::from_float<T>(st.y * (g - s1 - xh * s2));
  }
}

constexpr int kColRows = 256;  // rows per partial sum of the column kernel

// Partial sums of dgamma and dbeta: block (column strip, row chunk).
template <class T>
__global__ void __launch_bounds__(kThreads)
k_norm_bwd_cols(const T* x, const T* dy, const float2* stats, float* part, int64_t n, int64_t c) {
  const int64_t j = blockIdx.y * int64_t(kThreads) + threadIdx.x;
  if (j >= c) return;
  const int64_t r0 = blockIdx.x * int64_t(kColRows), r1 = min(n, r0 + kColRows);
  float dg = 0.f, db = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    const float2 st = stats[r];
    const float g = rows::to_float(dy[r * c + j]);
    dg += g * ((rows::to_float(x[r * c + j]) - st.x) * st.y);
    db += g;
  }
  part[(blockIdx.x * 2 + 0) * c + j] = dg;
  part[(blockIdx.x * 2 + 1) * c + j] = db;
}

__global__ void __launch_bounds__(kThreads)
k_norm_bwd_join(const float* part, float* dgamma, float* dbeta, int64_t parts, int64_t c) {
  const int64_t j = blockIdx.x * int64_t(kThreads) + threadIdx.x;
  if (j >= c) return;
  float dg = 0.f, db = 0.f;
  for (int64_t p = 0; p < parts; ++p) {
    dg += part[(p * 2 + 0) * c + j];
    db += part[(p * 2 + 1) * c + j];
  }
  dgamma[j] = dg;
  dbeta[j] = db;
}

int64_t chunks(int64_t n) { return (n + kColRows - 1) / kColRows; }

}  // namespace

int layer_norm(const void* x, const float* gamma, const float* beta, void* out, int64_t n,
               int64_t c, int dtype, float eps, cudaStream_t s) {
  return rows::by_type(dtype, [&](auto tag) {
    using T = decltype(tag);
    k_norm<T><<<unsigned(n), kThreads, 0, s>>>(static_cast<const T*>(x), gamma, beta,
                                               static_cast<T*>(out), c, eps);
    return cudaGetLastError() == cudaSuccess ? SMC_OK : SMC_ERR_CUDA;
  });
}

int64_t layer_norm_backward_workspace(int64_t n, int64_t c, int) {
  return n * int64_t(sizeof(float2)) + chunks(n) * 2 * c * int64_t(sizeof(float));
}

int layer_norm_backward(const void* x, const float* gamma, const void* dy, void* dx,
                        float* dgamma, float* dbeta, int64_t n, int64_t c, int dtype, float eps,
                        void* workspace, cudaStream_t s) {
  return rows::by_type(dtype, [&](auto tag) {
    using T = decltype(tag);
    float2* stats = static_cast<float2*>(workspace);
    float* part = reinterpret_cast<float*>(stats + n);
    if (n > 0)
      k_norm_bwd<T><<<unsigned(n), kThreads, 0, s>>>(static_cast<const T*>(x), gamma,
                                                     static_cast<const T*>(dy),
                                                     static_cast<T*>(dx), stats, c, eps);
    if (dgamma) {
      const unsigned strips = unsigned((c + kThreads - 1) / kThreads);
      if (n > 0)
        k_norm_bwd_cols<T><<<dim3(unsigned(chunks(n)), strips), kThreads, 0, s>>>(
            static_cast<const T*>(x), static_cast<const T*>(dy), stats, part, n, c);
      k_norm_bwd_join<<<strips, kThreads, 0, s>>>(part, dgamma, dbeta, chunks(n), c);
    }
    return cudaGetLastError() == cudaSuccess ? SMC_OK : SMC_ERR_CUDA;
  });
}

}  // namespace smc
