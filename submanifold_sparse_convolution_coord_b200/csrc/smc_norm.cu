// Layer norm over feature rows and its backward pass.
//
//   y = (x - mean) r gamma + beta, r = 1 / sqrt(var + eps)
//   dx = r (g - mean(g) - xhat mean(g xhat)), g = dy gamma, xhat = (x - mean) r
//   dgamma = sum over rows of dy xhat, dbeta = sum over rows of dy
//
// Both passes move each row once and do a few operations per element, so they
// are bound by memory: a row stays in registers from its one load to its store,
// and the backward computes the row's statistics from it again instead of
// reading saved ones.
//
// A row belongs to a group of G threads, G a power of two from 1 to 256: each
// holds VECS vectors of V values (16 bytes where the row length allows it),
// strided by G vectors so that a warp's accesses are contiguous.  Groups of up
// to a warp sum by shuffles, wider ones through shared memory.  Rows too long
// for the registers of 256 threads go through k_norm_long and its kind, which
// read them again from cache.
#include <algorithm>

#include "smc_internal.h"
#include "smc_rows.cuh"

namespace smc {
namespace {

constexpr int kThreads = 256;

// V values of T as one access (V * sizeof(T) <= 16 bytes).
template <class T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};

// Sum over the G threads of a row's group.  Groups wider than a warp use
// `smem`, one float per warp; all threads of the block call it.
template <int G>
__device__ __forceinline__ float group_sum(float v, float* smem) {
#pragma unroll
  for (int o = (G < 32 ? G : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (G > 32) {
    __syncthreads();  // the previous sum has been read
    if (threadIdx.x % 32 == 0) smem[threadIdx.x / 32] = v;
    __syncthreads();
    const float* mine = smem + threadIdx.x / G * (G / 32);
    v = 0.f;
#pragma unroll
    for (int w = 0; w < G / 32; ++w) v += mine[w];
  }
  return v;
}
// Two sums at once.
template <int G>
__device__ __forceinline__ float2 group_sum2(float2 v, float2* smem) {
#pragma unroll
  for (int o = (G < 32 ? G : 32) / 2; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if constexpr (G > 32) {
    __syncthreads();
    if (threadIdx.x % 32 == 0) smem[threadIdx.x / 32] = v;
    __syncthreads();
    const float2* mine = smem + threadIdx.x / G * (G / 32);
    v = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < G / 32; ++w) {
      v.x += mine[w].x;
      v.y += mine[w].y;
    }
  }
  return v;
}

// A group's share of a row in registers.
template <class T, int V, int G, int VECS>
struct RowShare {
  Vec<T, V> raw[VECS];
  __device__ __forceinline__ void load(const T* row, int lane, int c, bool ok) {
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int at = (lane + i * G) * V;
      if (ok && at < c)
        raw[i] = *reinterpret_cast<const Vec<T, V>*>(row + at);
      else
        raw[i] = Vec<T, V>{};
    }
  }
  __device__ __forceinline__ float value(int i, int j) const { return rows::to_float(raw[i].v[j]); }
};

// The mean and 1 / sqrt(var + eps) of a row, the variance about the mean found
// first; c divides by `inv_c` exactly as 1.f / c rounds.
template <class T, int V, int G, int VECS>
__device__ __forceinline__ float2 share_stats(const RowShare<T, V, G, VECS>& x, int lane, int c,
                                              float inv_c, float eps, float* smem) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < VECS; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) s += x.value(i, j);  // 0 outside the row
  const float mean = group_sum<G>(s, smem) * inv_c;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < VECS; ++i)
    if ((lane + i * G) * V < c) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = x.value(i, j) - mean;
        s += d * d;
      }
    }
  return make_float2(mean, rsqrtf(group_sum<G>(s, smem) * inv_c + eps));
}

// Rows per group and step: enough bytes in flight per thread for short rows
// (two vectors at least), one for long ones.
template <int VECS>
constexpr int rows_per_step() {
  return VECS == 1 ? 4 : (VECS == 2 ? 2 : 1);
}

template <class T, int V, int G, int VECS>
__global__ void __launch_bounds__(kThreads)
k_norm(const T* x, const float* __restrict__ gamma, const float* __restrict__ beta, T* out,
       int64_t n, int c, float inv_c, float eps) {
  constexpr int R = rows_per_step<VECS>();
  constexpr int kGroups = kThreads / G;
  __shared__ float smem[kThreads / 32];
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  const int64_t r0 = blockIdx.x * int64_t(kGroups * R) + group;
  RowShare<T, V, G, VECS> share[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int64_t r = r0 + k * kGroups;
    share[k].load(x + r * c, lane, c, r < n);
  }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int64_t r = r0 + k * kGroups;
    const float2 st = share_stats(share[k], lane, c, inv_c, eps, smem);
    if (r >= n) continue;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int at = (lane + i * G) * V;
      if (at >= c) continue;
      Vec<T, V> o;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float v = (share[k].value(i, j) - st.x) * st.y;
        if (gamma) v *= gamma[at + j];
        if (beta) v += beta[at + j];
        o.v[j] = rows::from_float<T>(v);
      }
      *reinterpret_cast<Vec<T, V>*>(out + r * c + at) = o;
    }
  }
}

// Blocks walk the rows with a stride; a thread keeps the sums of dgamma and
// dbeta for its columns, which are the same in every row, and the block joins
// its groups' sums at the end: part[block][2][c].
template <class T, int V, int G, int VECS>
__global__ void __launch_bounds__(kThreads)
k_norm_bwd(const T* __restrict__ x, const float* __restrict__ gamma, const T* __restrict__ dy,
           T* __restrict__ dx, float* __restrict__ part, int64_t n, int c, float inv_c, float eps) {
  constexpr int kGroups = kThreads / G;
  __shared__ float smem[kThreads / 32];
  __shared__ float2 smem2[kThreads / 32];
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  float dg[VECS][V] = {}, db[VECS][V] = {};
  float gm[VECS][V];
#pragma unroll
  for (int i = 0; i < VECS; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int at = (lane + i * G) * V + j;
      gm[i][j] = gamma && at < c ? gamma[at] : 1.f;
    }
  // the block's rows run out together, so that every thread takes part in the sums
  for (int64_t base = blockIdx.x * int64_t(kGroups); base < n; base += int64_t(gridDim.x) * kGroups) {
    const int64_t r = base + group;
    const bool ok = r < n;
    RowShare<T, V, G, VECS> xs, gs;
    xs.load(x + r * c, lane, c, ok);
    gs.load(dy + r * c, lane, c, ok);
    float2 st = share_stats(xs, lane, c, inv_c, eps, smem);
    if (!ok) st.y = 0.f;  // eps = 0 made it infinite
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < VECS; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = gs.value(i, j), xh = (xs.value(i, j) - st.x) * st.y;
        const float g = d * gm[i][j];
        s.x += g;
        s.y += g * xh;
        dg[i][j] += d * xh;
        db[i][j] += d;
      }
    s = group_sum2<G>(s, smem2);
    if (!ok) continue;
    s.x *= inv_c;
    s.y *= inv_c;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int at = (lane + i * G) * V;
      if (at >= c) continue;
      Vec<T, V> o;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float xh = (xs.value(i, j) - st.x) * st.y;
        o.v[j] = rows::from_float<T>(st.y * (gs.value(i, j) * gm[i][j] - s.x - xh * s.y));
      }
      *reinterpret_cast<Vec<T, V>*>(dx + r * c + at) = o;
    }
  }
  if (!part) return;
  // join the groups, one value of dg and db per thread at a time
  float* to = part + blockIdx.x * 2 * int64_t(c);
  __shared__ float2 acc[kThreads];
#pragma unroll
  for (int i = 0; i < VECS; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      __syncthreads();
      acc[threadIdx.x] = make_float2(dg[i][j], db[i][j]);
      __syncthreads();
      const int at = (lane + i * G) * V + j;
      if (group == 0 && at < c) {
        float2 t = acc[lane];
        for (int g = 1; g < kGroups; ++g) {
          t.x += acc[g * G + lane].x;
          t.y += acc[g * G + lane].y;
        }
        to[at] = t.x;
        to[c + at] = t.y;
      }
    }
}

// ---------------------------------------------------------------------------
// rows of any length: one block per row, read again from cache in each pass
// ---------------------------------------------------------------------------
template <class T>
__device__ __forceinline__ float2 long_stats(const T* x, int64_t c, float eps, float* smem) {
  float s = 0.f;
  for (int64_t j = threadIdx.x; j < c; j += kThreads) s += rows::to_float(x[j]);
  const float mean = group_sum<kThreads>(s, smem) / float(c);
  s = 0.f;
  for (int64_t j = threadIdx.x; j < c; j += kThreads) {
    const float d = rows::to_float(x[j]) - mean;
    s += d * d;
  }
  return make_float2(mean, rsqrtf(group_sum<kThreads>(s, smem) / float(c) + eps));
}

template <class T>
__global__ void __launch_bounds__(kThreads)
k_norm_long(const T* x, const float* gamma, const float* beta, T* out, int64_t c, float eps) {
  __shared__ float smem[kThreads / 32];
  x += blockIdx.x * c;
  out += blockIdx.x * c;
  const float2 st = long_stats(x, c, eps, smem);
  for (int64_t j = threadIdx.x; j < c; j += kThreads) {
    float v = (rows::to_float(x[j]) - st.x) * st.y;
    if (gamma) v *= gamma[j];
    if (beta) v += beta[j];
    out[j] = rows::from_float<T>(v);
  }
}

template <class T>
__global__ void __launch_bounds__(kThreads)
k_norm_bwd_long(const T* x, const float* gamma, const T* dy, T* dx, float2* stats, int64_t c,
                float eps) {
  __shared__ float smem[kThreads / 32];
  __shared__ float2 smem2[kThreads / 32];
  x += blockIdx.x * c;
  dy += blockIdx.x * c;
  dx += blockIdx.x * c;
  const float2 st = long_stats(x, c, eps, smem);
  if (threadIdx.x == 0) stats[blockIdx.x] = st;
  float2 s = make_float2(0.f, 0.f);
  for (int64_t j = threadIdx.x; j < c; j += kThreads) {
    const float g = rows::to_float(dy[j]) * (gamma ? gamma[j] : 1.f);
    s.x += g;
    s.y += g * ((rows::to_float(x[j]) - st.x) * st.y);
  }
  s = group_sum2<kThreads>(s, smem2);
  s.x /= float(c);
  s.y /= float(c);
  for (int64_t j = threadIdx.x; j < c; j += kThreads) {
    const float g = rows::to_float(dy[j]) * (gamma ? gamma[j] : 1.f);
    const float xh = (rows::to_float(x[j]) - st.x) * st.y;
    dx[j] = rows::from_float<T>(st.y * (g - s.x - xh * s.y));
  }
}

constexpr int kColRows = 256;  // rows per partial sum of the column kernel

// Partial sums of dgamma and dbeta: block (row chunk, column strip).
template <class T>
__global__ void __launch_bounds__(kThreads)
k_norm_cols(const T* x, const T* dy, const float2* stats, float* part, int64_t n, int64_t c) {
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

// dgamma and dbeta from the partial sums: a block takes 32 of the 2 c columns,
// 32 warps each every 32nd partial, then the warps in order.
__global__ void __launch_bounds__(1024)
k_norm_join(const float* __restrict__ part, float* __restrict__ dgamma, float* __restrict__ dbeta,
            int64_t parts, int64_t c) {
  __shared__ float sums[32][33];
  const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t col = blockIdx.x * int64_t(32) + lane;
  float s = 0.f;
  if (col < 2 * c) {
#pragma unroll 8
    for (int64_t p = w; p < parts; p += 32) s += part[p * 2 * c + col];
  }
  sums[w][lane] = s;
  __syncthreads();
  if (w == 0 && col < 2 * c) {
    for (int i = 1; i < 32; ++i) s += sums[i][lane];
    if (col < c)
      dgamma[col] = s;
    else
      dbeta[col - c] = s;
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
int launched() { return cudaGetLastError() == cudaSuccess ? SMC_OK : SMC_ERR_CUDA; }

int64_t chunks(int64_t n) { return (n + kColRows - 1) / kColRows; }

int sm_count() {
  constexpr int kMaxDev = 64;
  static int cache[kMaxDev] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < kMaxDev && cache[dev] > 0) return cache[dev];
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) {
    cudaGetLastError();
    sms = 148;
  }
  if (dev >= 0 && dev < kMaxDev) cache[dev] = sms;
  return sms;
}

// How a row of c values is dealt to a group: the widest vector that divides
// the row, then the narrowest group whose threads hold at most kVecs vectors.
constexpr int kVecs = 4;
struct Deal {
  int v, g, vecs;  // vecs = 0: the row is too long for registers
};
Deal deal(int64_t c, int elem) {
  Deal d{16 / elem, 1, 0};
  while (c % d.v != 0) d.v /= 2;
  const int64_t vectors = c / d.v;
  // narrow vectors carry few bytes: more of them per thread
  const int most = d.v * elem >= 8 ? kVecs : 2 * kVecs;
  while (d.g < kThreads && vectors > int64_t(d.g) * (d.g < 32 ? 1 : most)) d.g *= 2;
  const int64_t need = (vectors + d.g - 1) / d.g;
  d.vecs = need <= most ? (need <= 1 ? 1 : need <= 2 ? 2 : need <= 4 ? 4 : 8) : 0;
  return d;
}

template <class T, class F>
int by_deal(const Deal& d, F&& f) {
  auto with = [&](auto v, auto g) {
    constexpr int V = decltype(v)::value, G = decltype(g)::value;
    if constexpr (G < 32) {  // one vector a thread, by the rule above
      return f(v, g, std::integral_constant<int, 1>());
    } else {
      switch (d.vecs) {
        case 1: return f(v, g, std::integral_constant<int, 1>());
        case 2: return f(v, g, std::integral_constant<int, 2>());
        case 4: return f(v, g, std::integral_constant<int, 4>());
        default:
          if constexpr (V * sizeof(T) < 8) return f(v, g, std::integral_constant<int, 8>());
          return int(SMC_ERR_INVALID);
      }
    }
  };
  auto wide = [&](auto v) {
    switch (d.g) {
      case 1: return with(v, std::integral_constant<int, 1>());
      case 2: return with(v, std::integral_constant<int, 2>());
      case 4: return with(v, std::integral_constant<int, 4>());
      case 8: return with(v, std::integral_constant<int, 8>());
      case 16: return with(v, std::integral_constant<int, 16>());
      case 32: return with(v, std::integral_constant<int, 32>());
      case 64: return with(v, std::integral_constant<int, 64>());
      case 128: return with(v, std::integral_constant<int, 128>());
      default: return with(v, std::integral_constant<int, 256>());
    }
  };
  switch (d.v) {
    case 1: return wide(std::integral_constant<int, 1>());
    case 2: return wide(std::integral_constant<int, 2>());
    case 4: return wide(std::integral_constant<int, 4>());
    default:
      if constexpr (sizeof(T) == 2) return wide(std::integral_constant<int, 8>());
      return int(SMC_ERR_INVALID);
  }
}

// Blocks of the backward kernel: a few per SM (each leaves one partial sum),
// and no more than there are groups of rows.
int64_t bwd_blocks(int64_t n, const Deal& d) {
  const int64_t groups = kThreads / d.g;
  return std::max<int64_t>(1, std::min<int64_t>((n + groups - 1) / groups, int64_t(sm_count()) * 4));
}

}  // namespace

int layer_norm(const void* x, const float* gamma, const float* beta, void* out, int64_t n,
               int64_t c, int dtype, float eps, cudaStream_t s) {
  return rows::by_type(dtype, [&](auto tag) {
    using T = decltype(tag);
    const T* in = static_cast<const T*>(x);
    T* o = static_cast<T*>(out);
    const Deal d = deal(c, sizeof(T));
    if (d.vecs == 0) {
      k_norm_long<T><<<unsigned(n), kThreads, 0, s>>>(in, gamma, beta, o, c, eps);
      return launched();
    }
    return by_deal<T>(d, [&](auto v, auto g, auto vecs) {
      constexpr int V = decltype(v)::value, G = decltype(g)::value, K = decltype(vecs)::value;
      const int64_t step = kThreads / G * rows_per_step<K>();
      k_norm<T, V, G, K><<<unsigned((n + step - 1) / step), kThreads, 0, s>>>(
          in, gamma, beta, o, n, int(c), 1.f / float(c), eps);
      return launched();
    });
  });
}

int64_t layer_norm_backward_workspace(int64_t n, int64_t c, int dtype) {
  const Deal d = deal(c, dtype == SMC_F32 ? 4 : 2);
  if (n == 0) return 0;
  if (d.vecs == 0)
    return n * int64_t(sizeof(float2)) + chunks(n) * 2 * c * int64_t(sizeof(float));
  return bwd_blocks(n, d) * 2 * c * int64_t(sizeof(float));
}

int layer_norm_backward(const void* x, const float* gamma, const void* dy, void* dx,
                        float* dgamma, float* dbeta, int64_t n, int64_t c, int dtype, float eps,
                        void* workspace, cudaStream_t s) {
  return rows::by_type(dtype, [&](auto tag) {
    using T = decltype(tag);
    const T *in = static_cast<const T*>(x), *g_out = static_cast<const T*>(dy);
    T* g_in = static_cast<T*>(dx);
    const Deal d = deal(c, sizeof(T));
    float* part = static_cast<float*>(workspace);
    int64_t parts = 0;
    if (n > 0 && d.vecs == 0) {
      float2* stats = static_cast<float2*>(workspace);
      part = reinterpret_cast<float*>(stats + n);
      k_norm_bwd_long<T><<<unsigned(n), kThreads, 0, s>>>(in, gamma, g_out, g_in, stats, c, eps);
      if (dgamma) {
        parts = chunks(n);
        k_norm_cols<T><<<dim3(unsigned(parts), unsigned((c + kThreads - 1) / kThreads)), kThreads,
                         0, s>>>(in, g_out, stats, part, n, c);
      }
    } else if (n > 0) {
      const int64_t blocks = bwd_blocks(n, d);
      if (dgamma) parts = blocks;
      const int rc = by_deal<T>(d, [&](auto v, auto g, auto vecs) {
        constexpr int V = decltype(v)::value, G = decltype(g)::value, K = decltype(vecs)::value;
        k_norm_bwd<T, V, G, K><<<unsigned(blocks), kThreads, 0, s>>>(
            in, gamma, g_out, g_in, dgamma ? part : nullptr, n, int(c), 1.f / float(c), eps);
        return launched();
      });
      if (rc != SMC_OK) return rc;
    }
    if (dgamma)
      k_norm_join<<<unsigned((2 * c + 31) / 32), 1024, 0, s>>>(part, dgamma, dbeta, parts, c);
    return launched();
  });
}

}  // namespace smc
