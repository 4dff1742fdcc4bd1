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
#include "smc_ptx.cuh"
#include "smc_rows.cuh"

namespace smc {
namespace {

using rows::add2;
using rows::fma2;
using rows::mul2;

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

// sum / c by c's rounded reciprocal, corrected by what it leaves: a row whose
// values are all alike, and whose sum is exact, has that value as its mean and so
// xhat = 0.  (Without the correction x - sum * inv_c leaves up to 2^-24 of x, which
// eps = 1e-5 lets through as an xhat of up to 0.02 for rows of 1000.)
__device__ __forceinline__ float mean_of(float sum, int c, float inv_c) {
  const float m = sum * inv_c;
  return fmaf(fmaf(-m, float(c), sum), inv_c, m);
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
// first; inv_c = 1 / c.
template <class T, int V, int G, int VECS>
__device__ __forceinline__ float2 share_stats(const RowShare<T, V, G, VECS>& x, int lane, int c,
                                              float inv_c, float eps, float* smem) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < VECS; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) s += x.value(i, j);  // 0 outside the row
  const float mean = mean_of(group_sum<G>(s, smem), c, inv_c);
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

// A thread's share of a row as pairs: value k is vector k / V, element k % V.
// WHOLE: the row fills every thread's share.
template <class T, int V, int G, int VECS, bool WHOLE>
struct Share {
  static constexpr int N = VECS * V, P = (N + 1) / 2;
  // column of value k
  static __device__ __forceinline__ int column(int lane, int k) {
    return (lane + k / V * G) * V + k % V;
  }
  static __device__ __forceinline__ void raw(const T* row, int lane, int c, bool ok,
                                             Vec<T, V> (&q)[VECS]) {
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int at = (lane + i * G) * V;
      q[i] = Vec<T, V>{};
      if (ok && (WHOLE || at < c)) q[i] = *reinterpret_cast<const Vec<T, V>*>(row + at);
    }
  }
  static __device__ __forceinline__ void expand(const Vec<T, V> (&q)[VECS], float2 (&v)[P]) {
    float f[2 * P];
    f[2 * P - 1] = 0.f;
#pragma unroll
    for (int i = 0; i < VECS; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) f[i * V + j] = rows::to_float(q[i].v[j]);
#pragma unroll
    for (int p = 0; p < P; ++p) v[p] = make_float2(f[2 * p], f[2 * p + 1]);
  }
  static __device__ __forceinline__ void load(const T* row, int lane, int c, float2 (&v)[P]) {
    Vec<T, V> q[VECS];
    raw(row, lane, c, true, q);
    expand(q, v);
  }
  // Takes the mean from the values (columns outside the row stay 0) and gives
  // the sum of their squares.
  static __device__ __forceinline__ float centre(float2 (&v)[P], float mean, int lane, int c) {
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      float2 m = make_float2(-mean, -mean);
      if constexpr (!WHOLE || N % 2 != 0) {
        if (2 * p + 1 >= N || column(lane, 2 * p + 1) >= c) m.y = 0.f;
        if (column(lane, 2 * p) >= c) m.x = 0.f;
      }
      v[p] = add2(v[p], m);
      s = fma2(v[p], v[p], s);
    }
    return s.x + s.y;
  }
  static __device__ __forceinline__ float sum(const float2 (&v)[P]) {
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int p = 0; p < P; ++p) s = add2(s, v[p]);
    return s.x + s.y;
  }
};

// V consecutive floats (16-byte aligned when V is a multiple of 4).
template <int V>
__device__ __forceinline__ void load_floats(const float* p, float (&v)[V]) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const float4 q = *reinterpret_cast<const float4*>(p + j);
      v[j] = q.x, v[j + 1] = q.y, v[j + 2] = q.z, v[j + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = p[j];
  }
}

// Rows per group: enough bytes in flight per thread for short rows.
template <class T, int V, int VECS>
constexpr int rows_per_group() {
  constexpr int bytes = VECS * V * int(sizeof(T));
  return bytes <= 16 ? 4 : (bytes <= 32 ? 2 : 1);
}

// Small blocks for rows of up to a warp: more of them are at different stages
// on an SM (4,749,279 x 64 bf16, before the arithmetic in pairs: 238 us with 256
// threads, 200 us with 128; with it 194 us of the 186 that its 1.2 GB take).
template <int G>
constexpr int norm_threads() {
  return G <= 32 ? 128 : kThreads;
}

template <class T, int V, int G, int VECS, bool WHOLE>
__global__ void __launch_bounds__(norm_threads<G>(),
                                  G > 32 ? 1 : (VECS == 1 ? 8 : (VECS * V <= 16 ? 4 : 2)))
k_norm(const T* x, const float* __restrict__ gamma, const float* __restrict__ beta, T* out,
       int64_t n, int c, float inv_c, float eps) {
  using S = Share<T, V, G, VECS, WHOLE>;
  constexpr int R = rows_per_group<T, V, VECS>(), P = S::P;
  constexpr int kGroups = norm_threads<G>() / G;
  __shared__ float smem[kThreads / 32];
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  const int64_t base = blockIdx.x * int64_t(kGroups * R);
  const int rows_here = int(min(n - base, int64_t(kGroups * R)));
  x += base * c;
  out += base * c;
  Vec<T, V> raw[R][VECS];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int r = group + k * kGroups;
    S::raw(x + int64_t(r) * c, lane, c, r < rows_here, raw[k]);
  }
  // one vector a thread: gamma and beta in registers for all R rows
  constexpr bool kHold = VECS == 1;
  float gm[kHold ? VECS : 1][V], bt[kHold ? VECS : 1][V];
  if constexpr (kHold) {
    if (gamma && (WHOLE || lane * V < c)) load_floats(gamma + lane * V, gm[0]);
    if (beta && (WHOLE || lane * V < c)) load_floats(beta + lane * V, bt[0]);
  }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int r = group + k * kGroups;
    float2 v[P];
    S::expand(raw[k], v);
    const float mean = mean_of(group_sum<G>(S::sum(v), smem), c, inv_c);
    const float squares = S::centre(v, mean, lane, c);
    const float rstd = rsqrtf(group_sum<G>(squares, smem) * inv_c + eps);
    if (r >= rows_here) continue;
    float y[2 * P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const float2 q = mul2(v[p], make_float2(rstd, rstd));
      y[2 * p] = q.x;
      y[2 * p + 1] = q.y;
    }
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int at = (lane + i * G) * V, h = kHold ? i : 0;
      if (!WHOLE && at >= c) continue;
      if constexpr (!kHold) {
        if (gamma) load_floats(gamma + at, gm[0]);
        if (beta) load_floats(beta + at, bt[0]);
      }
      float* z = y + i * V;
      if constexpr (V % 2 == 0) {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
          float2 q = make_float2(z[j], z[j + 1]);
          if (gamma) q = mul2(q, make_float2(gm[h][j], gm[h][j + 1]));
          if (beta) q = add2(q, make_float2(bt[h][j], bt[h][j + 1]));
          z[j] = q.x;
          z[j + 1] = q.y;
        }
      } else {
        if (gamma) z[0] *= gm[h][0];
        if (beta) z[0] += bt[h][0];
      }
      Vec<T, V> o;
#pragma unroll
      for (int j = 0; j < V; ++j) o.v[j] = rows::from_float<T>(z[j]);
      *reinterpret_cast<Vec<T, V>*>(out + int64_t(r) * c + at) = o;
    }
  }
}

// ---------------------------------------------------------------------------
// backward, rows of up to a warp
// ---------------------------------------------------------------------------
constexpr int kRingWarps = 8;
// Two blocks per SM with three slots a warp, or, where a lane's share of a row
// is more than 16 values (registers for one block), one with four.
constexpr int ring_blocks(int values) { return values > 16 ? 1 : 2; }
constexpr int ring_stages(int values) { return values > 16 ? 4 : 3; }

// Each warp streams its own chunks of `chunk_rows` consecutive rows of x and dy
// through a ring of slots in shared memory, filled by 16-byte
// asynchronous copies from the 16-byte boundary below the chunk: what is in
// flight does not depend on registers, and rows of any length arrive with whole
// 16-byte accesses.  A lane keeps the sums of dgamma and dbeta for
// its columns, which are the same in every row; the block joins them at the
// end: part[block][2][c].  (209,715 x 128 fp16: 37 us with loads to registers,
// 33 us with chunks of 2 KB, 31 us with 1 KB.)
template <class T, int V, int G, int VECS, bool WHOLE>
__global__ void __launch_bounds__(32 * kRingWarps, ring_blocks(VECS * V))
k_norm_bwd(const T* __restrict__ x, const float* __restrict__ gamma, const T* __restrict__ dy,
           T* __restrict__ dx, float* __restrict__ part, int64_t n, int c, int chunk_rows,
           int slot_bytes, float inv_c, float eps) {
  rows::let_next_start();  // the join
  using S = Share<T, V, G, VECS, WHOLE>;
  constexpr int P = S::P, N = S::N, kRingStages = ring_stages(N);
  constexpr bool kKeep = N <= 20;  // dy * gamma stays in registers, else dy is read again
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x / 32, wl = threadIdx.x % 32, lane = wl % G, group = wl / G;
  const int chunk_bytes = chunk_rows * c * int(sizeof(T));
  uint8_t* ring = smem + warp * (kRingStages * 2) * slot_bytes;  // slot: x, then dy
  const int64_t total = n * c * int64_t(sizeof(T));
  const int64_t chunks = (n + chunk_rows - 1) / chunk_rows;
  const int64_t stride = int64_t(gridDim.x) * kRingWarps;

  float2 gm[P], dg[P] = {}, db[P] = {};
#pragma unroll
  for (int k = 0; k < 2 * P; ++k) {
    const int col = S::column(lane, k);
    const float v = gamma && k < N && col < c ? gamma[col] : 1.f;
    (k & 1 ? gm[k / 2].y : gm[k / 2].x) = v;
  }
  const uint32_t ring0 = ptx::smem_addr(ring) + wl * 16;
  auto fill = [&](int64_t chunk, int slot) {
    if (chunk < chunks) {
      const int64_t from = chunk * chunk_bytes & ~int64_t(15);
      const uint32_t to = ring0 + slot * 2 * slot_bytes;
      const uint8_t* px = reinterpret_cast<const uint8_t*>(x) + from + wl * 16;
      const uint8_t* pd = reinterpret_cast<const uint8_t*>(dy) + from + wl * 16;
      if (from + slot_bytes <= total) {
        for (int at = 0; at < slot_bytes - wl * 16; at += 512) {
          ptx::cp_async_16(to + at, px + at, 16);
          ptx::cp_async_16(to + slot_bytes + at, pd + at, 16);
        }
      } else {  // nothing behind the last row is read
        for (int at = 0; at < slot_bytes - wl * 16; at += 512) {
          const int64_t left = total - from - wl * 16 - at;
          const uint32_t bytes = left >= 16 ? 16u : (left > 0 ? uint32_t(left) : 0u);
          ptx::cp_async_16(to + at, left > 0 ? px + at : reinterpret_cast<const uint8_t*>(x),
                           bytes);
          ptx::cp_async_16(to + slot_bytes + at,
                           left > 0 ? pd + at : reinterpret_cast<const uint8_t*>(dy), bytes);
        }
      }
    }
    ptx::cp_async_commit();
  };
  int64_t chunk = blockIdx.x * int64_t(kRingWarps) + warp;
#pragma unroll
  for (int k = 0; k < kRingStages - 1; ++k) fill(chunk + k * stride, k);
  for (int slot = 0; chunk < chunks; chunk += stride) {
    ptx::cp_async_wait_group<kRingStages - 2>();
    __syncwarp();  // every lane's copies have landed; the slot before this one is free
    fill(chunk + (kRingStages - 1) * stride, slot == 0 ? kRingStages - 1 : slot - 1);
    const uint8_t* here = ring + slot * 2 * slot_bytes + (chunk * chunk_bytes & 15);
    const T* xs = reinterpret_cast<const T*>(here);
    const T* ds = reinterpret_cast<const T*>(here + slot_bytes);
    slot = slot + 1 == kRingStages ? 0 : slot + 1;
    for (int row = group; row < chunk_rows; row += 32 / G) {
      const int64_t r = chunk * chunk_rows + row;
      const bool ok = r < n;
      float2 xc[P], g[P];
      S::load(xs + row * c, lane, c, xc);
      const float mean = mean_of(group_sum<G>(S::sum(xc), nullptr), c, inv_c);
      const float squares = S::centre(xc, mean, lane, c);
      float rstd = rsqrtf(group_sum<G>(squares, nullptr) * inv_c + eps);
      if (!ok) rstd = 0.f;  // a row that does not exist: eps = 0 made it infinite
      const float2 rr = make_float2(rstd, rstd);
      float2 s1 = make_float2(0.f, 0.f), s2 = s1;
      S::load(ds + row * c, lane, c, g);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const float2 d = g[p];
        xc[p] = mul2(xc[p], rr);  // xhat: products with the inverse root's powers could overflow
        db[p] = add2(db[p], d);
        dg[p] = fma2(d, xc[p], dg[p]);
        const float2 q = mul2(d, gm[p]);
        s1 = add2(s1, q);
        s2 = fma2(q, xc[p], s2);
        if (kKeep) g[p] = q;
      }
      const float2 sums = group_sum2<G>(make_float2(s1.x + s1.y, s2.x + s2.y), nullptr);
      // dx = r g - r mean(g) - xhat r mean(g xhat)
      const float k1 = -sums.x * inv_c * rstd, k2 = -sums.y * inv_c * rstd;
      const float2 kk1 = make_float2(k1, k1), kk2 = make_float2(k2, k2);
      if constexpr (!kKeep) {
        S::load(ds + row * c, lane, c, g);
#pragma unroll
        for (int p = 0; p < P; ++p) g[p] = mul2(g[p], gm[p]);
      }
      float out[2 * P];
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const float2 o = fma2(xc[p], kk2, fma2(g[p], rr, kk1));
        out[2 * p] = o.x;
        out[2 * p + 1] = o.y;
      }
      if (!ok) continue;
#pragma unroll
      for (int i = 0; i < VECS; ++i) {
        const int at = (lane + i * G) * V;
        if (!WHOLE && at >= c) continue;
        Vec<T, V> o;
#pragma unroll
        for (int j = 0; j < V; ++j) o.v[j] = rows::from_float<T>(out[i * V + j]);
        *reinterpret_cast<Vec<T, V>*>(dx + r * c + at) = o;
      }
    }
  }
  ptx::cp_async_wait_group<0>();
  if (!part) return;
  // join the warp's groups by shuffles, the warps through shared memory
  __syncthreads();  // the rings are free
  float* acc = reinterpret_cast<float*>(smem);  // [kRingWarps][2][c]
#pragma unroll
  for (int k = 0; k < N; ++k) {
    float a = k & 1 ? dg[k / 2].y : dg[k / 2].x, b = k & 1 ? db[k / 2].y : db[k / 2].x;
#pragma unroll
    for (int o = G; o < 32; o <<= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    const int col = S::column(lane, k);
    if (group == 0 && col < c) {
      acc[(warp * 2 + 0) * c + col] = a;
      acc[(warp * 2 + 1) * c + col] = b;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * c; i += 32 * kRingWarps) {
    float t = 0.f;
    for (int w = 0; w < kRingWarps; ++w) t += acc[w * 2 * c + i];
    part[blockIdx.x * 2 * int64_t(c) + i] = t;
  }
}

// ---------------------------------------------------------------------------
// backward, rows of more than a warp
// ---------------------------------------------------------------------------
// As k_norm_bwd, but a row takes G = 64 to 256 threads, each with enough
// vectors of it that loads to registers, one row ahead, keep memory busy.
template <class T, int V, int G, int VECS>
__global__ void __launch_bounds__(kThreads)
k_norm_bwd_wide(const T* __restrict__ x, const float* __restrict__ gamma, const T* __restrict__ dy,
           T* __restrict__ dx, float* __restrict__ part, int64_t n, int c, float inv_c, float eps) {
  rows::let_next_start();  // the join
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
  const int64_t step = int64_t(gridDim.x) * kGroups;
  int64_t base = blockIdx.x * int64_t(kGroups);
  RowShare<T, V, G, VECS> xn, gn;  // the next row, asked for while this one is worked on
  xn.load(x + (base + group) * c, lane, c, base + group < n);
  gn.load(dy + (base + group) * c, lane, c, base + group < n);
  for (; base < n; base += step) {
    const int64_t r = base + group;
    const bool ok = r < n;
    const RowShare<T, V, G, VECS> xs = xn, gs = gn;
    xn.load(x + (r + step) * c, lane, c, r + step < n);
    gn.load(dy + (r + step) * c, lane, c, r + step < n);
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

// Partial sums of dgamma and dbeta: a block takes 256 columns of a row chunk.
// The chunks are in the grid's first dimension, the only one that holds 2^31 rows'.
template <class T>
__global__ void __launch_bounds__(kThreads)
k_norm_cols(const T* x, const T* dy, const float2* stats, float* part, int64_t n, int64_t c) {
  const unsigned strips = unsigned((c + kThreads - 1) / kThreads), chunk = blockIdx.x / strips;
  const int64_t j = blockIdx.x % strips * int64_t(kThreads) + threadIdx.x;
  if (j >= c) return;
  const int64_t r0 = chunk * int64_t(kColRows), r1 = min(n, r0 + kColRows);
  float dg = 0.f, db = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    const float2 st = stats[r];
    const float g = rows::to_float(dy[r * c + j]);
    dg += g * ((rows::to_float(x[r * c + j]) - st.x) * st.y);
    db += g;
  }
  part[(chunk * int64_t(2) + 0) * c + j] = dg;
  part[(chunk * int64_t(2) + 1) * c + j] = db;
}

// dgamma and dbeta from the partial sums: a block takes 32 of the 2 c columns,
// 32 warps each every 32nd partial, then the warps in order.
__global__ void __launch_bounds__(1024)
k_norm_join(const float* __restrict__ part, float* __restrict__ dgamma, float* __restrict__ dbeta,
            int64_t parts, int64_t c) {
  __shared__ float sums[32][33];
  rows::let_next_start();
  rows::after_previous();
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

// How a row of c values is dealt to a group.  The widest vector that divides
// the row; vectors of 8 bytes and more: the narrowest group whose threads hold
// one vector (up to a warp) or up to four; narrower ones, which carry few
// bytes each: a warp with up to 20 a thread, so that the row's sums stay
// shuffles (26,213 rows of 515 fp32 values, backward: 47.6 us with 128 threads
// and block barriers, 33 us with a warp), then 256 threads.
struct Deal {
  int v, g, vecs;  // vecs = 0: the row is too long for registers
};
template <class I>
Deal deal(I c, int elem) {
  Deal d{16 / elem, 1, 0};
  while (c % d.v != 0) d.v /= 2;
  const int64_t vectors = c / d.v;
  const bool narrow = d.v * elem < 8;
  if (!narrow) {
    while (d.g < kThreads && vectors > int64_t(d.g) * (d.g < 32 ? 1 : 4)) d.g *= 2;
    const int64_t need = (vectors + d.g - 1) / d.g;
    if (need <= 4) d.vecs = int(need);
    return d;
  }
  while (d.g < 32 && vectors > d.g) d.g *= 2;
  if (vectors > 32 * 20) d.g = kThreads;
  const int64_t need = (vectors + d.g - 1) / d.g;
  for (int k : {1, 2, 4, 8, 12, 16, 20})
    if (d.vecs == 0 && need <= k && (d.g <= 32 || k <= 8)) d.vecs = k;
  return d;
}

// The backward's ring kernel has the rows in shared memory, where a warp may
// read them in any way: from eight vectors on, two vectors a thread, which
// halves the steps of the sums.
template <class I>
Deal deal_bwd(I c, int elem) {
  Deal d = deal(c, elem);
  const int64_t vectors = c / d.v;
  if (d.v * elem >= 8 && d.g >= 16 && d.g <= 32 && vectors <= 64) {
    d.g = vectors <= 16 ? 8 : (vectors <= 32 ? 16 : 32);
    d.vecs = 2;
  }
  return d;
}

// Whether deal (deal_bwd) gives K vectors of V values to each of G threads for
// any row: kernels exist for these only.  Vectors narrower than 16 bytes come in
// odd numbers, as a wider one would divide the row otherwise.
template <class T, bool BWD>
constexpr bool dealt(int v, int g, int k) {
  if (v * int(sizeof(T)) < 16 && g == 2) return false;
  if (v * int(sizeof(T)) < 8) {
    if (g == 32) return k == 1 || k == 2 || (k % 4 == 0 && k <= 20);
    return g < 32 ? k == 1 : g == kThreads && (k == 4 || k == 8);
  }
  if (g > 32) return k == 3 || k == 4;
  if (BWD && g >= 16) return k == 2 || (g == 32 && (k == 3 || k == 4));
  if (BWD && g == 8) return k <= 2;
  return k == 1 || (g == 32 && k <= 4);
}

// f(V, G, K) as compile-time values.
template <class T, bool BWD, class F>
int by_deal(const Deal& d, F&& f) {
  auto with = [&](auto v, auto g) -> int {
    constexpr int V = decltype(v)::value, G = decltype(g)::value;
    int rc = SMC_ERR_INVALID;
    auto one = [&](auto k) {
      if constexpr (dealt<T, BWD>(V, G, decltype(k)::value))
        if (d.vecs == decltype(k)::value) rc = f(v, g, k);
    };
    one(std::integral_constant<int, 1>());
    one(std::integral_constant<int, 2>());
    one(std::integral_constant<int, 3>());
    one(std::integral_constant<int, 4>());
    one(std::integral_constant<int, 8>());
    one(std::integral_constant<int, 12>());
    one(std::integral_constant<int, 16>());
    one(std::integral_constant<int, 20>());
    return rc;
  };
  auto wide = [&](auto v) -> int {
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

// run(WHOLE): rows that fill every thread's share (`whole`) are the common ones
// and go without masks, from vectors of 8 bytes on.  Shares of one or two vectors
// a row are always full; vectors narrower than 16 bytes, of which there is an odd
// number, fill a share of one only.
template <class T, int V, int G, class F>
int by_fill(bool whole, F&& run) {
  if constexpr (V * sizeof(T) >= 8 && G <= 2) {
    return run(std::true_type());
  } else {
    if constexpr (V * sizeof(T) == 16)
      if (whole) return run(std::true_type());
    return run(std::false_type());
  }
}

// Launch of the backward kernels.  Ring (groups of up to a warp): chunks of the
// fewest whole passes of a warp that hold 1 KB, one or two blocks per SM.  (The
// most passes within 2 KB: 209,715 x 128 fp16 37.6 us, 34.2 so, 200,000 x 96 the
// same 39.6; within 1 KB, one pass where that is 600 to 800 bytes: 96 channels
// 41.5; more slots of 1 KB, 128 channels 37.4 with four, 39 with six.)  Wide
// groups: a few blocks per SM.  Each block leaves one partial sum, and there are
// no more blocks than work.
struct BwdPlan {
  Deal d;
  int chunk_rows = 0, slot_bytes = 0, smem = 0;
  int64_t blocks = 1;
  BwdPlan(int64_t n, int64_t c, int elem) : d(deal_bwd(c, elem)) {
    if (d.vecs == 0) return;
    const int64_t most = int64_t(sm_count());
    if (d.g > 32) {
      const int64_t groups = kThreads / d.g;
      blocks = std::max<int64_t>(1, std::min((n + groups - 1) / groups, most * 4));
      return;
    }
    const int pass = 32 / d.g;
    chunk_rows = pass * int((1024 + pass * c * elem - 1) / (pass * c * elem));
    slot_bytes = int((chunk_rows * c * elem + 15 + 15) / 16 * 16);
    const int values = d.vecs * d.v;
    smem = std::max(kRingWarps * ring_stages(values) * 2 * slot_bytes, kRingWarps * 2 * int(c) * 4);
    const int64_t chunks = (n + chunk_rows - 1) / chunk_rows;
    blocks = std::max<int64_t>(1, std::min((chunks + kRingWarps - 1) / kRingWarps,
                                           most * ring_blocks(values)));
  }
};

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
    return by_deal<T, false>(d, [&](auto v, auto g, auto vecs) {
      constexpr int V = decltype(v)::value, G = decltype(g)::value, K = decltype(vecs)::value;
      const int64_t step = norm_threads<G>() / G * rows_per_group<T, V, K>();
      return by_fill<T, V, G>(c == G * K * V, [&](auto whole) -> int {
        k_norm<T, V, G, K, decltype(whole)::value>
            <<<unsigned((n + step - 1) / step), norm_threads<G>(), 0, s>>>(
                in, gamma, beta, o, n, int(c), 1.f / float(c), eps);
        return launched();
      });
    });
  });
}

int64_t layer_norm_backward_workspace(int64_t n, int64_t c, int dtype) {
  if (n == 0) return 0;
  const BwdPlan p(n, c, dtype == SMC_F32 ? 4 : 2);
  if (p.d.vecs == 0)
    return n * int64_t(sizeof(float2)) + chunks(n) * 2 * c * int64_t(sizeof(float));
  return p.blocks * 2 * c * int64_t(sizeof(float));
}

int layer_norm_backward(const void* x, const float* gamma, const void* dy, void* dx,
                        float* dgamma, float* dbeta, int64_t n, int64_t c, int dtype, float eps,
                        void* workspace, cudaStream_t s) {
  return rows::by_type(dtype, [&](auto tag) {
    using T = decltype(tag);
    const T *in = static_cast<const T*>(x), *g_out = static_cast<const T*>(dy);
    T* g_in = static_cast<T*>(dx);
    const BwdPlan p(n, c, sizeof(T));
    float* part = static_cast<float*>(workspace);
    int64_t parts = 0;
    if (n > 0 && p.d.vecs == 0) {
      float2* stats = static_cast<float2*>(workspace);
      part = reinterpret_cast<float*>(stats + n);
      k_norm_bwd_long<T><<<unsigned(n), kThreads, 0, s>>>(in, gamma, g_out, g_in, stats, c, eps);
      if (launched() != SMC_OK) return int(SMC_ERR_CUDA);
      if (dgamma) {
        parts = chunks(n);
        // n c <= 2^44: at most 2^28 blocks and one more per strip and per chunk
        const int64_t blocks = (c + kThreads - 1) / kThreads * parts;
        k_norm_cols<T><<<unsigned(blocks), kThreads, 0, s>>>(in, g_out, stats, part, n, c);
        if (launched() != SMC_OK) return int(SMC_ERR_CUDA);
      }
    } else if (n > 0) {
      if (dgamma) parts = p.blocks;
      float* to = dgamma ? part : nullptr;
      const int rc = by_deal<T, true>(p.d, [&](auto v, auto g, auto vecs) {
        constexpr int V = decltype(v)::value, G = decltype(g)::value, K = decltype(vecs)::value;
        if constexpr (G > 32) {
          k_norm_bwd_wide<T, V, G, K><<<unsigned(p.blocks), kThreads, 0, s>>>(
              in, gamma, g_out, g_in, to, n, int(c), 1.f / float(c), eps);
          return launched();
        } else {
          return by_fill<T, V, G>(c == G * K * V, [&](auto whole) -> int {
            auto kern = k_norm_bwd<T, V, G, K, decltype(whole)::value>;
            constexpr int kMaxDev = 64;
            static bool attr_set[kMaxDev] = {};  // per device
            int dev = -1;
            if (cudaGetDevice(&dev) != cudaSuccess) return int(SMC_ERR_CUDA);
            if (!(dev >= 0 && dev < kMaxDev && attr_set[dev])) {
              if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       227 * 1024) != cudaSuccess)
                return int(SMC_ERR_CUDA);
              if (dev >= 0 && dev < kMaxDev) attr_set[dev] = true;
            }
            kern<<<unsigned(p.blocks), 32 * kRingWarps, p.smem, s>>>(
                in, gamma, g_out, g_in, to, n, int(c), p.chunk_rows, p.slot_bytes, 1.f / float(c),
                eps);
            return launched();
          });
        }
      });
      if (rc != SMC_OK) return rc;
    }
    if (dgamma)
      return rows::launch_after(true, k_norm_join, dim3(unsigned((2 * c + 31) / 32)), 1024, 0, s,
                                static_cast<const float*>(part), dgamma, dbeta, parts, c);
    return launched();
  });
}

}  // namespace smc
