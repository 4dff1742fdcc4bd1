// Dropout from a counter-based generator, with the residual sum of a block's
// end: out = residual + keep * x * scale.  The mask is never stored; the
// backward pass draws it again from the same counters.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "smc_internal.h"
#include "smc_rows.cuh"

namespace smc {
namespace {

using rows::add2;
using rows::dup2;
using rows::mul2;

constexpr int kRounds = 10;

struct DropArgs {
  uint2 key[kRounds];  // the key of each round (without `state`)
  uint64_t offset;
  const uint64_t* state;
  uint32_t threshold;  // an element is kept when its bits, as the upper half of
                       // a word, are >= this; and
  bool live;           // p rounds to less than 1
  float scale;
};

__host__ __device__ inline uint2 round_key(uint64_t seed, int r) {
  return make_uint2(uint32_t(seed) + uint32_t(r) * 0x9E3779B9u,
                    uint32_t(seed >> 32) + uint32_t(r) * 0xBB67AE85u);
}

// One round of Philox-4x32 (Salmon, Moraes, Dror and Shaw, SC 2011): two
// 32 x 32 -> 64 bit products, their high words mixed with the other two words
// and the key.
__device__ __forceinline__ uint4 philox_round(uint4 c, uint2 k) {
  const uint64_t a = uint64_t(0xD2511F53u) * c.x, b = uint64_t(0xCD9E8D57u) * c.z;
  return make_uint4(uint32_t(b >> 32) ^ c.y ^ k.x, uint32_t(b), uint32_t(a >> 32) ^ c.w ^ k.y,
                    uint32_t(a));
}

// A group of eight elements as 16-byte pieces.
template <class T>
struct alignas(16) Group {
  T v[8];
};

template <class T>
__device__ __forceinline__ float2 pair_of(const Group<T>& g, int j) {
  if constexpr (sizeof(T) == 4)
    return make_float2(g.v[2 * j], g.v[2 * j + 1]);
  else
    return rows::unpack2<T>(reinterpret_cast<const uint32_t*>(g.v)[j]);
}

// One counter, so eight elements, per thread, in blocks that leave room for the
// SM's 2,048 threads: their loads in flight cover the generator's arithmetic.
// That arithmetic is what comes next to the memory: with the keys of the rounds
// computed per thread, values one by one and the bits shifted down it was 228
// instructions a group, and 209,715 x 512 bf16 with a residual took 115 us (issue
// slots 76 % used); with the keys as arguments, values in pairs and the bits
// compared where they lie 99 us, 6.5 TB/s.  RES: with a residual; STATE: with
// `state`.
constexpr int kThreads = 256;
template <class T, bool RES, bool STATE>
__global__ void __launch_bounds__(kThreads, 2048 / kThreads)
k_dropout(const T* x, const T* residual, T* out, int64_t count,
          const __grid_constant__ DropArgs a) {
  const int64_t g = blockIdx.x * int64_t(kThreads) + threadIdx.x;
  if (g * 8 >= count) return;
  const bool whole = g * 8 + 8 <= count;
  Group<T> xs, rs, o;
  if (whole) {
    xs = reinterpret_cast<const Group<T>*>(x)[g];
    if constexpr (RES) rs = reinterpret_cast<const Group<T>*>(residual)[g];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {  // the last elements, one by one
      const bool in = g * 8 + j < count;
      xs.v[j] = in ? x[g * 8 + j] : rows::from_float<T>(0.f);
      if constexpr (RES) rs.v[j] = in ? residual[g * 8 + j] : rows::from_float<T>(0.f);
    }
  }
  uint64_t offset = a.offset, seed = 0;
  if constexpr (STATE) {
    seed = a.state[0];
    offset += a.state[1];
  }
  uint4 w = make_uint4(uint32_t(g), uint32_t(uint64_t(g) >> 32), uint32_t(offset),
                       uint32_t(offset >> 32));
#pragma unroll
  for (int r = 0; r < kRounds; ++r) w = philox_round(w, STATE ? round_key(seed, r) : a.key[r]);
  const uint32_t words[4] = {w.x, w.y, w.z, w.w};
  float2 v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 y = mul2(pair_of(xs, j), dup2(a.scale));
    v[j].x = a.live && (words[j] << 16) >= a.threshold ? y.x : 0.f;
    v[j].y = a.live && words[j] >= a.threshold ? y.y : 0.f;
    if constexpr (RES) v[j] = add2(v[j], pair_of(rs, j));
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (sizeof(T) == 4) {
      o.v[2 * j] = v[j].x;
      o.v[2 * j + 1] = v[j].y;
    } else {
      reinterpret_cast<uint32_t*>(o.v)[j] = rows::pack2_of<T>(v[j]);
    }
  }
  if (whole) {
    reinterpret_cast<Group<T>*>(out)[g] = o;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (g * 8 + j < count) out[g * 8 + j] = o.v[j];
  }
}

}  // namespace

int dropout(const void* x, const void* residual, void* out, int64_t count, int dtype, double p,
            uint64_t seed, uint64_t offset, const uint64_t* state, cudaStream_t s) {
  DropArgs a = {};
  for (int r = 0; r < kRounds; ++r) a.key[r] = round_key(seed, r);
  a.offset = offset;
  a.state = state;
  const uint32_t t = uint32_t(std::nearbyint(p * 65536.0));
  a.live = t < 65536;
  a.threshold = a.live ? t << 16 : 0;
  a.scale = a.live ? float(65536.0 / double(65536 - t)) : 0.f;
  return rows::by_type(dtype, [&](auto tag) {
    using T = decltype(tag);
    const int64_t per_block = 8 * kThreads;
    const unsigned blocks = unsigned((count + per_block - 1) / per_block);
    const T *in = static_cast<const T*>(x), *res = static_cast<const T*>(residual);
    auto kern = res ? (state ? k_dropout<T, true, true> : k_dropout<T, true, false>)
                    : (state ? k_dropout<T, false, true> : k_dropout<T, false, false>);
    kern<<<blocks, kThreads, 0, s>>>(in, res, static_cast<T*>(out), count, a);
    return cudaGetLastError() == cudaSuccess ? SMC_OK : SMC_ERR_CUDA;
  });
}

}  // namespace smc
