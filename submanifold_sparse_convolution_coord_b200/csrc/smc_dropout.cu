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

// One round and the key schedule of Philox-4x32 (Salmon, Moraes, Dror and
// Shaw, SC 2011): two 32 x 32 -> 64 bit products, their high words mixed with
// the other two words and the key.
__device__ __forceinline__ uint4 philox_4x32_10(uint4 c, uint2 k) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = uint64_t(0xD2511F53u) * c.x, b = uint64_t(0xCD9E8D57u) * c.z;
    c = make_uint4(uint32_t(b >> 32) ^ c.y ^ k.x, uint32_t(b), uint32_t(a >> 32) ^ c.w ^ k.y,
                   uint32_t(a));
    k.x += 0x9E3779B9u;
    k.y += 0xBB67AE85u;
  }
  return c;
}

struct DropArgs {
  uint64_t seed, offset;
  const uint64_t* state;
  uint32_t threshold;  // keep an element when its 16 bits are >= this
  float scale;
};

// A group of eight elements as 16-byte pieces.
template <class T>
struct alignas(16) Group {
  T v[8];
};

// One counter, so eight elements, per thread, in blocks that leave room for the
// SM's 2,048 threads: their loads in flight cover the generator's arithmetic
// (about 115 instructions a group against 48 bytes with a residual).  Measured
// on 209,715 x 512 bf16 with a residual: 117 us (5.5 TB/s); two groups a thread
// without that bound took 158 us, with it 119.  RES: with a residual.
constexpr int kThreads = 256;
template <class T, bool RES>
__global__ void __launch_bounds__(kThreads, 2048 / kThreads)
k_dropout(const T* x, const T* residual, T* out, int64_t count, DropArgs a) {
  uint64_t seed = a.seed, offset = a.offset;
  if (a.state) {
    seed = a.state[0];
    offset += a.state[1];
  }
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
  const uint4 w = philox_4x32_10(
      make_uint4(uint32_t(g), uint32_t(uint64_t(g) >> 32), uint32_t(offset),
                 uint32_t(offset >> 32)),
      make_uint2(uint32_t(seed), uint32_t(seed >> 32)));
  const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t bits = j & 1 ? words[j / 2] >> 16 : words[j / 2] & 0xFFFFu;
    float v = bits >= a.threshold ? rows::to_float(xs.v[j]) * a.scale : 0.f;
    if constexpr (RES) v += rows::to_float(rs.v[j]);
    o.v[j] = rows::from_float<T>(v);
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
  DropArgs a{seed, offset, state, uint32_t(std::nearbyint(p * 65536.0)), 0.f};
  if (a.threshold < 65536) a.scale = float(65536.0 / double(65536 - a.threshold));
  return rows::by_type(dtype, [&](auto tag) {
    using T = decltype(tag);
    const int64_t per_block = 8 * kThreads;
    const unsigned blocks = unsigned((count + per_block - 1) / per_block);
    const T *in = static_cast<const T*>(x), *res = static_cast<const T*>(residual);
    if (res)
      k_dropout<T, true><<<blocks, kThreads, 0, s>>>(in, res, static_cast<T*>(out), count, a);
    else
      k_dropout<T, false><<<blocks, kThreads, 0, s>>>(in, res, static_cast<T*>(out), count, a);
    return cudaGetLastError() == cudaSuccess ? SMC_OK : SMC_ERR_CUDA;
  });
}

}  // namespace smc
