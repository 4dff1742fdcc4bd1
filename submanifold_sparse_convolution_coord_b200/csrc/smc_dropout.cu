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

template <class T>
__global__ void __launch_bounds__(256)
k_dropout(const T* x, const T* residual, T* out, int64_t count, DropArgs a) {
  uint64_t seed = a.seed, offset = a.offset;
  if (a.state) {
    seed = a.state[0];
    offset += a.state[1];
  }
  const int64_t groups = (count + 7) / 8;
  for (int64_t g = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; g < groups;
       g += int64_t(gridDim.x) * blockDim.x) {
    const uint4 w = philox_4x32_10(make_uint4(uint32_t(g), uint32_t(uint64_t(g) >> 32),
                                              uint32_t(offset), uint32_t(offset >> 32)),
                                   make_uint2(uint32_t(seed), uint32_t(seed >> 32)));
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
    for (int j = 0; j < 8; ++j) {
      const int64_t i = g * 8 + j;
      if (i >= count) break;
      const uint32_t bits = (words[j / 2] >> (16 * (j & 1))) & 0xFFFFu;
      float v = bits >= a.threshold ? rows::to_float(x[i]) * a.scale : 0.f;
      if (residual) v += rows::to_float(residual[i]);
      out[i] = rows::from_float<T>(v);
    }
  }
}

}  // namespace

int dropout(const void* x, const void* residual, void* out, int64_t count, int dtype, double p,
            uint64_t seed, uint64_t offset, const uint64_t* state, cudaStream_t s) {
  DropArgs a{seed, offset, state, uint32_t(std::nearbyint(p * 65536.0)), 0.f};
  if (a.threshold < 65536) a.scale = float(65536.0 / double(65536 - a.threshold));
  return rows::by_type(dtype, [&](auto tag) {
    using T = decltype(tag);
    const int64_t blocks = ((count + 7) / 8 + 255) / 256;
    k_dropout<T><<<unsigned(blocks < 148 * 8 ? blocks : 148 * 8), 256, 0, s>>>(
        static_cast<const T*>(x), static_cast<const T*>(residual), static_cast<T*>(out), count, a);
    return cudaGetLastError() == cudaSuccess ? SMC_OK : SMC_ERR_CUDA;
  });
}

}  // namespace smc
