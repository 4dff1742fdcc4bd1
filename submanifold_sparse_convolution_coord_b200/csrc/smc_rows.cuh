// Helpers of the row operators (layer norm, dropout, gated feed-forward):
// element conversions and the dispatch over element types.  Internal header,
// not part of the C ABI.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "smc_internal.h"

namespace smc {
namespace rows {

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// Round to nearest even.
template <class T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __half from_float<__half>(float v) {
  return __float2half_rn(v);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Pairs of floats: one instruction for two of them (add, multiply, multiply-add
// on 64-bit register pairs), for kernels whose arithmetic counts next to their
// memory traffic or their matrix products.
__device__ __forceinline__ uint64_t bits2(float2 v) { return *reinterpret_cast<uint64_t*>(&v); }
__device__ __forceinline__ float2 float2_of(uint64_t v) { return *reinterpret_cast<float2*>(&v); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return float2_of(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return float2_of(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return float2_of(r);
}
__device__ __forceinline__ float2 dup2(float v) { return make_float2(v, v); }

// Two 16-bit values of a word, low half first.
template <class T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Two floats rounded to a word of two 16-bit values.
template <class T>
__device__ __forceinline__ uint32_t pack2_of(float2 v);
template <>
__device__ __forceinline__ uint32_t pack2_of<__half>(float2 v) {
  const __half2 h = __float22half2_rn(v);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2_of<__nv_bfloat16>(float2 v) {
  const __nv_bfloat162 h = __float22bfloat162_rn(v);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A kernel of a chain may be placed on the GPU while the one before it in the
// stream runs out (launch_after): it sets itself up, and waits with
// after_previous() before it touches memory that another kernel may use.
// let_next_start() lets the next one of the chain be placed likewise.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// early = false: an ordinary launch.
template <class... P, class... A>
int launch_after(bool early, void (*kernel)(P...), dim3 grid, int threads, size_t smem,
                 cudaStream_t s, A... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(unsigned(threads));
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &attr;
  c.numAttrs = early ? 1 : 0;
  if (cudaLaunchKernelEx(&c, kernel, P(args)...) != cudaSuccess) {
    cudaGetLastError();
    return SMC_ERR_CUDA;
  }
  return SMC_OK;
}

// f(T()) for the element type T of an smc_dtype.
template <class F>
int by_type(int dtype, F&& f) {
  switch (dtype) {
    case SMC_F32:
      return f(float());
    case SMC_F16:
      return f(__half());
    case SMC_BF16:
      return f(__nv_bfloat16());
    default:
      return SMC_ERR_INVALID;
  }
}

}  // namespace rows
}  // namespace smc
