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
