// Element formats of the KV cache: the working type, or one byte per element
// (int8 or e4m3) with a scale per block of tokens and kv head.
#pragma once

#include <cuda_fp8.h>

#include "kernels.h"

namespace ccgqa {

// 8 codes <-> 8 fp32 code values (scale not applied).
template <int FMT>
__device__ __forceinline__ void decode8(uint2 w, float (&x)[8]) {
  const uint32_t u[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t byte = (u[i >> 2] >> ((i & 3) * 8)) & 0xffu;
    if constexpr (FMT == kCacheI8) {
      x[i] = static_cast<float>(static_cast<int8_t>(byte));
    } else {
      __nv_fp8_e4m3 f;
      f.__x = static_cast<__nv_fp8_storage_t>(byte);
      x[i] = static_cast<float>(f);
    }
  }
}

// Rounds to the nearest code, ties to even; past the largest code, the largest.
template <int FMT>
__device__ __forceinline__ uint32_t encode1(float x) {
  if constexpr (FMT == kCacheI8) {
    const int q = min(max(__float2int_rn(x), -127), 127);   // NaN converts to 0
    return static_cast<uint32_t>(q) & 0xffu;
  } else {
    return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
  }
}
template <int FMT>
__device__ __forceinline__ uint2 encode8(const float (&x)[8]) {
  uint32_t u[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i >> 2] |= encode1<FMT>(x[i]) << ((i & 3) * 8);
  return make_uint2(u[0], u[1]);
}

}  // namespace ccgqa
