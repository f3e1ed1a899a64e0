// Element formats of the KV cache: the working type, or one byte per element
// (int8 or e4m3) with a scale per block of tokens and kv head.
#pragma once

#include <cuda_fp8.h>

#include "kernels.h"

namespace ccgqa {

// 8 codes <-> 8 fp32 code values (scale not applied).  int8: the byte, plus 128,
// in the low mantissa bits of 2^23, and 1.5 2^23 added to round: neither needs the
// slow integer conversions.
template <int FMT>
__device__ __forceinline__ void decode8(uint2 w, float (&x)[8]) {
  const uint32_t u[2] = {w.x, w.y};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (FMT == kCacheI8) {
      const uint32_t b = u[h] ^ 0x80808080u;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[h * 4 + i] = __uint_as_float(__byte_perm(b, 0x4b000000u, 0x7440 + i)) - 8388736.0f;   // 2^23 + 128
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(u[h] >> (16 * i)), __NV_E4M3);
        const float2 f = __half22float2(__half2(r));
        x[h * 4 + 2 * i] = f.x;
        x[h * 4 + 2 * i + 1] = f.y;
      }
    }
  }
}

// Rounds to the nearest code, ties to even; past the largest code, the largest.
template <int FMT>
__device__ __forceinline__ uint2 encode8(const float (&x)[8]) {
  uint32_t u[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (FMT == kCacheI8) {
      uint32_t b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        b[i] = __float_as_uint(fminf(fmaxf(x[h * 4 + i], -127.0f), 127.0f) + 12582912.0f);
      u[h] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    } else {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[h * 4], x[h * 4 + 1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[h * 4 + 2], x[h * 4 + 3]), __NV_SATFINITE, __NV_E4M3);
      u[h] = lo | hi << 16;
    }
  }
  return make_uint2(u[0], u[1]);
}

}  // namespace ccgqa
