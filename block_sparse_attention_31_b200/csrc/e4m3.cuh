// e4m3.cuh -- e4m3 codes with a power-of-two scale, shared by the quantiser and the norm.
#pragma once
#include <cuda_fp8.h>
#include <stdint.h>

namespace vsa {

// Smallest e with a <= 448 * 2^e for a > 0: with a = f * 2^E, f in [0.5, 1), and
// 448 = 0.875 * 2^9, that is E - 9 when f <= 0.875 and E - 8 otherwise.
__device__ __forceinline__ int e4m3_block_exponent(float amax) {
  if (!(amax > 0.f)) return 0;
  int E;
  const float f = frexpf(amax, &E);
  return f <= 0.875f ? E - 9 : E - 8;
}

// Division by 2^e, exact but for results below the normal range.
struct E4m3Scale {
  float inv;
  int e;
  bool plain;  // 2^-e is a normal float
  __device__ explicit E4m3Scale(int exponent)
      : inv(1.f), e(exponent), plain(exponent >= -127 && exponent <= 126) {
    if (plain) inv = __int_as_float((127 - e) << 23);
  }
  __device__ float operator()(float x) const { return plain ? x * inv : ldexpf(x, -e); }
};

// Two codes (nearest even, saturating at 448), the first in the low byte.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3) & 0xffffu;
}

}  // namespace vsa
