// e4m3.cuh -- e4m3 codes with a power-of-two scale, shared by the quantiser and the norm.
#pragma once
#include <cuda_fp8.h>
#include <stdint.h>

namespace vsa {

// Smallest e with a <= 448 * 2^e for a > 0 (0 for 0): 448 = 1.75 * 2^8, so e is a's exponent - 8, one more
// when a's mantissa is above 1.75.
__device__ __forceinline__ int e4m3_block_exponent(float a) {
  if (!(a > 0.f)) return 0;
  const bool small = a < 1.17549435e-38f;  // subnormal: scaled up by 2^32
  const int bits = __float_as_int(small ? a * 4294967296.f : a);
  return ((bits + 0x1fffff) >> 23) - 135 - (small ? 32 : 0);
}

// Division by 2^e for |e| < 252 as one or two products with normal powers of two (2^-e itself may be out of
// range).  Exact for every result that is not far below the smallest code.
struct E4m3Scale {
  float a, b;
  bool twice;
  __device__ explicit E4m3Scale(int e) : twice(e < -126 || e > 126) {
    const int h = twice ? e / 2 : e;
    a = __int_as_float((127 - h) << 23);
    b = __int_as_float((127 - (e - h)) << 23);
  }
  __device__ float operator()(float x) const { return twice ? x * a * b : x * a; }
};

// Two codes (nearest even, saturating at 448), the first in the low byte.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3) & 0xffffu;
}

}  // namespace vsa
