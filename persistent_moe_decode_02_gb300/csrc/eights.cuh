// 8-bit values: e4m3 codes with a power-of-two scale for several of them.
#pragma once
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

namespace mk {

constexpr int GROUP = 32;        // values of a row that share a scale (mk_norm, mk_quantize, mk_experts_*)

// Smallest k with amax <= 448 * 2^k (448 = 0.875 * 2^9, the largest e4m3
// value), from the bits of amax: exact, no rounding of a logarithm.
__device__ __forceinline__ int scale_exp(float amax) {
  if (amax == 0.f) return -127;
  int e;
  const float m = frexpf(amax, &e);              // amax = m 2^e, m in [0.5, 1)
  if (!isfinite(amax)) return 127;
  const int k = m <= 0.875f ? e - 9 : e - 8;
  return k < -127 ? -127 : k;
}

__device__ __forceinline__ float pow2(int k) { return __int_as_float((k + 127) << 23); }   // k in [-126, 127]

// Four values by 2^-k as codes, the first in the lowest byte; in two factors:
// 2^127 and beyond is no factor of its own.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float f, float g) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a * f * g, b * f * g), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c * f * g, d * f * g), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}
struct Factors {
  float f, g;
};
__device__ __forceinline__ Factors factors(int k) { return {pow2(-(k >> 1)), pow2(-(k - (k >> 1)))}; }

}  // namespace mk
