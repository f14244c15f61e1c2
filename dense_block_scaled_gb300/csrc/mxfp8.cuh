// mxfp8.cuh -- the MXFP8 number format on the device: E4M3 codes, one E8M0 scale per 32.
#pragma once
#include <cuda_fp16.h>

#include <cstdint>

namespace tkg {

// Two FP32 -> E4M3 (RNE, saturating); `lo` lands in the low byte.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two E4M3 codes (the low 16 bits) -> FP32, exactly.
__device__ __forceinline__ float2 e4m3x2_values(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(codes)));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// Value 2^(code - 127) of an E8M0 code; 2^-127 is subnormal, 255 is NaN.
__device__ __forceinline__ float e8m0_value(uint32_t code) {
  return __uint_as_float(code == 0 ? 0x00400000u : (code == 255 ? 0x7fc00000u : code << 23));
}

// MXFP8 scale exponent: smallest e with 448 * 2^e >= amax, clamped to [-127, 127].
// With amax = M * 2^E (M in [1, 2)), 448 = 1.75 * 2^8, that is
// e = E - 8 + (M > 1.75); subnormal or zero amax gives -127.
__device__ __forceinline__ int mx_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int eb = int((u >> 23) & 0xFFu);
  if (eb == 0) return -127;
  int e = (eb - 127) - 8 + (((u & 0x7FFFFFu) > 0x600000u) ? 1 : 0);
  return e < -127 ? -127 : (e > 127 ? 127 : e);
}

}  // namespace tkg
