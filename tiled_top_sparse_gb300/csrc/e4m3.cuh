// e4m3 codes and the power-of-two scales of the grouped-query cache's pages.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace tts {

constexpr uint32_t kMinScaleExp = 127 - 60;

// Smallest power of two s >= 2^-60 with amax <= 448 s (448 = 1.75 * 2^8); amax finite, >= 0.
__device__ __forceinline__ float block_scale(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return __uint_as_float((uint32_t)(e > (int)kMinScaleExp ? e : (int)kMinScaleExp) << 23);
}

__device__ __forceinline__ float finite_abs(float x) {  // 0 for inf and NaN: they set no scale
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;
}

// Two values to e4m3 (nearest even, saturating), lo in the low byte.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 codes (low byte first) to floats, exactly.
__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  float2 f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

}  // namespace tts
