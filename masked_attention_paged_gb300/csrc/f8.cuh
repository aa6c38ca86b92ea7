// f8.cuh -- e4m3 codes and the power-of-two scales of an e4m3 KV cache.
#pragma once

#include <stdint.h>

namespace attn {

// The exponent of the smallest power of two that brings a (finite, > 0) to 448 = 1.75 *
// 2^8 or below, from its bits; at least -126.
__device__ __forceinline__ int f8_scale_exponent(float a) {
  const uint32_t u = __float_as_uint(a);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -126 ? -126 : e;  // (a subnormal a too)
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Two codes, of `lo` in bits 0..7: rounded to nearest even, +-448 past the range, NaN for NaN.
__device__ __forceinline__ uint32_t f8_codes(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// The two values as an fp16 pair (exact).
__device__ __forceinline__ uint32_t f8_half2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}
__device__ __forceinline__ void half2_f32(uint32_t x, float& lo, float& hi) {
  asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(x));
}

// bytes that are NaN codes, as 0x80 each
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

}  // namespace attn
