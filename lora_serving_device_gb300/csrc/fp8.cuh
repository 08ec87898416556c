// e4m3 codes and their scales (the cache in 8 bits).
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace lora {

constexpr int kScaleBlock = 16;  // tokens of a scale, in pages of 16 and more

// Scale bytes are 1 .. 253, so that a scale and its inverse are normal numbers; others
// read as the nearest of them.  Byte b stands for 2^(b - 127).
__device__ __forceinline__ int scale_read(int b) { return b < 1 ? 1 : b > 253 ? 253 : b; }
__device__ __forceinline__ float scale_of(int b) {
  return __uint_as_float(static_cast<uint32_t>(b) << 23);
}

// The byte of the least power of two that a block whose largest magnitude is `top` fits
// under with 448 codes: top = 1.f x 2^E needs 2^(E - 8) up to 1.75 x 2^E.
__device__ __forceinline__ int scale_byte(float top) {
  const uint32_t u = __float_as_uint(top);
  const int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < 1 ? 1 : e;
}

// Four values to codes, round to nearest even, saturating at 448.
__device__ __forceinline__ uint32_t pack4_e4m3(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}
__device__ __forceinline__ float2 unpack2_e4m3(uint32_t two) {
  return __half22float2(__half2(
      __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xffffu), __NV_E4M3)));
}

// Eight codes as f16, exactly, times f2 (a power of two, twice).
__device__ __forceinline__ void widen4_e4m3(uint32_t four, uint32_t f2, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t.reg .b32 x, y;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 x, a;\n\tcvt.rn.f16x2.e4m3x2 y, b;\n\t"
      "mul.rn.f16x2 %0, x, %3;\n\tmul.rn.f16x2 %1, y, %3;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four), "r"(f2));
}
__device__ __forceinline__ uint4 widen8_e4m3(uint32_t a, uint32_t b, uint32_t f2) {
  uint4 y;
  widen4_e4m3(a, f2, y.x, y.y);
  widen4_e4m3(b, f2, y.z, y.w);
  return y;
}
// Two fp32 rounded to f16.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t y;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
  return y;
}

// Four f16 (magnitudes up to 448) as the sum of two e4m3 terms.
__device__ __forceinline__ void split4_e4m3(uint32_t a, uint32_t b, uint32_t& t1, uint32_t& t2) {
  asm("{\n\t.reg .b16 p, q;\n\t.reg .b32 x, y;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 p, %2;\n\tcvt.rn.satfinite.e4m3x2.f16x2 q, %3;\n\t"
      "mov.b32 %0, {p, q};\n\t"
      "cvt.rn.f16x2.e4m3x2 x, p;\n\tcvt.rn.f16x2.e4m3x2 y, q;\n\t"
      "sub.rn.f16x2 x, %2, x;\n\tsub.rn.f16x2 y, %3, y;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 p, x;\n\tcvt.rn.satfinite.e4m3x2.f16x2 q, y;\n\t"
      "mov.b32 %1, {p, q};\n\t}"
      : "=&r"(t1), "=r"(t2)
      : "r"(a), "r"(b));
}

}  // namespace lora
