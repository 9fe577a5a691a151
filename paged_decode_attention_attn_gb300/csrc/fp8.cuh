// e4m3 conversions (sm_103a): 4 significant bits, largest value 448, smallest
// subnormal 2^-9, one NaN code per sign (0x7f / 0xff), no infinities.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

namespace pa {
namespace fp8 {

// Two fp32 values to e4m3 (nearest even, saturating at 448; NaN stays NaN);
// `lo` lands in the low byte.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// The same from fp16.
__device__ __forceinline__ uint32_t pack2(__half2 x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;"
      : "=h"(r)
      : "r"(*reinterpret_cast<const uint32_t*>(&x)));
  return r;
}

__device__ __forceinline__ uint32_t pack4(__half2 x, __half2 y) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f16x2 lo, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 hi, %2;\n\tmov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "r"(*reinterpret_cast<const uint32_t*>(&x)), "r"(*reinterpret_cast<const uint32_t*>(&y)));
  return r;
}

// Two e4m3 codes to fp16 (exact), to fp32.
__device__ __forceinline__ __half2 unpack2_half(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
  return *reinterpret_cast<const __half2*>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t codes) {
  return __half22float2(unpack2_half(codes));
}

__device__ __forceinline__ void unpack4(uint32_t codes, float (&y)[4]) {
  const float2 a = unpack2(codes & 0xffffu), b = unpack2(codes >> 16);
  y[0] = a.x;
  y[1] = a.y;
  y[2] = b.x;
  y[3] = b.y;
}

// Four codes times `by`, rounded to e4m3 again.
__device__ __forceinline__ uint32_t scale4(uint32_t codes, float by) {
  float y[4];
  unpack4(codes, y);
  return pack4(y[0] * by, y[1] * by, y[2] * by, y[3] * by);
}

}  // namespace fp8
}  // namespace pa
