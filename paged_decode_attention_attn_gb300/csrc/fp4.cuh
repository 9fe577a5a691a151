// e2m1 conversions (sm_103a): a sign, two exponent bits of bias 1 and a fraction
// bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6; no infinities, no NaN.  Scales are bytes e that
// stand for 2^(e - 127), 255 for NaN.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

namespace pa {
namespace fp4 {

constexpr int kNanScale = 255, kScaleBias = 127;
constexpr int kMinScaleExp = -60;   // of the scales written

// Eight fp32 values to e2m1 (nearest even, saturating at 6), y[0] in the low bits.
__device__ __forceinline__ uint32_t pack8(const float (&y)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}

// Eight codes to fp16 (exact): byte i of the word, low code first, in h[i].
__device__ __forceinline__ void unpack8(uint32_t codes, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
}
__device__ __forceinline__ void unpack8(uint32_t codes, float (&y)[8]) {
  uint32_t h[4];
  unpack8(codes, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    y[2 * i] = f.x;
    y[2 * i + 1] = f.y;
  }
}

// log2 of the smallest scale s >= 2^-60 with amax <= 6 s (6 = 1.5 * 4), from the bits
// of a finite amax >= 0.
__device__ __forceinline__ int scale_exp(unsigned amax_bits) {
  const int e = (int)(amax_bits >> 23) - 127 - 2 + ((amax_bits & 0x7fffffu) > 0x400000u ? 1 : 0);
  return max(e, kMinScaleExp);
}

// What a scale's byte stands for.
__device__ __forceinline__ float scale_of(unsigned byte) {
  if (byte == 0) return __uint_as_float(0x00400000u);   // 2^-127, a subnormal
  return byte == kNanScale ? __int_as_float(0x7fc00000) : __uint_as_float(byte << 23);
}

}  // namespace fp4
}  // namespace pa
