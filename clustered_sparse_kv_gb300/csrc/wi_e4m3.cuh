// wi_e4m3.cuh -- 8-bit values and their groups' scales: conversions shared by the paged cache's kernels.
#pragma once
#include <cuda_fp16.h>

#include "wi_common.cuh"
#include "wi_paged.h"

// Two e4m3 values (low byte first) as f16: exact, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo;\n\tcvt.u16.u32 lo, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(w));
  return h;
}
// Eight of them, the halves of a word named as they are (masked and shifted out of it, an instruction each in front of a
// conversion, a tile's attention took 1.1% more).
__device__ __forceinline__ uint4 e4m3x8_to_f16x8(uint32_t a, uint32_t b) {
  uint4 h;
  asm("{\n\t.reg .b16 p, q, r, s;\n\tmov.b32 {p, q}, %4;\n\tmov.b32 {r, s}, %5;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, p;\n\tcvt.rn.f16x2.e4m3x2 %1, q;\n\tcvt.rn.f16x2.e4m3x2 %2, r;\n\tcvt.rn.f16x2.e4m3x2 %3, s;\n\t}"
      : "=r"(h.x), "=r"(h.y), "=r"(h.z), "=r"(h.w)
      : "r"(a), "r"(b));
  return h;
}
__device__ __forceinline__ float2 e4m3x2_to_f32x2(uint32_t w) {
  const uint32_t h = e4m3x2_to_f16x2(w);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Two fp32 values rounded to e4m3, to nearest; beyond 448 they saturate, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
  uint32_t w;
  asm("{\n\t.reg .b16 x;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\tcvt.u32.u16 %0, x;\n\t}" : "=r"(w) : "f"(lo), "f"(hi));
  return w;
}
__device__ __forceinline__ uint32_t e4m3x2_of_f16x2(uint32_t h) {
  uint32_t w;
  asm("{\n\t.reg .b16 x;\n\tcvt.rn.satfinite.e4m3x2.f16x2 x, %1;\n\tcvt.u32.u16 %0, x;\n\t}" : "=r"(w) : "r"(h));
  return w;
}
__device__ __forceinline__ uint32_t e4m3x4_of(float a, float b, float c, float d) {
  return e4m3x2_of(a, b) | e4m3x2_of(c, d) << 16;
}

// 2^e for -127 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(e > -127 ? (uint32_t)(e + 127) << 23 : 0x00400000u); }

// A scale's exponent from its byte (255, no number, is taken as 2^127).
__device__ __forceinline__ int scale_exponent(unsigned char b) { return min((int)b, 254) - kScaleBias; }
// The exponent of the smallest power of two with which a group's largest value (fp32 bits, sign off) is 448 = 1.75 * 2^8
// at most: the sum carries into the exponent where the mantissa is above 1.75's.
__device__ __forceinline__ int scale_needed(uint32_t top) {
  return max((int)((top + 0x1FFFFFu) >> 23) - 127 - 8, kScaleLowest);
}
