// The 8-bit cache format: rows of e4m3 codes with one power-of-two exponent
// byte each (a code c stands for c * 2^(byte - 127)).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

namespace pkv {
namespace quant {

constexpr int kExpMin = -31, kExpMax = 31, kExpBias = 127;

// 2^e for -126 <= e <= 127: the exponent field of an fp32 number.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// The power of two that an exponent byte stands for; bytes that no write stores
// (a slot that was never written) count as the nearer bound.
__device__ __forceinline__ int clamp_exp(int byte) {
  return max(kExpMin + kExpBias, min(kExpMax + kExpBias, byte)) - kExpBias;
}

// Exponent of a row whose largest finite magnitude has the bf16 bits `a`: the
// smallest e with a <= 448 * 2^e = 1.75 * 2^(e + 8), clamped.  With a = 1.f *
// 2^x that is x - 8, or x - 7 when the fraction is above .75 (96 / 128).  A
// subnormal or zero a lands far below the clamp.
__device__ __forceinline__ int row_exponent(uint32_t a) {
  const int e = static_cast<int>(a >> 7) - 127 - 8 + ((a & 0x7Fu) > 96u ? 1 : 0);
  return max(kExpMin, min(kExpMax, e));
}

// Two fp32 -> two e4m3 codes (lo in bits 0-7), nearest even, held at +-448;
// NaN -> 0x7F.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two e4m3 codes (the low or high half of a word) -> two fp16, exactly: every
// e4m3 value, subnormals included, is a normal fp16 number or zero; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(codes));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(codes));
  return r;
}

}  // namespace quant
}  // namespace pkv
