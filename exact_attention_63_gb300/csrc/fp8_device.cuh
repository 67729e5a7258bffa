// E4M3 codes with a power-of-two scale for each block of 16 slots and key head.
//
// A code c of a block whose exponent byte is b stands for c·2^(b − 127).  The byte is kept
// between 10 and 246 (2^−117 … 2^119): the codes' smallest step is 2^−9 and their largest
// value 448, so every value is a bf16 number, none is subnormal and none overflows.  With
// powers of two a scale loses nothing of a code's four significant bits, and rows that get
// a larger scale later are exact unless they fall below the codes' normal range.
#pragma once

#include <cstdint>

#include "cache_launch.h"

namespace attn {

__device__ __forceinline__ int scale_byte(uint8_t b) {
  return min(max(static_cast<int>(b), kFp8Lowest), kFp8Highest);
}
// 2^(e − 127) of a byte as a float, e in [1, 254].
__device__ __forceinline__ float power_of(int e) { return __uint_as_float(static_cast<uint32_t>(e) << 23); }

// The smallest byte e with |x| ≤ 448·2^(e − 127), clamped, of the bits of a finite bf16
// |x|: 448 is 1.75·2^8.
__device__ __forceinline__ int byte_for(uint32_t bits) {
  const int e = static_cast<int>(bits >> 7) - 8 + ((bits & 0x7Fu) > 0x60u);
  return min(max(e, kFp8Lowest), kFp8Highest);
}

// Codes of two floats, to nearest even; beyond ±448 the largest code, NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two codes as f16 numbers (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
__device__ __forceinline__ void f16x2_to_f32(uint32_t h, float& lo, float& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}

}  // namespace attn
