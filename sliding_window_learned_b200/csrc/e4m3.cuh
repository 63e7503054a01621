// e4m3.cuh -- the 8-bit cache's number format: e4m3 codes under a power-of-two
// scale (e8m0) for each row of D channels (one position of one kv head, K or V).
//
//   e    = the smallest integer in [-117, 119] with max|x| <= 448 * 2^e, over the
//          row's finite x; scale byte = e + 127
//   code = x * 2^-e rounded to e4m3, nearest even (the product is exact in f32)
//
// A power of two costs no accuracy against a scale of max|x| / 448: e4m3 is a
// floating-point format, so its relative step (2^-4 at most half of it) does not
// depend on where in the range a value falls, and only the subnormal end moves
// by less than one binade.  In return code * 2^e is exact in bf16 and f32, the
// scale takes one byte, and every implementation gets the same bits.  The
// limits of e keep code * 2^e exact in bf16 (the smallest code is 2^-9) and
// finite; a magnitude above 448 * 2^119 (only the top binade of bf16) saturates.
// NaN and infinities become the NaN code (e4m3 has no infinity), so that they
// stay visible; they do not enter the row's maximum.
#pragma once
#include <stdint.h>

namespace attnsink {

constexpr int kScaleExpMin = -117, kScaleExpMax = 119;

// Scale byte of a row from its largest finite magnitude, given as bf16 bits
// without the sign.  448 = 1.75 * 2^8.
__device__ __forceinline__ int row_scale_byte(uint32_t amax_bf16) {
  const int e = static_cast<int>(amax_bf16 >> 7) - 127 - 8 + ((amax_bf16 & 0x7Fu) > 0x60u ? 1 : 0);
  return min(max(e, kScaleExpMin), kScaleExpMax) + 127;
}

// 2^(127 - byte): what a row is multiplied by before the rounding (exact; the
// byte is in [10, 246]).
__device__ __forceinline__ float row_inv_scale(int byte) {
  return __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);
}

// The value of a scale byte: 2^(byte - 127), 0 gives the subnormal 2^-127, 255
// NaN.  (Bytes outside [10, 246] are never written here, but a pool may hold
// anything.)
__device__ __forceinline__ float scale_value(uint32_t byte) {
  const uint32_t odd = byte == 0u ? 0x00400000u : 0x7FC00000u;
  return __uint_as_float(byte - 1u < 254u ? byte << 23 : odd);
}

// Two f32 to two e4m3 codes (low byte first), nearest even, saturating; NaN
// gives the NaN code.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four e4m3 codes (low byte first) to two f16 pairs; exact, NaN stays NaN.
__device__ __forceinline__ uint2 e4m3x4_to_f16x2x2(uint32_t w) {
  uint2 h;
  asm("{.reg .b16 lo, hi; mov.b32 {lo, hi}, %2; cvt.rn.f16x2.e4m3x2 %0, lo; cvt.rn.f16x2.e4m3x2 %1, hi;}"
      : "=r"(h.x), "=r"(h.y)
      : "r"(w));
  return h;
}

}  // namespace attnsink
