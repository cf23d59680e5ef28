// kvq_fp8.cuh: the FP8 pool's elements. A block of 16 tokens of one kv head
// holds e4m3 codes c and one scale byte e; a code stands for c * 2^(e - 127),
// and every code of a block with e = 0 for zero.
//
// Why a power of two: an e4m3 value has the same relative step over its whole
// range, so a scale need not be finer than a factor of two; raising it by a
// power of two moves codes exactly (all but those that reach the subnormals),
// which is what a block that fills token by token does; and the kernels apply
// it by an exponent, with no rounding.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace kvq {

// The value of one unit of a block's codes.
__device__ __forceinline__ float fp8_scale(uint32_t e) { return __uint_as_float(e << 23); }

// The smallest scale byte that holds |x| <= amax without saturating (448 is
// e4m3's largest value): the smallest e >= 1 with amax <= 448 * 2^(e - 127);
// 0 for amax = 0. amax = 1.m * 2^q fits 1.75 * 2^8 * 2^(e - 127) when
// e = q - 8 + 127, one more where 1.m > 1.75. bits: amax as fp32 bits.
__device__ __forceinline__ uint32_t fp8_scale_for(uint32_t bits) {
  if (bits == 0u) return 0u;
  const int e = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(e < 1 ? 1 : e);
}

// Two codes of a word (bytes 0 and 1, or 2 and 3) as an fp16 pair, exactly.
__device__ __forceinline__ uint32_t e4m3_lo_to_f16(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}"
      : "=r"(r)
      : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_hi_to_f16(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, hi;\n}"
      : "=r"(r)
      : "r"(w));
  return r;
}

// x and y rounded to the nearest e4m3 (ties to even; beyond 448 to 448, NaN
// to NaN), x in the low byte.
__device__ __forceinline__ uint32_t f32_to_e4m3(float x, float y) {
  uint32_t r;
  asm("{\n .reg .b16 c;\n cvt.rn.satfinite.e4m3x2.f32 c, %2, %1;\n cvt.u32.u16 %0, c;\n}"
      : "=r"(r)
      : "f"(x), "f"(y));
  return r;
}

}  // namespace kvq
