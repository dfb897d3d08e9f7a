// pack8.cuh -- the 8-bit form of a group of 32 FP32 values: scale byte and codes.
#pragma once

#include <stdint.h>

namespace mlp {

// The scale byte s of a group from the bits of its largest |x| (NaN bits compare above infinity's,
// which compare above every number's): the smallest s with |x| <= 127.5 * 2^(s - 127), or 255 for a
// NaN or an infinity. For |x| = f * 2^E with f in [1, 2), that is E - 6, one more when f > 127.5 / 64.
// At most 248: at 249 a code of 64 would stand for 2^128, so the few numbers above 127.5 * 2^121 are
// held to 127 * 2^121 instead, and what was finite stays finite.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  const uint32_t E = amax_bits >> 23;
  if (E == 255u) return 255u;
  const int s = int(E) - 6 + ((amax_bits & 0x7FFFFFu) > 0x7F0000u ? 1 : 0);
  return s > 0 ? uint32_t(s < 248 ? s : 248) : 0u;
}

// 1 / step of scale byte s <= 248, exactly: 2^(127 - s). (s = 255: 0, all codes of the group are 0.)
__device__ __forceinline__ float inv_step(uint32_t s) { return s == 255u ? 0.f : __uint_as_float((254u - s) << 23); }

// The code of x, one multiplication by a power of two and one rounding to nearest even away from
// x / step; 127.5 steps, a tie that would round to 128, is held to 127.
__device__ __forceinline__ int code_of(float x, float inv, uint32_t s) {
  const int q = s == 255u ? 0 : __float2int_rn(x * inv);
  return q > 127 ? 127 : (q < -127 ? -127 : q);
}

}  // namespace mlp
