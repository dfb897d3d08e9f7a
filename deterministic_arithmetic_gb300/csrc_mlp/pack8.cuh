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

// Four codes in a word: x times 1 / step (exact), held to +-127 (127.5 steps, a tie, would round to
// 128), and one rounding to nearest even: 1.5 * 2^23 + v has round(v) in its low bits, two's
// complement. NaN and infinity: s = 255, whose codes are 0.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float inv, uint32_t s) {
  const float v[4] = {a, b, c, d};
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = __float_as_uint(fminf(fmaxf(v[i] * inv, -127.f), 127.f) + 12582912.f);
  const uint32_t w = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
  return s == 255u ? 0u : w;
}

}  // namespace mlp
