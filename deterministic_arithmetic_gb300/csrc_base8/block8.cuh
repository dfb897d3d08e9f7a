// block8.cuh -- the 8-bit form of a block: its power-of-two scale from the largest magnitude, and e4m3 codes.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace mlp {

constexpr int kBlock = 128;                        // columns (of weights also rows) of a block

// Elements of a row of codes.
__host__ __device__ constexpr int64_t code_ld(int64_t k) { return (k + 15) & ~int64_t(15); }

// The scale of a block from the bits of its largest |x| (NaN bits compare above infinity's, which
// compare above every number's). |x| = f * 2^E with f in [1, 2), and 448 = 1.75 * 2^8: the smallest 2^e
// with |x| <= 448 * 2^e has e = E - 8, one more when f > 1.75. From 2^-124, so that the smallest code, 2^-9,
// stands for bf16's smallest value, to 2^119, so that the largest, 448, stays finite.
struct BlockScale {
  float scale, inv;                                // inv = 1 / scale exactly; 0 in a block that is not finite
};
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return {__uint_as_float(0x7FC00000u), 0.f};
  const int e = int(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  const int c = max(-124, min(119, e));
  return {__uint_as_float(uint32_t(127 + c) << 23), __uint_as_float(uint32_t(127 - c) << 23)};
}

// Two codes: v * inv is exact but for what lies below the smallest code, then one rounding to nearest even,
// held to +-448. inv = 0: zeros (v may be infinite or NaN).
__device__ __forceinline__ uint32_t codes2(float a, float b, float inv) {
  const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(a * inv, b * inv), __NV_SATFINITE, __NV_E4M3);
  return inv == 0.f ? 0u : c;
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float inv) {
  return codes2(a, b, inv) | (codes2(c, d, inv) << 16);
}
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
  return make_uint2(codes4(v[0], v[1], v[2], v[3], inv), codes4(v[4], v[5], v[6], v[7], inv));
}

// The two e4m3 values in the low 16 bits, exactly.
__device__ __forceinline__ float2 values2(uint32_t w) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w), __NV_E4M3);
  return __half22float2(__half2(h));
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

}  // namespace mlp
