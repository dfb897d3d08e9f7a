// elems.cuh -- loads and stores of VEC consecutive elements of a row as FP32
// values, for the element kinds the MLP-block operators take: bf16, fp32, and
// 8-bit codes with a scale byte per group of 32.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace mlp {

constexpr int kBf16 = 0, kF32 = 1, kPacked = 2;   // element kinds (0, 1: the LORA_BF16, LORA_F32 codes)

// The step 2^(s - 127) of scale byte s. s = 0 is a subnormal; s = 255, the mark of a group that
// holds a NaN or an infinity, becomes NaN, and so do all the group's values.
__device__ __forceinline__ float scale_step(uint32_t s) {
  return __uint_as_float(s == 0u ? 0x00400000u : (s == 255u ? 0x7FC00000u : s << 23));
}

// The VEC elements as they lie in memory. VEC is 8 (bf16) or 4 (fp32): whole 16-byte loads; 2 (bf16)
// or 1 for rows whose length those do not divide.
template <int KIND, int VEC>
struct Raw;
template <>
struct Raw<kBf16, 8> {
  uint4 v;
  __device__ __forceinline__ void load(const void* p, const void*, int64_t row, int64_t ld, int c) {
    load_at(p, nullptr, row * ld + c);
  }
  __device__ __forceinline__ void load_at(const void* p, const void*, int64_t at) {
    v = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at));
  }
  __device__ __forceinline__ void get(float (&o)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = __uint_as_float(w[i] << 16);
      o[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Raw<kF32, 4> {
  float4 v;
  __device__ __forceinline__ void load(const void* p, const void*, int64_t row, int64_t ld, int c) {
    v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + row * ld + c));
  }
  __device__ __forceinline__ void get(float (&o)[4]) const { o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w; }
};
template <>
struct Raw<kBf16, 1> {
  uint16_t v;
  __device__ __forceinline__ void load(const void* p, const void*, int64_t row, int64_t ld, int c) {
    v = __ldg(static_cast<const uint16_t*>(p) + row * ld + c);
  }
  __device__ __forceinline__ void get(float (&o)[1]) const { o[0] = __uint_as_float(uint32_t(v) << 16); }
};
template <>
struct Raw<kBf16, 2> {
  uint32_t v;
  __device__ __forceinline__ void load(const void* p, const void*, int64_t row, int64_t ld, int c) {
    v = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p) + row * ld + c));
  }
  __device__ __forceinline__ void get(float (&o)[2]) const {
    o[0] = __uint_as_float(v << 16);
    o[1] = __uint_as_float(v & 0xFFFF0000u);
  }
};
template <>
struct Raw<kF32, 1> {
  float v;
  __device__ __forceinline__ void load(const void* p, const void*, int64_t row, int64_t ld, int c) {
    v = __ldg(static_cast<const float*>(p) + row * ld + c);
  }
  __device__ __forceinline__ void get(float (&o)[1]) const { o[0] = v; }
};
// Packed: `ld` codes (a multiple of 32) and ld / 32 scale bytes a row; a vector never crosses a group.
template <int VEC>
struct Raw<kPacked, VEC> {
  uint32_t w[(VEC + 3) / 4];
  uint8_t s;
  __device__ __forceinline__ void load(const void* p, const void* scales, int64_t row, int64_t ld, int c) {
    load_at(p, scales, row * ld + c);
  }
  // from code `at` of the storage (rows of ld codes one after the other, a scale byte every 32)
  __device__ __forceinline__ void load_at(const void* p, const void* scales, int64_t at) {
    const int8_t* q = static_cast<const int8_t*>(p) + at;
    if constexpr (VEC == 8) {
      const uint2 t = __ldg(reinterpret_cast<const uint2*>(q));
      w[0] = t.x;
      w[1] = t.y;
    } else if constexpr (VEC == 4) {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(q));
    } else if constexpr (VEC == 2) {
      w[0] = __ldg(reinterpret_cast<const uint16_t*>(q));
    } else {
      w[0] = uint32_t(uint8_t(__ldg(q)));
    }
    s = __ldg(static_cast<const uint8_t*>(scales) + (at >> 5));
  }
  __device__ __forceinline__ void get(float (&o)[VEC]) const {
    const float step = scale_step(s);
    if constexpr (VEC >= 4) {
      // a code as FP32: 2^23 + (code + 128) has the byte at the bottom, and the difference is exact
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        o[i] = (__uint_as_float(__byte_perm(w[i / 4] ^ 0x80808080u, 0x4B000000u, 0x7440u + i % 4)) - 8388736.f) * step;
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] = float(int8_t(w[0] >> (8 * i))) * step;
    }
  }
};

// Elements per row of the storage: the row length, or the padded length of packed rows.
template <int KIND>
__device__ __forceinline__ int64_t row_ld(int64_t n) {
  return KIND == kPacked ? ((n + 31) & ~int64_t(31)) : n;
}

// One value of a vector of parameters (bf16 or fp32, `type`).
__device__ __forceinline__ float param_at(const void* p, int type, int64_t i) {
  return type == kBf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}
// VEC consecutive ones, c a multiple of VEC.
template <int VEC>
__device__ __forceinline__ void params_at(const void* p, int type, int c, float (&o)[VEC]) {
  if constexpr (VEC < 4) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) o[i] = param_at(p, type, c + i);
  } else if (type == kBf16) {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const uint2 t = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + c) + i);
      o[4 * i] = __uint_as_float(t.x << 16);
      o[4 * i + 1] = __uint_as_float(t.x & 0xFFFF0000u);
      o[4 * i + 2] = __uint_as_float(t.y << 16);
      o[4 * i + 3] = __uint_as_float(t.y & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const float4 t = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + c) + i);
      o[4 * i] = t.x;
      o[4 * i + 1] = t.y;
      o[4 * i + 2] = t.z;
      o[4 * i + 3] = t.w;
    }
  }
}

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
// Stores VEC values (rounded once, to nearest even) at element i of an output that nothing in the
// same kernel reads again.
template <int KIND, int VEC>
__device__ __forceinline__ void store_vec(void* p, int64_t i, const float (&v)[VEC]) {
  if constexpr (KIND == kBf16 && VEC == 8) {
    uint4 t = make_uint4(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]),
                         bf16x2_bits(v[6], v[7]));
    __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i), t);
  } else if constexpr (KIND == kBf16 && VEC == 2) {
    *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p) + i) = bf16x2_bits(v[0], v[1]);
  } else if constexpr (KIND == kBf16) {
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v[0]);
  } else if constexpr (VEC == 4) {
    __stcs(reinterpret_cast<float4*>(static_cast<float*>(p) + i), make_float4(v[0], v[1], v[2], v[3]));
  } else {
    static_cast<float*>(p)[i] = v[0];
  }
}

}  // namespace mlp
