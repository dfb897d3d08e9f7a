// pack8.cu -- activation checkpoints in 8 bits: packing and unpacking.
//
// The form (include/lora_mlp.h): groups of 32 along the row, a power-of-two step
// per group, codes of 7 bits and a sign. The step is a power of two so that the
// value a code stands for is a bf16 value exactly: the tensor cores take it as
// an operand with nothing lost after the one rounding at packing, and packing a
// value that was unpacked gives the same codes again. A free scale would gain at
// most one bit of the seven and cost a second rounding in every consumer.
//
// Packing and unpacking are bound by HBM: x once in, 33 / 32 bytes an element
// out, and back. 8192 x 4096 bf16: 17.6 us (5.8 TB/s) and 11.4 us (codes partly
// from L2).
#include "../csrc/common.cuh"
#include "../csrc/kernels.h"
#include "elems.cuh"
#include "mlp.h"
#include "pack8.cuh"

namespace mlp {
namespace {

using lora::grid_dependency_wait;
using lora::grid_dependents_launch;
using lora::launch_pdl;

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// A thread's 8 consecutive elements of a row: loaded, their largest magnitude's bits, packed with the
// other three lanes of their group.
template <int KIND>
struct Octet;
template <>
struct Octet<kBf16> {
  uint4 r;
  __device__ __forceinline__ void clear() { r = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void load(const void* x, int64_t i) {
    r = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(x) + i));
  }
  __device__ __forceinline__ uint32_t amax() const {   // bf16 bits order as their values do
    const uint32_t m = __vmaxu2(__vmaxu2(r.x & 0x7FFF7FFFu, r.y & 0x7FFF7FFFu), __vmaxu2(r.z & 0x7FFF7FFFu, r.w & 0x7FFF7FFFu));
    return max(m << 16, m & 0xFFFF0000u);
  }
  __device__ __forceinline__ uint2 codes(float inv, uint32_t s) const {
    return make_uint2(pair4(r.x, r.y, inv, s), pair4(r.z, r.w, inv, s));
  }
  static __device__ __forceinline__ uint32_t pair4(uint32_t a, uint32_t b, float inv, uint32_t s) {
    return codes4(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u), __uint_as_float(b << 16),
                  __uint_as_float(b & 0xFFFF0000u), inv, s);
  }
};
template <>
struct Octet<kF32> {
  float4 a, b;
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const void* x, int64_t i) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + i);
    a = __ldcs(p);
    b = __ldcs(p + 1);
  }
  __device__ __forceinline__ uint32_t amax() const {
    const uint32_t m = max(max(abs_bits(a.x), abs_bits(a.y)), max(abs_bits(a.z), abs_bits(a.w)));
    return max(m, max(max(abs_bits(b.x), abs_bits(b.y)), max(abs_bits(b.z), abs_bits(b.w))));
  }
  __device__ __forceinline__ uint2 codes(float inv, uint32_t s) const {
    return make_uint2(codes4(a.x, a.y, a.z, a.w, inv, s), codes4(b.x, b.y, b.z, b.w, inv, s));
  }
};

constexpr int kDeep = 4;               // vectors a thread has in flight

// K a multiple of 8: a thread takes 8 consecutive elements, four neighbouring lanes a group, kDeep
// groups apart at a time. FLAT (K a multiple of 32): no group is padded, so x is one long row.
template <int KIND, bool FLAT>
__global__ void __launch_bounds__(256)
    pack8_kernel(const void* __restrict__ x, int64_t items, uint32_t K, uint32_t per_row, uint2* __restrict__ codes,
                 uint8_t* __restrict__ scales) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t first = int64_t(blockIdx.x) * (256 * kDeep) + threadIdx.x;
  Octet<KIND> v[kDeep];
#pragma unroll
  for (int j = 0; j < kDeep; ++j) {
    const int64_t i = first + 256 * j;
    v[j].clear();
    if (i < items) {
      if constexpr (FLAT) {
        v[j].load(x, 8 * i);
      } else {
        const int64_t row = i / per_row;
        const uint32_t c = uint32_t(i - row * per_row) * 8;
        if (c < K) v[j].load(x, row * K + c);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kDeep; ++j) {
    const int64_t i = first + 256 * j;
    uint32_t m = v[j].amax();            // items is a multiple of 4: the lanes of a group go together
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t s = scale_byte(m);
    if (i < items) {
      codes[i] = v[j].codes(inv_step(s), s);
      if ((threadIdx.x & 3) == 0) scales[i >> 2] = uint8_t(s);
    }
  }
}

// Any K: a warp takes a group, a lane an element.
template <int KIND>
__global__ void __launch_bounds__(256)
    pack8_any_kernel(const void* __restrict__ x, int64_t groups, uint32_t K, uint32_t per_row, int8_t* __restrict__ codes,
                     uint8_t* __restrict__ scales) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int lane = threadIdx.x & 31;
  const int64_t first = int64_t(blockIdx.x) * (8 * kDeep) + (threadIdx.x >> 5);
  float v[kDeep];
#pragma unroll
  for (int j = 0; j < kDeep; ++j) {
    const int64_t i = first + 8 * j;
    v[j] = 0.f;
    if (i < groups) {
      const int64_t row = i / per_row;
      const uint32_t c = uint32_t(i - row * per_row) * kGroup + lane;
      if (c < K) v[j] = param_at(x, KIND, row * K + c);
    }
  }
#pragma unroll
  for (int j = 0; j < kDeep; ++j) {
    const int64_t i = first + 8 * j;
    if (i >= groups) continue;
    const uint32_t s = scale_byte(__reduce_max_sync(0xffffffffu, abs_bits(v[j])));
    codes[i * kGroup + lane] = int8_t(codes4(v[j], 0.f, 0.f, 0.f, inv_step(s), s));
    if (lane == 0) scales[i] = uint8_t(s);
  }
}

// VEC elements a thread (K a multiple of VEC). FLAT (K a multiple of 32): one long row.
template <int KIND, int VEC, bool FLAT>
__global__ void __launch_bounds__(256)
    unpack8_kernel(const void* __restrict__ codes, const void* __restrict__ scales, int64_t items, uint32_t K,
                   uint32_t per_row, void* __restrict__ out) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t first = int64_t(blockIdx.x) * (256 * kDeep) + threadIdx.x;
  const int64_t ld = row_ld<kPacked>(K);
  Raw<kPacked, VEC> r[kDeep];
#pragma unroll
  for (int j = 0; j < kDeep; ++j) {
    const int64_t i = first + 256 * j;
    if (i < items) {
      if constexpr (FLAT) {
        r[j].load_at(codes, scales, i * VEC);
      } else {
        const int64_t row = i / per_row;
        r[j].load_at(codes, scales, row * ld + uint32_t(i - row * per_row) * VEC);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kDeep; ++j) {
    const int64_t i = first + 256 * j;
    if (i < items) {                     // the rows of the output lie one after the other: element i VEC
      float v[VEC];
      r[j].get(v);
      store_vec<KIND, VEC>(out, i * VEC, v);
    }
  }
}

}  // namespace
}  // namespace mlp

using namespace mlp;

extern "C" {

lora_status lora_pack8(const void* x, int x_type, int64_t M, int64_t K, void* codes, void* scales, void* stream) {
  if (!size_ok(M) || !size_ok(K) || K < 1 || !type_ok(x_type)) return LORA_ERR_SHAPE;
  if (M == 0) return LORA_OK;
  lora_status s = check_ptrs(x, codes, scales);
  if (s != LORA_OK) return s;
  int nsm = 0;
  if ((s = device_ready(&nsm)) != LORA_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const uint32_t k = uint32_t(K), G = uint32_t(groups(K));
  uint8_t* sc = static_cast<uint8_t*>(scales);
  cudaError_t e;
  if (K % 8 == 0) {
    const int64_t items = M * G * 4;
    const dim3 grid(unsigned(cdiv(items, 256 * kDeep)));
    auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(256), 0, st, x, items, k, 4 * G, static_cast<uint2*>(codes), sc); };
    const bool flat = K % kGroup == 0;
    e = x_type == LORA_BF16 ? (flat ? go(pack8_kernel<kBf16, true>) : go(pack8_kernel<kBf16, false>))
                            : (flat ? go(pack8_kernel<kF32, true>) : go(pack8_kernel<kF32, false>));
  } else {
    const dim3 grid(unsigned(cdiv(M * G, 8 * kDeep)));
    auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(256), 0, st, x, M * G, k, G, static_cast<int8_t*>(codes), sc); };
    e = x_type == LORA_BF16 ? go(pack8_any_kernel<kBf16>) : go(pack8_any_kernel<kF32>);
  }
  return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

lora_status lora_unpack8(const void* codes, const void* scales, int64_t M, int64_t K, void* out, int out_type,
                         void* stream) {
  if (!size_ok(M) || !size_ok(K) || K < 1 || !type_ok(out_type)) return LORA_ERR_SHAPE;
  if (M == 0) return LORA_OK;
  lora_status s = check_ptrs(codes, scales, out);
  if (s != LORA_OK) return s;
  int nsm = 0;
  if ((s = device_ready(&nsm)) != LORA_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int vec = out_type == LORA_BF16 ? (K % 8 == 0 ? 8 : 1) : (K % 4 == 0 ? 4 : 1);
  const int64_t per_row = K / vec, items = M * per_row;
  const dim3 grid(unsigned(cdiv(items, 256 * kDeep)));
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(256), 0, st, codes, scales, items, uint32_t(K), uint32_t(per_row), out);
  };
  cudaError_t e;
  if (K % kGroup == 0) e = out_type == LORA_BF16 ? go(unpack8_kernel<kBf16, 8, true>) : go(unpack8_kernel<kF32, 4, true>);
  else if (vec > 1) e = out_type == LORA_BF16 ? go(unpack8_kernel<kBf16, 8, false>) : go(unpack8_kernel<kF32, 4, false>);
  else e = out_type == LORA_BF16 ? go(unpack8_kernel<kBf16, 1, false>) : go(unpack8_kernel<kF32, 1, false>);
  return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

}  // extern "C"
