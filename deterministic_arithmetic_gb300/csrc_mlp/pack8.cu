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
// out, and back.
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

// K a multiple of 8: a thread takes 8 consecutive elements, four neighbouring lanes a group.
template <int KIND>
__global__ void __launch_bounds__(256)
    pack8_kernel(const void* __restrict__ x, int64_t M, int K, int G, uint2* __restrict__ codes,
                 uint8_t* __restrict__ scales) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t items = M * G * 4;       // a multiple of 4: the lanes of a group stay together
  for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < items; i += int64_t(gridDim.x) * blockDim.x) {
    const int64_t row = i / (G * 4);
    const int c = int(i - row * (G * 4)) * 8;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
    if (c < K) {
      if constexpr (KIND == kBf16) {
        Raw<kBf16, 8> r;
        r.load(x, nullptr, row, K, c);
        r.get(v);
      } else {
        Raw<kF32, 4> a, b;
        a.load(x, nullptr, row, K, c);
        b.load(x, nullptr, row, K, c + 4);
        a.get(reinterpret_cast<float(&)[4]>(v[0]));
        b.get(reinterpret_cast<float(&)[4]>(v[4]));
      }
    }
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, abs_bits(v[e]));
    const unsigned quad = 0xFu << (threadIdx.x & 28u);
    m = max(m, __shfl_xor_sync(quad, m, 1));
    m = max(m, __shfl_xor_sync(quad, m, 2));
    const uint32_t s = scale_byte(m);
    const float inv = inv_step(s);
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e / 4] |= (uint32_t(code_of(v[e], inv, s)) & 0xFFu) << (8 * (e % 4));
    codes[i] = make_uint2(w[0], w[1]);
    if ((threadIdx.x & 3) == 0) scales[i >> 2] = uint8_t(s);
  }
}

// Any K: a warp takes a group, a lane an element.
template <int KIND>
__global__ void __launch_bounds__(256)
    pack8_any_kernel(const void* __restrict__ x, int64_t M, int K, int G, int8_t* __restrict__ codes,
                     uint8_t* __restrict__ scales) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int lane = threadIdx.x & 31;
  const int64_t items = M * G;
  for (int64_t i = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; i < items;
       i += int64_t(gridDim.x) * blockDim.x >> 5) {
    const int64_t row = i / G;
    const int c = int(i - row * G) * kGroup + lane;
    float v[1] = {0.f};
    if (c < K) {
      Raw<KIND, 1> r;
      r.load(x, nullptr, row, K, c);
      r.get(v);
    }
    const uint32_t s = scale_byte(__reduce_max_sync(0xffffffffu, abs_bits(v[0])));
    codes[i * kGroup + lane] = int8_t(code_of(v[0], inv_step(s), s));
    if (lane == 0) scales[i] = uint8_t(s);
  }
}

// VEC elements a thread (K a multiple of VEC).
template <int KIND, int VEC>
__global__ void __launch_bounds__(256)
    unpack8_kernel(const void* __restrict__ codes, const void* __restrict__ scales, int64_t M, int K,
                   void* __restrict__ out) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t ld = row_ld<kPacked>(K);
  const int per = K / VEC;
  const int64_t items = M * per;
  for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < items; i += int64_t(gridDim.x) * blockDim.x) {
    const int64_t row = i / per;
    const int c = int(i - row * per) * VEC;
    Raw<kPacked, VEC> r;
    float v[VEC];
    r.load(codes, scales, row, ld, c);
    r.get(v);
    store_vec<KIND, VEC>(out, row * K + c, v);
  }
}

// CTAs of 256 threads for a grid-stride loop over `items` threads' work.
unsigned stride_grid(int64_t items, int nsm) {
  const int64_t want = cdiv(items, 256), most = int64_t(nsm) * 32;
  return unsigned(want < most ? want : most);
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
  const int k = int(K), G = int(groups(K));
  cudaError_t e;
  if (K % 8 == 0) {
    const dim3 grid(stride_grid(M * G * 4, nsm));
    uint2* q = static_cast<uint2*>(codes);
    e = x_type == LORA_BF16 ? launch_pdl(pack8_kernel<kBf16>, grid, dim3(256), 0, st, x, M, k, G, q, static_cast<uint8_t*>(scales))
                            : launch_pdl(pack8_kernel<kF32>, grid, dim3(256), 0, st, x, M, k, G, q, static_cast<uint8_t*>(scales));
  } else {
    const dim3 grid(stride_grid(M * G * 32, nsm));
    int8_t* q = static_cast<int8_t*>(codes);
    e = x_type == LORA_BF16 ? launch_pdl(pack8_any_kernel<kBf16>, grid, dim3(256), 0, st, x, M, k, G, q, static_cast<uint8_t*>(scales))
                            : launch_pdl(pack8_any_kernel<kF32>, grid, dim3(256), 0, st, x, M, k, G, q, static_cast<uint8_t*>(scales));
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
  const int k = int(K), vec = out_type == LORA_BF16 ? (K % 8 == 0 ? 8 : 1) : (K % 4 == 0 ? 4 : 1);
  const dim3 grid(stride_grid(M * (K / vec), nsm));
  cudaError_t e;
  if (out_type == LORA_BF16)
    e = vec == 8 ? launch_pdl(unpack8_kernel<kBf16, 8>, grid, dim3(256), 0, st, codes, scales, M, k, out)
                 : launch_pdl(unpack8_kernel<kBf16, 1>, grid, dim3(256), 0, st, codes, scales, M, k, out);
  else
    e = vec == 4 ? launch_pdl(unpack8_kernel<kF32, 4>, grid, dim3(256), 0, st, codes, scales, M, k, out)
                 : launch_pdl(unpack8_kernel<kF32, 1>, grid, dim3(256), 0, st, codes, scales, M, k, out);
  return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

}  // extern "C"
