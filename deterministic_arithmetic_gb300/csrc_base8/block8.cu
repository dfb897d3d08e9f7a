// block8.cu -- tensors in 8-bit blocks of 128 (lora_block8, lora_unblock8 of include/lora_base8.h).
//
// One pass: a block's elements are read once into registers, their largest magnitude is found by shuffles (and,
// for a weight's 128 x 128, through shared memory), and the codes are written. Bound by HBM: 3 bytes an element of
// a bf16 tensor.
#include "../csrc/common.cuh"
#include "../csrc/kernels.h"
#include "../csrc_mlp/elems.cuh"
#include "base8.h"
#include "block8.cuh"

namespace mlp {
namespace {

using lora::grid_dependency_wait;
using lora::grid_dependents_launch;
using lora::launch_pdl;

// 8 consecutive elements of a row that starts on a 16-byte boundary.
template <int KIND>
struct Eight;
template <>
struct Eight<kBf16> {
  Raw<kBf16, 8> r;
  __device__ __forceinline__ void load(const void* p, int64_t at) { r.load_at(p, nullptr, at); }
  __device__ __forceinline__ void get(float (&v)[8]) const { r.get(v); }
  __device__ __forceinline__ void clear() { r.v = make_uint4(0, 0, 0, 0); }
};
template <>
struct Eight<kF32> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    a = __ldg(q);
    b = __ldg(q + 1);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
};

__device__ __forceinline__ uint32_t amax8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
  return m;
}

// Blocks of one row, K a multiple of 8: 16 lanes a block, 8 elements a lane, DEEP blocks of a half warp in flight.
// Item i of the grid is vector i & 15 of block i >> 4, blocks row by row.
template <int KIND, int DEEP>
__global__ void __launch_bounds__(256)
    block8_rows_kernel(const void* __restrict__ x, int64_t blocks, uint32_t K, uint32_t per_row,
                       uint8_t* __restrict__ codes, float* __restrict__ scales) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t first = int64_t(blockIdx.x) * (16 * DEEP) + (threadIdx.x >> 4);
  const uint32_t lane = threadIdx.x & 15u, ld = uint32_t(code_ld(K));
  Eight<KIND> r[DEEP];
  int64_t row[DEEP];
  uint32_t col[DEEP];
#pragma unroll
  for (int j = 0; j < DEEP; ++j) {
    const int64_t b = first + 16 * j;
    r[j].clear();
    row[j] = b / per_row;
    col[j] = uint32_t(b - row[j] * per_row) * kBlock + 8 * lane;
    if (b < blocks && col[j] < K) r[j].load(x, row[j] * K + col[j]);
  }
#pragma unroll
  for (int j = 0; j < DEEP; ++j) {
    const int64_t b = first + 16 * j;
    float v[8];
    r[j].get(v);
    uint32_t m = amax8(v);
#pragma unroll
    for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const BlockScale s = block_scale(m);
    if (b < blocks && col[j] < ld) *reinterpret_cast<uint2*>(codes + row[j] * ld + col[j]) = codes8(v, s.inv);
    if (b < blocks && lane == 0) scales[b] = s.scale;
  }
}

// Any K: a warp a block, its elements 32 apart.
template <int KIND>
__global__ void __launch_bounds__(256)
    block8_rows_any_kernel(const void* __restrict__ x, int64_t blocks, uint32_t K, uint32_t per_row,
                           uint8_t* __restrict__ codes, float* __restrict__ scales) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t b = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (b >= blocks) return;
  const uint32_t lane = threadIdx.x & 31u, ld = uint32_t(code_ld(K));
  const int64_t row = b / per_row;
  const uint32_t c0 = uint32_t(b - row * per_row) * kBlock + lane;
  float v[4];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = c0 + 32 * j < K ? param_at(x, KIND, row * K + c0 + 32 * j) : 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) m = max(m, abs_bits(v[j]));
  const BlockScale s = block_scale(__reduce_max_sync(0xffffffffu, m));
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (c0 + 32 * j < ld) codes[row * ld + c0 + 32 * j] = uint8_t(codes2(v[j], 0.f, s.inv));
  if (lane == 0) scales[b] = s.scale;
}

// The largest over the CTA's 256 threads.
__device__ __forceinline__ uint32_t cta_max(uint32_t m) {
  __shared__ uint32_t part[8];
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31u) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, part[i]);
  return m;
}

// Blocks of 128 x 128, a CTA each: 16 lanes a row of a block, 16 rows at a time.
template <int KIND>
__global__ void __launch_bounds__(256)
    block8_tiles_kernel(const void* __restrict__ x, int64_t M, uint32_t K, uint8_t* __restrict__ codes,
                        float* __restrict__ scales) {
  grid_dependency_wait();
  grid_dependents_launch();
  const uint32_t per_row = (K + kBlock - 1) / kBlock, ld = uint32_t(code_ld(K));
  const int64_t rb = blockIdx.x / per_row;
  const uint32_t cb = uint32_t(blockIdx.x - rb * per_row), col = cb * kBlock + 8 * (threadIdx.x & 15u);
  const int64_t row0 = rb * kBlock + (threadIdx.x >> 4);
  Eight<KIND> r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    r[j].clear();
    if (row0 + 16 * j < M && col < K) r[j].load(x, (row0 + 16 * j) * K + col);
  }
  uint32_t m = 0;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    r[j].get(v);
    m = max(m, amax8(v));
  }
  const BlockScale s = block_scale(cta_max(m));
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    r[j].get(v);
    if (row0 + 16 * j < M && col < ld) *reinterpret_cast<uint2*>(codes + (row0 + 16 * j) * ld + col) = codes8(v, s.inv);
  }
  if (threadIdx.x == 0) scales[blockIdx.x] = s.scale;
}

// Any K: 128 threads a row, two rows at a time.
template <int KIND>
__global__ void __launch_bounds__(256)
    block8_tiles_any_kernel(const void* __restrict__ x, int64_t M, uint32_t K, uint8_t* __restrict__ codes,
                            float* __restrict__ scales) {
  grid_dependency_wait();
  grid_dependents_launch();
  const uint32_t per_row = (K + kBlock - 1) / kBlock, ld = uint32_t(code_ld(K));
  const int64_t rb = blockIdx.x / per_row;
  const uint32_t cb = uint32_t(blockIdx.x - rb * per_row), col = cb * kBlock + (threadIdx.x & 127u);
  const int64_t row0 = rb * kBlock + (threadIdx.x >> 7);
  float v[64];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 64; ++j) v[j] = row0 + 2 * j < M && col < K ? param_at(x, KIND, (row0 + 2 * j) * K + col) : 0.f;
#pragma unroll
  for (int j = 0; j < 64; ++j) m = max(m, abs_bits(v[j]));
  const BlockScale s = block_scale(cta_max(m));
#pragma unroll
  for (int j = 0; j < 64; ++j)
    if (row0 + 2 * j < M && col < ld) codes[(row0 + 2 * j) * ld + col] = uint8_t(codes2(v[j], 0.f, s.inv));
  if (threadIdx.x == 0) scales[blockIdx.x] = s.scale;
}

// The values: VEC (8, or 1 for rows that vectors do not fit) elements a thread, DEEP times.
template <int KIND, int VEC, int DEEP>
__global__ void __launch_bounds__(256)
    unblock8_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scales, int tile_log2, int64_t items,
                    uint32_t K, uint32_t per_row, void* __restrict__ out) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t first = int64_t(blockIdx.x) * (256 * DEEP) + threadIdx.x, ld = code_ld(K);
  const uint32_t cblocks = (K + kBlock - 1) / kBlock;
  uint2 c[DEEP];
  float s[DEEP];
#pragma unroll
  for (int j = 0; j < DEEP; ++j) {
    const int64_t i = first + 256 * j;
    if (i < items) {
      const int64_t row = i / per_row;
      const uint32_t col = uint32_t(i - row * per_row) * VEC;
      const uint8_t* at = codes + row * ld + col;
      if constexpr (VEC == 8) c[j] = __ldg(reinterpret_cast<const uint2*>(at));
      else c[j].x = __ldg(at);
      s[j] = __ldg(scales + (row >> tile_log2) * cblocks + col / kBlock);
    }
  }
#pragma unroll
  for (int j = 0; j < DEEP; ++j) {
    const int64_t i = first + 256 * j;
    if (i >= items) continue;
    if constexpr (VEC == 1) {
      const float v[1] = {values2(c[j].x).x * s[j]};
      store_vec<KIND, 1>(out, i, v);
    } else {
      float v[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = values2(((k < 2 ? c[j].x : c[j].y) >> (16 * (k & 1))) & 0xFFFFu);
        v[2 * k] = f.x * s[j];
        v[2 * k + 1] = f.y * s[j];
      }
      if constexpr (KIND == kBf16) {
        store_vec<kBf16, 8>(out, 8 * i, v);
      } else {
        const float a[4] = {v[0], v[1], v[2], v[3]}, b[4] = {v[4], v[5], v[6], v[7]};
        store_vec<kF32, 4>(out, 8 * i, a);
        store_vec<kF32, 4>(out, 8 * i + 4, b);
      }
    }
  }
}

bool args_ok(int type, int tile, int64_t M, int64_t K) {
  return size_ok(M) && size_ok(K) && K >= 1 && type_ok(type) && (tile == 1 || tile == kBlock);
}

}  // namespace
}  // namespace mlp

using namespace mlp;

extern "C" {

lora_status lora_block8(const void* x, int x_type, int tile, int64_t M, int64_t K, void* codes, float* scales,
                        void* stream) {
  if (!args_ok(x_type, tile, M, K)) return LORA_ERR_SHAPE;
  if (M == 0) return LORA_OK;
  lora_status s = check_ptrs(x, static_cast<const void*>(codes), static_cast<const void*>(scales));
  if (s != LORA_OK) return s;
  const int64_t per_row = blocks128(K), blocks = cdiv(M, tile) * per_row;
  constexpr int kDeep = 4;
  const int64_t ctas = tile != 1 ? blocks : cdiv(blocks, K % 8 == 0 ? 16 * kDeep : 8);
  if (!size_ok(ctas)) return LORA_ERR_SHAPE;
  int nsm = 0;
  if ((s = device_ready(&nsm)) != LORA_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* c = static_cast<uint8_t*>(codes);
  const uint32_t k = uint32_t(K);
  auto rows = [&](auto kernel) {
    return launch_pdl(kernel, dim3(unsigned(ctas)), dim3(256), 0, st, x, blocks, k, uint32_t(per_row), c, scales);
  };
  auto tiles = [&](auto kernel) { return launch_pdl(kernel, dim3(unsigned(ctas)), dim3(256), 0, st, x, M, k, c, scales); };
  const bool vec = K % 8 == 0, bf = x_type == LORA_BF16;
  cudaError_t e;
  if (tile == 1 && vec) e = bf ? rows(block8_rows_kernel<kBf16, kDeep>) : rows(block8_rows_kernel<kF32, kDeep>);
  else if (tile == 1) e = bf ? rows(block8_rows_any_kernel<kBf16>) : rows(block8_rows_any_kernel<kF32>);
  else if (vec) e = bf ? tiles(block8_tiles_kernel<kBf16>) : tiles(block8_tiles_kernel<kF32>);
  else e = bf ? tiles(block8_tiles_any_kernel<kBf16>) : tiles(block8_tiles_any_kernel<kF32>);
  return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

lora_status lora_unblock8(const void* codes, const float* scales, int tile, int64_t M, int64_t K, void* out,
                          int out_type, void* stream) {
  if (!args_ok(out_type, tile, M, K)) return LORA_ERR_SHAPE;
  if (M == 0) return LORA_OK;
  lora_status s = check_ptrs(codes, static_cast<const void*>(scales), static_cast<const void*>(out));
  if (s != LORA_OK) return s;
  constexpr int kDeep = 4;
  const int vec = K % 8 == 0 ? 8 : 1;
  const int64_t per_row = K / vec, items = M * per_row, ctas = cdiv(items, 256 * kDeep);
  if (!size_ok(ctas)) return LORA_ERR_SHAPE;
  int nsm = 0;
  if ((s = device_ready(&nsm)) != LORA_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3(unsigned(ctas)), dim3(256), 0, st, static_cast<const uint8_t*>(codes), scales,
                      tile == 1 ? 0 : 7, items, uint32_t(K), uint32_t(per_row), out);
  };
  const bool bf = out_type == LORA_BF16;
  const cudaError_t e = vec == 8 ? (bf ? go(unblock8_kernel<kBf16, 8, kDeep>) : go(unblock8_kernel<kF32, 8, kDeep>))
                                 : (bf ? go(unblock8_kernel<kBf16, 1, kDeep>) : go(unblock8_kernel<kF32, 1, kDeep>));
  return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

}  // extern "C"
