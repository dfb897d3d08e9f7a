// block8.cu -- tensors in 8-bit blocks of 128 (lora_block8, lora_unblock8 of include/lora_base8.h).
//
// One pass: a block's elements are read once into registers, their largest magnitude is found by shuffles (and,
// for a weight's 128 x 128, through shared memory), and the codes are written. Bound by HBM: 3 bytes an element of
// a bf16 tensor (17408 x 5120 in 128 x 128 40 us, 6.7 TB/s; back 41).
#include "../csrc/common.cuh"
#include "../csrc/kernels.h"
#include "../csrc_mlp/elems.cuh"
#include "base8.h"
#include "block8.cuh"

#include <type_traits>

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

// Item i of a CTA's (of items dealt row by row, per_row a row, the CTA's first being item rem of row `row`): which row, which of
// its items. One 64-bit division a CTA; rows shorter than the CTA's items take a 32-bit one an item.
struct At {
  int64_t row;
  uint32_t i;
};
__device__ __forceinline__ At item_at(int64_t row, uint32_t i, uint32_t per_row, uint32_t most) {
  const uint32_t r = per_row >= most ? uint32_t(i >= per_row) : i / per_row;
  return {row + r, i - r * per_row};
}

// Blocks of one row, K a multiple of 8: 16 lanes a block, 8 elements a lane, DEEP blocks of a half warp in flight. FLAT (K a
// multiple of 128): the rows' blocks lie one after the other.
template <int KIND, bool FLAT, int DEEP>
__global__ void __launch_bounds__(256)
    block8_rows_kernel(const void* __restrict__ x, int64_t blocks, uint32_t K, uint32_t per_row,
                       uint8_t* __restrict__ codes, float* __restrict__ scales) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t first = int64_t(blockIdx.x) * (16 * DEEP), b0 = first + (threadIdx.x >> 4);
  const uint32_t lane = threadIdx.x & 15u, ld = uint32_t(code_ld(K));
  const int64_t row0 = FLAT ? 0 : first / per_row;
  const uint32_t rem = FLAT ? 0 : uint32_t(first - row0 * per_row) + (threadIdx.x >> 4);
  Eight<KIND> r[DEEP];
  int64_t to[DEEP];                                // where in the codes, -1: nowhere
#pragma unroll
  for (int j = 0; j < DEEP; ++j) {
    r[j].clear();
    to[j] = -1;
    if (b0 + 16 * j >= blocks) continue;
    if constexpr (FLAT) {
      to[j] = (b0 + 16 * j) * kBlock + 8 * lane;
      r[j].load(x, to[j]);
    } else {
      const At a = item_at(row0, rem + 16 * j, per_row, 16 * (DEEP + 1));
      const uint32_t col = a.i * kBlock + 8 * lane;
      if (col < ld) to[j] = a.row * ld + col;
      if (col < K) r[j].load(x, a.row * K + col);
    }
  }
#pragma unroll
  for (int j = 0; j < DEEP; ++j) {
    float v[8];
    r[j].get(v);
    uint32_t m = amax8(v);
#pragma unroll
    for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const BlockScale s = block_scale(m);
    if (to[j] >= 0) *reinterpret_cast<uint2*>(codes + to[j]) = codes8(v, s.inv);
    if (lane == 0 && b0 + 16 * j < blocks) scales[b0 + 16 * j] = s.scale;
  }
}

// Any K: a warp a block, its elements 32 apart, DEEP blocks in flight.
template <int KIND, int DEEP>
__global__ void __launch_bounds__(256)
    block8_rows_any_kernel(const void* __restrict__ x, int64_t blocks, uint32_t K, uint32_t per_row,
                           uint8_t* __restrict__ codes, float* __restrict__ scales) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t first = int64_t(blockIdx.x) * (8 * DEEP), row0 = first / per_row, b0 = first + (threadIdx.x >> 5);
  const uint32_t rem = uint32_t(first - row0 * per_row) + (threadIdx.x >> 5);
  const uint32_t lane = threadIdx.x & 31u, ld = uint32_t(code_ld(K));
  float v[DEEP][4];
#pragma unroll
  for (int j = 0; j < DEEP; ++j) {
    const At a = item_at(row0, rem + 8 * j, per_row, 8 * (DEEP + 1));
    const uint32_t c0 = a.i * kBlock + lane;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v[j][e] = b0 + 8 * j < blocks && c0 + 32 * e < K ? param_at(x, KIND, a.row * K + c0 + 32 * e) : 0.f;
  }
#pragma unroll
  for (int j = 0; j < DEEP; ++j) {
    const At a = item_at(row0, rem + 8 * j, per_row, 8 * (DEEP + 1));
    const uint32_t c0 = a.i * kBlock + lane;
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) m = max(m, abs_bits(v[j][e]));
    const BlockScale s = block_scale(__reduce_max_sync(0xffffffffu, m));
    if (b0 + 8 * j >= blocks) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c0 + 32 * e < ld) codes[a.row * ld + c0 + 32 * e] = uint8_t(codes2(v[j][e], 0.f, s.inv));
    if (lane == 0) scales[b0 + 8 * j] = s.scale;
  }
}

// The largest over the CTA's threads.
template <int THREADS>
__device__ __forceinline__ uint32_t cta_max(uint32_t m) {
  __shared__ uint32_t part[THREADS / 32];
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31u) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) m = max(m, part[i]);
  return m;
}

// Blocks of 128 x 128, a CTA each: 16 lanes a row of a block, 16 rows at a time. (Four CTAs an SM, two of fp32: the block's
// elements stay in registers.)
template <int KIND>
__global__ void __launch_bounds__(256, KIND == kF32 ? 2 : 4)
    block8_tiles_kernel(const void* __restrict__ x, int64_t M, uint32_t K, uint8_t* __restrict__ codes,
                        float* __restrict__ scales) {
  grid_dependency_wait();
  grid_dependents_launch();
  const uint32_t per_row = (K + kBlock - 1) / kBlock, ld = uint32_t(code_ld(K));
  const uint32_t rb = blockIdx.x / per_row, cb = blockIdx.x - rb * per_row, col = cb * kBlock + 8 * (threadIdx.x & 15u);
  const int64_t row0 = int64_t(rb) * kBlock + (threadIdx.x >> 4);
  const int rows = int(min(int64_t(kBlock), M - row0));          // of this thread's from row0 on
  Eight<KIND> r[8];
  int64_t at = row0 * K + col;
#pragma unroll
  for (int j = 0; j < 8; ++j, at += 16 * int64_t(K)) {
    r[j].clear();
    if (16 * j < rows && col < K) r[j].load(x, at);
  }
  uint32_t m = 0;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    r[j].get(v);
    m = max(m, amax8(v));
  }
  const BlockScale s = block_scale(cta_max<256>(m));
  uint8_t* to = codes + row0 * ld + col;
#pragma unroll
  for (int j = 0; j < 8; ++j, to += 16 * int64_t(ld)) {
    r[j].get(v);
    if (16 * j < rows && col < ld) *reinterpret_cast<uint2*>(to) = codes8(v, s.inv);
  }
  if (threadIdx.x == 0) scales[blockIdx.x] = s.scale;
}

// Any K: 128 threads a row, four rows at a time.
template <int KIND>
__global__ void __launch_bounds__(512, 2)
    block8_tiles_any_kernel(const void* __restrict__ x, int64_t M, uint32_t K, uint8_t* __restrict__ codes,
                            float* __restrict__ scales) {
  grid_dependency_wait();
  grid_dependents_launch();
  const uint32_t per_row = (K + kBlock - 1) / kBlock, ld = uint32_t(code_ld(K));
  const uint32_t rb = blockIdx.x / per_row, cb = blockIdx.x - rb * per_row, col = cb * kBlock + (threadIdx.x & 127u);
  const int64_t row0 = int64_t(rb) * kBlock + (threadIdx.x >> 7);
  const int rows = int(min(int64_t(kBlock), M - row0));
  float v[32];
  uint32_t m = 0;
  int64_t at = row0 * K + col;
#pragma unroll
  for (int j = 0; j < 32; ++j, at += 4 * int64_t(K)) v[j] = 4 * j < rows && col < K ? param_at(x, KIND, at) : 0.f;
#pragma unroll
  for (int j = 0; j < 32; ++j) m = max(m, abs_bits(v[j]));
  const BlockScale s = block_scale(cta_max<512>(m));
  uint8_t* to = codes + row0 * ld + col;
#pragma unroll
  for (int j = 0; j < 32; ++j, to += 4 * int64_t(ld))
    if (4 * j < rows && col < ld) *to = uint8_t(codes2(v[j], 0.f, s.inv));
  if (threadIdx.x == 0) scales[blockIdx.x] = s.scale;
}

// The values: 8 elements a thread, DEEP times. ANY: rows of a length that 8 does not divide, whose values take the way through
// shared memory, since their rows start anywhere (2 bytes or 4 a lane straight from registers: 8192 x 4097 133 us, 51 so).
template <int KIND, bool ANY, int DEEP>
__global__ void __launch_bounds__(256)
    unblock8_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scales, int tile_log2, int64_t items,
                    uint32_t K, uint32_t per_row, void* __restrict__ out) {
  using T = typename std::conditional<KIND == kF32, float, __nv_bfloat16>::type;
  __shared__ T stage[ANY ? 256 * 8 : 1];
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t first = int64_t(blockIdx.x) * (256 * DEEP), row0 = first / per_row, ld = code_ld(K);
  const uint32_t rem = uint32_t(first - row0 * per_row) + threadIdx.x, cblocks = (K + kBlock - 1) / kBlock;
  uint2 c[DEEP];
  float s[DEEP];
#pragma unroll
  for (int j = 0; j < DEEP; ++j) {
    c[j] = make_uint2(0u, 0u);
    s[j] = 0.f;
    if (first + threadIdx.x + 256 * j < items) {
      const At a = item_at(row0, rem + 256 * j, per_row, 256 * (DEEP + 1));
      c[j] = __ldg(reinterpret_cast<const uint2*>(codes + a.row * ld + 8 * a.i));
      s[j] = __ldg(scales + (a.row >> tile_log2) * cblocks + a.i / (kBlock / 8));
    }
  }
#pragma unroll
  for (int j = 0; j < DEEP; ++j) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = values2(((k < 2 ? c[j].x : c[j].y) >> (16 * (k & 1))) & 0xFFFFu);
      v[2 * k] = f.x * s[j];
      v[2 * k + 1] = f.y * s[j];
    }
    if constexpr (!ANY) {
      const int64_t i = first + threadIdx.x + 256 * j;           // the rows lie one after the other
      if (i >= items) continue;
      if constexpr (KIND == kBf16) {
        store_vec<kBf16, 8>(out, 8 * i, v);
      } else {
        const float a[4] = {v[0], v[1], v[2], v[3]}, b[4] = {v[4], v[5], v[6], v[7]};
        store_vec<kF32, 4>(out, 8 * i, a);
        store_vec<kF32, 4>(out, 8 * i + 4, b);
      }
    } else {
      // a warp's 256 elements: its lanes' eights, some of them the next row's
      T* mine = stage + (threadIdx.x & ~31u) * 8;
      const uint32_t lane = threadIdx.x & 31u;
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 8; ++k) mine[8 * lane + k] = T(v[k]);
      __syncwarp();
      const uint32_t w0 = rem - lane + 256 * j;    // the warp's first item
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t e = 32 * k + lane;
        const At a = item_at(row0, w0 + e / 8, per_row, 256 * (DEEP + 1));
        const uint32_t col = 8 * a.i + e % 8;
        if (first + (threadIdx.x & ~31u) + 256 * j + e / 8 < items && col < K) static_cast<T*>(out)[a.row * K + col] = mine[e];
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
  constexpr int kDeep = 2;                         // (1, 2, 4, 8: 22.9, 20.3, 23.2, 28.1 us at 8192 x 4096 bf16)
  const int64_t ctas = tile != 1 ? blocks : cdiv(blocks, (K % 8 == 0 ? 16 : 8) * kDeep);
  if (!size_ok(ctas)) return LORA_ERR_SHAPE;
  int nsm = 0;
  if ((s = device_ready(&nsm)) != LORA_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* c = static_cast<uint8_t*>(codes);
  const uint32_t k = uint32_t(K);
  auto rows = [&](auto kernel) {
    return launch_pdl(kernel, dim3(unsigned(ctas)), dim3(256), 0, st, x, blocks, k, uint32_t(per_row), c, scales);
  };
  auto tiles = [&](auto kernel, int threads) {
    return launch_pdl(kernel, dim3(unsigned(ctas)), dim3(threads), 0, st, x, M, k, c, scales);
  };
  const bool vec = K % 8 == 0, flat = K % kBlock == 0, bf = x_type == LORA_BF16;
  cudaError_t e;
  if (tile == 1 && flat) e = bf ? rows(block8_rows_kernel<kBf16, true, kDeep>) : rows(block8_rows_kernel<kF32, true, kDeep>);
  else if (tile == 1 && vec) e = bf ? rows(block8_rows_kernel<kBf16, false, kDeep>) : rows(block8_rows_kernel<kF32, false, kDeep>);
  else if (tile == 1) e = bf ? rows(block8_rows_any_kernel<kBf16, kDeep>) : rows(block8_rows_any_kernel<kF32, kDeep>);
  else if (vec) e = bf ? tiles(block8_tiles_kernel<kBf16>, 256) : tiles(block8_tiles_kernel<kF32>, 256);
  else e = bf ? tiles(block8_tiles_any_kernel<kBf16>, 512) : tiles(block8_tiles_any_kernel<kF32>, 512);
  return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

lora_status lora_unblock8(const void* codes, const float* scales, int tile, int64_t M, int64_t K, void* out,
                          int out_type, void* stream) {
  if (!args_ok(out_type, tile, M, K)) return LORA_ERR_SHAPE;
  if (M == 0) return LORA_OK;
  lora_status s = check_ptrs(codes, static_cast<const void*>(scales), static_cast<const void*>(out));
  if (s != LORA_OK) return s;
  constexpr int kDeep = 4;
  const int64_t per_row = cdiv(K, 8), items = M * per_row, ctas = cdiv(items, 256 * kDeep);
  if (!size_ok(ctas)) return LORA_ERR_SHAPE;
  int nsm = 0;
  if ((s = device_ready(&nsm)) != LORA_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3(unsigned(ctas)), dim3(256), 0, st, static_cast<const uint8_t*>(codes), scales,
                      tile == 1 ? 0 : 7, items, uint32_t(K), uint32_t(per_row), out);
  };
  const bool bf = out_type == LORA_BF16;
  const cudaError_t e = K % 8 == 0 ? (bf ? go(unblock8_kernel<kBf16, false, kDeep>) : go(unblock8_kernel<kF32, false, kDeep>))
                                   : (bf ? go(unblock8_kernel<kBf16, true, kDeep>) : go(unblock8_kernel<kF32, true, kDeep>));
  return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

}  // extern "C"
