// mlp.h -- internal interface of the MLP-block operators: host checks shared by
// their entry points and the kernel launchers. Not installed; the public
// interface is include/lora_mlp.h.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/lora_mlp.h"
#include "ffn_plan.h"

namespace mlp {

constexpr int kGroup = 32;   // elements of a row that share one 8-bit scale

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t groups(int64_t k) { return cdiv(k, kGroup); }
inline size_t round256(size_t b) { return (b + 255) & ~size_t(255); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool size_ok(int64_t v) { return v >= 0 && v < (int64_t(1) << 31); }
inline bool type_ok(int t) { return t == LORA_BF16 || t == LORA_F32; }

// The checks every entry point makes of its pointers: none null, then all 16-byte aligned.
template <class... P>
lora_status check_ptrs(const P*... p) {
  const void* all[] = {p...};
  for (const void* q : all)
    if (!q) return LORA_ERR_NULL;
  for (const void* q : all)
    if (!aligned16(q)) return LORA_ERR_ALIGN;
  return LORA_OK;
}

// LORA_OK on an sm_103 device (with every kernel of the operators prepared on it); *nsm its SMs.
lora_status device_ready(int* nsm);
// Whether the machine has a CUDA device (and a driver for it) at all.
bool any_device();
// Whether p is device (or managed) memory.
bool in_device_memory(const void* p);

// Raise the shared-memory limits of the kernels (on the current device), and find what clusters it holds.
cudaError_t prepare_ffn(FfnFit* fit);
cudaError_t prepare_layer_norm();
cudaError_t prepare_pack8_da();

// The status block of the current device (common.cuh's layout): the operators of this folder run
// without a workspace of their own to hold one. Valid after device_ready; zero when loaded.
uint32_t* status_block();
// What the current device holds of the gated block's clusters. Valid after device_ready.
FfnFit ffn_fit();

// 2-D row-major map of a tensor [rows][cols] whose rows are `ld` elements apart; `swizzle` bytes
// (128, 64, 32; 0: none). False: the driver refused it.
enum class Elem { bf16, f32, u8 };
bool tensor_map(CUtensorMap* m, const void* ptr, Elem e, int64_t rows, int64_t cols, int64_t ld, int box_cols,
                int box_rows, int swizzle);
// The same bf16 tensor as 64-column blocks, [cols / 64][rows][64] (cols a multiple of 64): a box is
// `blocks` neighbouring blocks of box_rows rows, one after the other, 128-byte swizzle.
bool block_map(CUtensorMap* m, const void* ptr, int64_t rows, int64_t cols, int box_rows, int blocks);

}  // namespace mlp
