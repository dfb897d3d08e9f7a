// pack8_da.cu -- the adapter gradients of a packed x: dA = du^T x, and the whole
// backward pass of the LoRA delta. x is unpacked into the workspace first.
#include "../csrc/common.cuh"
#include "../csrc/kernels.h"
#include "mlp.h"

using namespace mlp;

namespace {

bool shape_ok(int64_t M, int64_t K) { return size_ok(M) && size_ok(K) && K > 0 && K % 8 == 0; }
bool rank_ok(int64_t R) { return R >= 8 && R <= 64 && R % 8 == 0; }

// Workspace of dA: the unpacked x, then one partial per 256-row chunk.
struct DaLayout {
  size_t part, bytes;
};
DaLayout da_layout(int64_t M, int64_t K, int64_t R) {
  DaLayout l;
  l.part = round256(size_t(M) * size_t(K) * 2);
  l.bytes = l.part + round256(size_t(cdiv(M, lora::kWgradChunk)) * lora::padded_rank(int(R)) * size_t(K) * 4);
  return l;
}

// The weight-gradient kernel reads its wide operand before its grid dependency wait (no kernel of
// the delta's own passes writes it). This empty launch between it and the unpacking starts the
// kernel's launch only after the unpacked rows are complete.
__global__ void after_unpack_kernel() {
  lora::grid_dependency_wait();
  lora::grid_dependents_launch();
}

}  // namespace

extern "C" {

size_t lora_pack8_da_workspace_size(int64_t M, int64_t K, int64_t R) {
  return shape_ok(M, K) && rank_ok(R) ? da_layout(M, K, R).bytes + 256 : 0;
}

lora_status lora_pack8_da(const void* du, const void* codes, const void* scales, int64_t M, int64_t K, int64_t R,
                          float* da, void* workspace, size_t workspace_bytes, void* stream) {
  if (!shape_ok(M, K)) return LORA_ERR_SHAPE;
  if (!rank_ok(R)) return LORA_ERR_RANK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  lora_status s;
  int nsm = 0;
  if (M == 0) {
    if ((s = check_ptrs(da)) != LORA_OK || (s = device_ready(&nsm)) != LORA_OK) return s;
    return cudaMemsetAsync(da, 0, size_t(R) * size_t(K) * 4, st) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
  }
  if ((s = check_ptrs(du, codes, scales, da, workspace)) != LORA_OK) return s;
  if (workspace_bytes < lora_pack8_da_workspace_size(M, K, R)) return LORA_ERR_WORKSPACE;
  if ((s = device_ready(&nsm)) != LORA_OK) return s;
  const int RP = lora::padded_rank(int(R));
  const DaLayout L = da_layout(M, K, R);
  float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + L.part);
  if ((s = lora_unpack8(codes, scales, M, K, workspace, LORA_BF16, stream)) != LORA_OK) return s;
  if (lora::launch_pdl(after_unpack_kernel, dim3(1), dim3(32), 0, st) != cudaSuccess) return LORA_ERR_CUDA;
  lora::WgArgs args{};
  args.n = 1;
  lora::WgSite& w = args.s[0];
  if (!tensor_map(&w.in, workspace, Elem::bf16, M, K, K, 64, 64, 128) ||
      !tensor_map(&w.g, du, Elem::bf16, M, R, R, RP, 64, RP * 2))
    return LORA_ERR_CUDA;
  w.part = part;
  w.M = int(M);
  w.Cw = int(K);
  w.alpha = 1.0f;
  const int64_t units = lora::wgrad_units(M, K, RP);
  if (lora::launch_wgrad(RP, false, args, status_block(), int(units < nsm ? units : nsm), st) != cudaSuccess)
    return LORA_ERR_CUDA;
  lora::CombineJobs jobs{};
  jobs.n = 1;
  jobs.j[0] = lora::CombineJob{part, da, int(cdiv(M, lora::kWgradChunk)), int(K), int(R), RP, 0};
  return lora::launch_combine(jobs, st) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

size_t lora_delta_bwd_packed8_workspace_size(int64_t M, int64_t K, int64_t N, int64_t R) {
  const size_t b = lora_delta_bwd_workspace_size(M, K, N, R);
  return b ? b + round256(size_t(M) * size_t(K) * 2) : 0;
}

lora_status lora_delta_bwd_packed8(const void* dy, const void* codes, const void* scales, const void* a, const void* b,
                                   const void* u, float alpha, int64_t M, int64_t K, int64_t N, int64_t R, float* dx,
                                   float* da, float* db, void* du, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  const size_t need = lora_delta_bwd_workspace_size(M, K, N, R);
  if (need && M > 0) {
    lora_status s = check_ptrs(dy, codes, scales, a, b, u, dx, da, db, du, workspace);
    if (s != LORA_OK) return s;
    if (workspace_bytes < lora_delta_bwd_packed8_workspace_size(M, K, N, R)) return LORA_ERR_WORKSPACE;
    if ((s = lora_unpack8(codes, scales, M, K, static_cast<uint8_t*>(workspace) + need, LORA_BF16, stream)) != LORA_OK)
      return s;
  }
  // a shape or rank that is refused, and M = 0, are lora_delta_bwd's to answer
  return lora_delta_bwd(dy, static_cast<uint8_t*>(workspace) + need, a, b, u, alpha, M, K, N, R, dx, da, db, du,
                        workspace, need, stream);
}

}  // extern "C"
