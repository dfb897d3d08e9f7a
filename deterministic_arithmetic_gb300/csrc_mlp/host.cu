// host.cu -- host-side state shared by the MLP-block operators: the device check
// and the tensor-map encoder, both looked up once per device.
#include <cudaTypedefs.h>

#include <mutex>

#include "../csrc_base8/base8.h"
#include "mlp.h"

namespace mlp {
namespace {

constexpr int kMaxDevices = 64;
struct Device {
  bool probed = false, usable = false;
  int nsm = 0;
  uint32_t* status = nullptr;
  FfnFit fit;
};
Device g_dev[kMaxDevices];
std::mutex g_mu;
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

// Status block of the operators' kernels: 64 words, all zero until a kernel gives up on a wait.
__device__ uint32_t g_status[64];

}  // namespace

lora_status device_ready(int* nsm) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return LORA_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return LORA_ERR_DEVICE;
  std::lock_guard<std::mutex> lock(g_mu);
  Device& d = g_dev[dev];
  if (!d.probed) {
    int major = 0, minor = 0, n = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return LORA_ERR_CUDA;
    if (!g_encode) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q;
      if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
              cudaSuccess ||
          q != cudaDriverEntryPointSuccess || !fn)
        return LORA_ERR_CUDA;
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    d.nsm = n;
    d.usable = major == 10 && minor == 3;
    if (d.usable) {
      void* p = nullptr;
      if (cudaGetSymbolAddress(&p, g_status) != cudaSuccess || !p) return LORA_ERR_CUDA;
      d.status = static_cast<uint32_t*>(p);
      d.fit.nsm = n;
      if (prepare_pack8_da() != cudaSuccess || prepare_ffn(&d.fit) != cudaSuccess ||
          prepare_layer_norm() != cudaSuccess || prepare_linear(dev) != cudaSuccess || prepare_distill() != cudaSuccess)
        return LORA_ERR_CUDA;
    }
    d.probed = true;
  }
  if (!d.usable) return LORA_ERR_DEVICE;
  *nsm = d.nsm;
  return LORA_OK;
}

bool any_device() {
  int n = 0;
  const cudaError_t e = cudaGetDeviceCount(&n);
  return e != cudaErrorNoDevice && e != cudaErrorInsufficientDriver && (e != cudaSuccess || n > 0);
}

bool in_device_memory(const void* p) {
  cudaPointerAttributes a{};
  return cudaPointerGetAttributes(&a, p) == cudaSuccess &&
         (a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeManaged);
}

uint32_t* status_block() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(g_mu);
  return g_dev[dev].status;
}

FfnFit ffn_fit() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FfnFit{};
  std::lock_guard<std::mutex> lock(g_mu);
  return g_dev[dev].fit;
}

bool tensor_map(CUtensorMap* m, const void* ptr, Elem e, int64_t rows, int64_t cols, int64_t ld, int box_cols,
                int box_rows, int swizzle) {
  const cuuint64_t size = e == Elem::f32 ? 4 : (e == Elem::bf16 ? 2 : 1);
  const CUtensorMapDataType type = e == Elem::f32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : e == Elem::bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                     : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
  cuuint64_t strides[1] = {cuuint64_t(ld) * size};
  cuuint32_t box[2] = {cuuint32_t(box_cols), cuuint32_t(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  const CUtensorMapSwizzle sw = swizzle == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                : swizzle == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                : swizzle == 32 ? CU_TENSOR_MAP_SWIZZLE_32B
                                                : CU_TENSOR_MAP_SWIZZLE_NONE;
  return g_encode(m, type, 2,
                  const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  sw,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool block_map(CUtensorMap* m, const void* ptr, int64_t rows, int64_t cols, int box_rows, int blocks) {
  cuuint64_t dims[3] = {64, cuuint64_t(rows), cuuint64_t(cols / 64)};
  cuuint64_t strides[2] = {cuuint64_t(cols) * 2, 128};
  cuuint32_t box[3] = {64, cuuint32_t(box_rows), cuuint32_t(blocks)};
  cuuint32_t estr[3] = {1, 1, 1};
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace mlp

extern "C" {

lora_status lora_mlp_device_status(int* code) {
  if (!code) return LORA_ERR_NULL;
  int nsm = 0;
  const lora_status s = mlp::device_ready(&nsm);
  if (s != LORA_OK) return s;
  uint32_t word = 0;
  // (the copy alone would not wait for streams that do not block on the default one, as torch's own do not)
  if (cudaDeviceSynchronize() != cudaSuccess) return LORA_ERR_CUDA;
  if (cudaMemcpy(&word, mlp::status_block(), sizeof(word), cudaMemcpyDeviceToHost) != cudaSuccess) return LORA_ERR_CUDA;
  *code = int(word);
  return word ? LORA_ERR_TIMEOUT : LORA_OK;
}

lora_status lora_mlp_device_status_reset(int stall_kind, int wait_limit_us) {
  int nsm = 0;
  const lora_status s = mlp::device_ready(&nsm);
  if (s != LORA_OK) return s;
  if (cudaDeviceSynchronize() != cudaSuccess) return LORA_ERR_CUDA;
  const uint32_t words[4] = {0u, 0u, uint32_t(stall_kind), uint32_t(wait_limit_us)};
  return cudaMemcpy(mlp::status_block(), words, sizeof(words), cudaMemcpyHostToDevice) == cudaSuccess ? LORA_OK
                                                                                                  : LORA_ERR_CUDA;
}

}  // extern "C"
