// linear.cu -- products with weights in 8-bit blocks (lora_block8_linear_* of include/lora_base8.h).
#include "linear.cuh"
#include "linear_plan.h"

#include <climits>

#include "block8.cuh"

namespace mlp {
namespace {

bool shape_ok(int64_t M, int64_t K, int64_t N) {
  const int64_t most = int64_t(1) << 22;
  return M >= 0 && M < most && K > 0 && K < most && N > 0 && N < most;
}

struct LinFit {
  int pairs;                                       // of CTAs that a device holds at once
  bool wide;                                       // the kernels of 256 columns have the registers that they share out
};
LinFit g_fit[64];

template <int MODE, int CG, int W, int DEEP, bool JOINS = false>
lora_status launch_as(LinArgs& P, const LinPlan& plan, const void* a, const void* w, int64_t red, int64_t w_rows,
                      int64_t w_cols, int nsm, int pairs, cudaStream_t st) {
  P.bn = plan.bn;
  // a batch smaller than a tile: only its rows are copied, and the ring holds more stages
  const int a_rows = P.m < kBM ? int((P.m + 7) & ~7) : kBM;
  constexpr int chunk = lin_chunk(W);
  if (!tensor_map(&P.a, a, Elem::u8, P.m, red, code_ld(red), kLinBK, a_rows, 128)) return LORA_ERR_CUDA;
  const bool b = MODE == kLinFwd
                     ? tensor_map(&P.b, w, Elem::u8, w_rows, w_cols, code_ld(w_cols), kLinBK, P.bn / CG, 128)
                     : tensor_map(&P.b, w, Elem::u8, w_rows, w_cols, code_ld(w_cols), chunk, kLinBK, chunk);
  if (!b) return LORA_ERR_CUDA;
  P.a_bytes = a_rows * kLinBK;
  P.block_bytes = P.a_bytes + P.bn / CG * kLinBK;
  if (P.boxes && !tensor_map(&P.o, P.out, P.out_f32 ? Elem::f32 : Elem::bf16, P.m, P.n, P.n, P.out_f32 ? 16 : 32, 32, 64)) return LORA_ERR_CUDA;
  if (JOINS && !tensor_map(&P.d, P.delta, Elem::f32, P.m, P.n, P.n, 16, 32, 64)) return LORA_ERR_CUDA;
  P.stages = std::min(kLinStages, lin_ring(W, JOINS) / (DEEP * P.block_bytes));
  P.tiles_m = int(cdiv(P.m, CG * kBM));
  P.tiles_n = int(cdiv(P.n, P.bn));
  const int64_t total = int64_t(P.tiles_m) * P.tiles_n;
  if (total >= int64_t(1) << 30) return LORA_ERR_SHAPE;
  P.total = int(total);
  const int most = CG == 2 ? pairs : nsm;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(CG * (P.total < most ? P.total : most)));
  cfg.blockDim = dim3(kLinThreads);
  cfg.dynamicSmemBytes = kLinSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {unsigned(CG), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = CG > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, linear_kernel<MODE, CG, W, DEEP, JOINS>, P, status_block()) == cudaSuccess ? LORA_OK
                                                                                                     : LORA_ERR_CUDA;
}

template <int MODE>
lora_status linear(const void* a, const float* sa, const void* w, const float* sw, const float* delta, int64_t M,
                   int64_t K, int64_t N, void* out, int out_type, void* stream) {
  if (!shape_ok(M, K, N) || !type_ok(out_type)) return LORA_ERR_SHAPE;
  if (M == 0) return LORA_OK;
  lora_status s = check_ptrs(a, static_cast<const void*>(sa), w, static_cast<const void*>(sw), static_cast<const void*>(out));
  if (s == LORA_OK && delta) s = check_ptrs(delta);
  if (s != LORA_OK) return s;
  int nsm = 0;
  if ((s = device_ready(&nsm)) != LORA_OK) return s;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return LORA_ERR_CUDA;
  const int64_t red = MODE == kLinFwd ? K : N, cols = MODE == kLinFwd ? N : K;
  LinArgs P{};
  P.m = int(M);
  P.n = int(cols);
  P.nk = int(blocks128(red));
  P.sa = sa;
  P.sb = sw;
  P.sb_out = MODE == kLinFwd ? blocks128(K) : 1;
  P.sb_red = MODE == kLinFwd ? 1 : blocks128(K);
  P.delta = delta;
  P.out = out;
  P.out_f32 = out_type == LORA_F32;
  P.vec = cols % 4 == 0;
  const int pairs = g_fit[dev].pairs;
  const LinPlan plan = lin_plan(MODE == kLinBwd, P.m, P.n, nsm, pairs, g_fit[dev].wide);
  P.boxes = plan.w == 256 && cols % (P.out_f32 ? 4 : 8) == 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto go = [&](auto cg, auto width, auto deep) {
    if constexpr (width.value == 256)
      if (P.boxes && P.delta) return launch_as<MODE, cg.value, 256, 1, true>(P, plan, a, w, red, N, K, nsm, pairs, st);
    return launch_as<MODE, cg.value, width.value, deep.value>(P, plan, a, w, red, N, K, nsm, pairs, st);
  };
  using std::integral_constant;
  if (plan.cg == 2) return go(integral_constant<int, 2>{}, integral_constant<int, 256>{}, integral_constant<int, 1>{});
  if (plan.w == 256) return go(integral_constant<int, 1>{}, integral_constant<int, 256>{}, integral_constant<int, 1>{});
  if (plan.w == 128) return go(integral_constant<int, 1>{}, integral_constant<int, 128>{}, integral_constant<int, 2>{});
  if (plan.w == 64) return go(integral_constant<int, 1>{}, integral_constant<int, 64>{}, integral_constant<int, 4>{});
  return go(integral_constant<int, 1>{}, integral_constant<int, 32>{}, integral_constant<int, 4>{});
}

template <int MODE>
cudaError_t prepare(LinFit* fit) {
  cudaError_t e = cudaSuccess;
  auto set = [&](auto kernel) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kLinSmem));
  };
  // The 256-column kernels share out the registers that they are launched with: compiled to fewer, some would wait for theirs for
  // ever. Narrower ones then take their place; nothing else in the library asks.
  auto set_shared = [&](auto kernel) {
    cudaFuncAttributes a;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, kernel);
    if (e == cudaSuccess && a.numRegs < kLinRegs) fit->wide = false;
    set(kernel);
  };
  set_shared(linear_kernel<MODE, 2, 256, 1, false>);
  set_shared(linear_kernel<MODE, 2, 256, 1, true>);
  set_shared(linear_kernel<MODE, 1, 256, 1, false>);
  set_shared(linear_kernel<MODE, 1, 256, 1, true>);
  set(linear_kernel<MODE, 1, 128, 2, false>);
  set(linear_kernel<MODE, 1, 64, 4, false>);
  set(linear_kernel<MODE, 1, 32, 4, false>);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(kLinThreads);
  cfg.dynamicSmemBytes = kLinSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {2, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int pairs = 0;
  if (cudaOccupancyMaxActiveClusters(&pairs, linear_kernel<MODE, 2, 256, 1, true>, &cfg) != cudaSuccess) {
    cudaGetLastError();                            // (an answer, not an error of a later call)
    pairs = 0;
  }
  fit->pairs = std::min(fit->pairs, pairs);
  return cudaSuccess;
}

}  // namespace

cudaError_t prepare_linear(int dev) {
  LinFit fit{INT_MAX, true};
  cudaError_t e;
  if ((e = prepare<kLinFwd>(&fit)) != cudaSuccess || (e = prepare<kLinBwd>(&fit)) != cudaSuccess) return e;
  g_fit[dev] = fit;
  return cudaSuccess;
}

}  // namespace mlp

using namespace mlp;

extern "C" {

lora_status lora_block8_linear_fwd(const void* x, const float* x_scales, const void* w, const float* w_scales,
                                   const float* delta, int64_t M, int64_t K, int64_t N, void* y, int out_type,
                                   void* stream) {
  return linear<kLinFwd>(x, x_scales, w, w_scales, delta, M, K, N, y, out_type, stream);
}

lora_status lora_block8_linear_bwd(const void* dy, const float* dy_scales, const void* w, const float* w_scales,
                                   const float* delta, int64_t M, int64_t K, int64_t N, void* dx, int out_type,
                                   void* stream) {
  return linear<kLinBwd>(dy, dy_scales, w, w_scales, delta, M, K, N, dx, out_type, stream);
}

}  // extern "C"
