// gated_ffn.cu -- the gated feed-forward block's entry points: h = act(x Wg^T + Dg) (x Wu^T + Du), and
// its backward pass.
//
// Backward: the element-wise step dU = dh act(G), dG = dh U act'(G) is a kernel of its own (bound by
// HBM: dh, G and U read, dG and dU written once; 4096 x 17408 from 8 bits: 95 us, 6.0 TB/s). Its outputs, rounded to bf16, are what the
// adapters of the two projections take as dY, and the operands of the products dx and dW.
#include "gemm.cuh"

namespace mlp {
namespace {

// dG and dU, 8 elements a thread at a time, kDeep times. XK: how G and U are kept (bf16 or packed). FLAT
// (bf16, or F a multiple of 32): the kept rows lie one after the other as those of dh do.
constexpr int kDeep = 2;
template <int XK, bool FLAT>
__global__ void __launch_bounds__(256)
    ffn_grad_kernel(const void* __restrict__ dh, const void* __restrict__ g, const void* __restrict__ u,
                    const void* __restrict__ gs, const void* __restrict__ us, int act, int64_t items, uint32_t F,
                    void* __restrict__ dg, void* __restrict__ du) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t first = int64_t(blockIdx.x) * (256 * kDeep) + threadIdx.x, ld = row_ld<XK>(F);
  const uint32_t per_row = F / 8;
  Raw<kBf16, 8> rh[kDeep];
  Raw<XK, 8> rg[kDeep], ru[kDeep];
#pragma unroll
  for (int j = 0; j < kDeep; ++j) {
    const int64_t i = first + 256 * j;
    if (i < items) {
      const int64_t row = FLAT ? 0 : i / per_row;
      const int64_t at = FLAT ? 8 * i : row * ld + (i - row * per_row) * 8;
      rh[j].load_at(dh, nullptr, 8 * i);
      rg[j].load_at(g, gs, at);
      ru[j].load_at(u, us, at);
    }
  }
#pragma unroll
  for (int j = 0; j < kDeep; ++j) {
    const int64_t i = first + 256 * j;
    if (i >= items) continue;
    float h[8], a[8], b[8];
    rh[j].get(h);
    rg[j].get(a);
    ru[j].get(b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float p = act_p(act, a[e]);
      const float dg_e = h[e] * b[e] * act_slope(act, a[e], p);
      b[e] = h[e] * (a[e] * p);
      a[e] = dg_e;
    }
    // plain stores: the products that follow read both again, from L2 as far as they fit
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(dg) + 8 * i) = pack_bf16x8(a);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(du) + 8 * i) = pack_bf16x8(b);
  }
}

// Sizes: k-blocks and tiles index with 32 bits, and a tile's reduction stays far inside the waits' limit.
int64_t round8(int64_t v) { return (v + 7) & ~int64_t(7); }

bool shape_ok(int64_t M, int64_t K, int64_t F) {
  const int64_t most = int64_t(1) << 22;
  return M >= 0 && M < most && K > 0 && K < most && F > 0 && F < most && K % 8 == 0 && F % 8 == 0;
}
bool kind_ok(int act, int keep) {
  return (act == LORA_ACT_SILU || act == LORA_ACT_GELU) &&
         (keep == LORA_KEEP_NONE || keep == LORA_KEEP_BF16 || keep == LORA_KEEP_PACKED8);
}

// The operands of a product: a [a_rows][a_cols] and b [b_rows][b_cols], two of each (the second may
// be the first), bf16.
struct Operands {
  const void *a[2], *b[2];
  int64_t a_rows, a_cols, b_rows, b_cols;
};

// The map of an operand whose rows lie along the reduction: one box of `blocks` 64-column blocks
// where the columns are whole blocks, else a box a block. One copy a stage instead of several: the
// copies' number, not their bytes, bounds these products (dW at 4096 x 5120 x 17408: 842 -> 751 us).
bool rows_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, bool blocked, int blocks) {
  return blocked ? block_map(m, p, rows, cols, kBK, blocks) : tensor_map(m, p, Elem::bf16, rows, cols, cols, 64, kBK, 128);
}

template <int MODE, int CG, int SPLIT = 0>
lora_status launch_as(FfnArgs& P, const Operands& o, int bn, const FfnFit& fit, cudaStream_t st) {
  constexpr int products = MODE == kDw ? 2 : 1;
  P.bn = bn;
  // a batch smaller than a tile: only its rows are copied, and the ring holds more stages (the other
  // rows of the tile reach only rows of the accumulator that nobody reads)
  const int a_rows = MODE != kDw && P.m < kBM ? int(round8(P.m)) : kBM;
  P.blocked = MODE == kDw ? o.a_cols % 64 == 0 && o.b_cols % 64 == 0 : o.b_cols % 64 == 0;
  for (int i = 0; i < 2; ++i) {
    const bool a = MODE == kDw ? rows_map(&P.a[i], o.a[i], o.a_rows, o.a_cols, P.blocked, kBM / 64)
                               : tensor_map(&P.a[i], o.a[i], Elem::bf16, o.a_rows, o.a_cols, o.a_cols, kBK, a_rows, 128);
    const bool b = MODE == kFwd ? tensor_map(&P.b[i], o.b[i], Elem::bf16, o.b_rows, o.b_cols, o.b_cols, kBK, bn, 128)
                                : rows_map(&P.b[i], o.b[i], o.b_rows, o.b_cols, P.blocked, bn / CG / 64);
    const bool out = MODE != kDw || tensor_map(&P.o[i], P.out[i], Elem::bf16, P.m, P.n, P.n, 32, 32, 64);
    if (!a || !b || !out) return LORA_ERR_CUDA;
  }
  const int b_bytes = (MODE == kFwd ? 2 : 1) * bn * 128 / CG;
  P.a_bytes = a_rows * kBK * 2;
  P.block_bytes = P.a_bytes + b_bytes;
  // what a split's CTAs send one another arrives behind the ring: a tile's sums, or 16 rows of every piece
  const int ring = kRingBytes + (SPLIT == 2   ? kRingSlack - bn * kBM * 4
                                 : SPLIT == 8 ? kRingSlack - SPLIT * 16 * (bn * 4 + 16)
                                              : 0);
  constexpr bool narrow = CG == 1 && (MODE == kFwd || SPLIT);      // tiles whose blocks may be few bytes
  const int deep = !narrow ? 1 : (ring >= 16 * P.block_bytes ? 4 : (ring >= 8 * P.block_bytes ? 2 : 1));
  P.stages = std::min(kMaxStages, ring / (deep * P.block_bytes));
  P.tiles_m = int(cdiv(P.m, CG * kBM));
  P.tiles_n = int(cdiv(P.n, bn));
  const int64_t total = int64_t(products) * P.tiles_m * P.tiles_n;
  if (total >= int64_t(1) << 30) return LORA_ERR_SHAPE;
  // The pairs take the tiles in rounds. A last round that would keep at most half of them at work is
  // dealt out as half tiles instead: it then takes half a tile's time.
  const int rest = CG == 2 ? int(total % fit.pairs) : 0;
  const bool halves = CG == 2 && 2 * rest <= fit.pairs;
  P.whole = int(halves ? total - rest : total);
  P.total = int(halves ? total + rest : total);
  constexpr int cluster = SPLIT ? SPLIT : CG;
  const int most = SPLIT ? P.total : (CG == 2 ? fit.pairs : fit.nsm);    // a split's clusters have a tile each
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(cluster * (P.total < most ? P.total : most)));
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = kGemmSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {unsigned(cluster), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  auto go = [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, P, status_block()) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA; };
  if constexpr (narrow) {
    if (deep == 4) return go(ffn_gemm_kernel<MODE, CG, SPLIT, 4>);
    if (deep == 2) return go(ffn_gemm_kernel<MODE, CG, SPLIT, 2>);
  }
  return go(ffn_gemm_kernel<MODE, CG, SPLIT>);
}

template <int MODE>
lora_status launch(FfnArgs& P, const Operands& o, const FfnFit& fit, cudaStream_t st) {
  const FfnPlan plan = ffn_plan(MODE, P.m, P.n, P.nk, P.piece, P.keep_kind == LORA_KEEP_PACKED8, fit);
  if (plan.cg == 2) return launch_as<MODE, 2>(P, o, plan.bn, fit, st);
  if constexpr (MODE == kDx) {
    if (plan.split == 2) return launch_as<kDx, 1, 2>(P, o, plan.bn, fit, st);
    if (plan.split == 8) return launch_as<kDx, 1, 8>(P, o, plan.bn, fit, st);
  }
  return launch_as<MODE, 1>(P, o, plan.bn, fit, st);
}

// How many of the kernel's clusters the device holds at once (0 where it can form none).
template <class K>
int resident(K* kernel, unsigned cluster) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster);
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = kGemmSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {cluster, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess) return n;
  cudaGetLastError();                              // (an answer, not an error of a later call)
  return 0;
}

template <int MODE, int CG, int SPLIT, int... DEEP>
cudaError_t set_smem() {
  cudaError_t e = cudaSuccess;
  auto set = [&](auto kernel) {
    return (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kGemmSmem))) == cudaSuccess;
  };
  (void)(set(ffn_gemm_kernel<MODE, CG, SPLIT, DEEP>) && ...);
  return e;
}

}  // namespace

cudaError_t prepare_ffn(FfnFit* fit) {
  cudaError_t e;
  if ((e = set_smem<kFwd, 1, 0, 1, 2, 4>()) != cudaSuccess || (e = set_smem<kDx, 1, 0, 1>()) != cudaSuccess ||
      (e = set_smem<kDw, 1, 0, 1>()) != cudaSuccess || (e = set_smem<kDx, 1, 2, 1, 2, 4>()) != cudaSuccess ||
      (e = set_smem<kDx, 1, 8, 1, 2, 4>()) != cudaSuccess || (e = set_smem<kFwd, 2, 0, 1>()) != cudaSuccess ||
      (e = set_smem<kDx, 2, 0, 1>()) != cudaSuccess || (e = set_smem<kDw, 2, 0, 1>()) != cudaSuccess)
    return e;
  fit->pairs = std::min({resident(ffn_gemm_kernel<kFwd, 2>, 2), resident(ffn_gemm_kernel<kDx, 2>, 2),
                         resident(ffn_gemm_kernel<kDw, 2>, 2)});
  fit->two = resident(ffn_gemm_kernel<kDx, 1, 2>, 2);
  fit->eight = resident(ffn_gemm_kernel<kDx, 1, 8>, 8);
  return cudaSuccess;
}

}  // namespace mlp

using namespace mlp;

extern "C" {

lora_status lora_gated_ffn_fwd(const void* x, const void* w_gate, const void* w_up, const float* delta_gate,
                               const float* delta_up, int act, int64_t M, int64_t K, int64_t F, void* h, int keep,
                               void* gate, void* up, void* gate_scales, void* up_scales, void* stream) {
  if (!shape_ok(M, K, F) || !kind_ok(act, keep)) return LORA_ERR_SHAPE;
  if (M == 0) return LORA_OK;
  lora_status s = check_ptrs(x, w_gate, w_up, h);
  if (s == LORA_OK && (delta_gate || delta_up)) s = check_ptrs(delta_gate, delta_up);
  if (s == LORA_OK && keep != LORA_KEEP_NONE) s = check_ptrs(gate, up);
  if (s == LORA_OK && keep == LORA_KEEP_PACKED8) s = check_ptrs(gate_scales, up_scales);
  if (s != LORA_OK) return s;
  int nsm = 0;
  if ((s = device_ready(&nsm)) != LORA_OK) return s;
  FfnArgs P{};
  P.m = int(M);
  P.n = int(F);
  P.nk = int(cdiv(K, kBK));
  P.out[0] = static_cast<__nv_bfloat16*>(h);
  P.delta[0] = delta_gate;
  P.delta[1] = delta_up;
  P.keep[0] = gate;
  P.keep[1] = up;
  P.keep_scales[0] = static_cast<uint8_t*>(gate_scales);
  P.keep_scales[1] = static_cast<uint8_t*>(up_scales);
  P.keep_kind = keep;
  P.act = act;
  const Operands o{{x, x}, {w_gate, w_up}, M, K, F, K};
  return launch<kFwd>(P, o, ffn_fit(), static_cast<cudaStream_t>(stream));
}

lora_status lora_gated_ffn_bwd(const void* dh, const void* x, const void* w_gate, const void* w_up, int keep,
                               const void* gate, const void* up, const void* gate_scales, const void* up_scales, int act,
                               int64_t M, int64_t K, int64_t F, void* dx, void* dgate, void* dup, void* dw_gate,
                               void* dw_up, void* stream) {
  if (!shape_ok(M, K, F) || !kind_ok(act, keep) || keep == LORA_KEEP_NONE) return LORA_ERR_SHAPE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool dw = dw_gate || dw_up;
  lora_status s = LORA_OK;
  int nsm = 0;
  if (dw) s = check_ptrs(dw_gate, dw_up);
  if (s == LORA_OK && M > 0) s = check_ptrs(dh, w_gate, w_up, gate, up, dx, dgate, dup);
  if (s == LORA_OK && M > 0 && dw) s = check_ptrs(x);
  if (s == LORA_OK && M > 0 && keep == LORA_KEEP_PACKED8) s = check_ptrs(gate_scales, up_scales);
  if (s != LORA_OK || (M == 0 && !dw)) return s;
  if ((s = device_ready(&nsm)) != LORA_OK) return s;
  if (M == 0) {                                     // sums over no rows
    const size_t bytes = size_t(F) * size_t(K) * 2;
    return cudaMemsetAsync(dw_gate, 0, bytes, st) == cudaSuccess && cudaMemsetAsync(dw_up, 0, bytes, st) == cudaSuccess
               ? LORA_OK
               : LORA_ERR_CUDA;
  }
  const FfnFit fit = ffn_fit();
  const int64_t items = M * (F / 8);
  const dim3 grid(unsigned(cdiv(items, 256 * kDeep)));
  auto grad = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(256), 0, st, dh, gate, up, gate_scales, up_scales, act, items, uint32_t(F), dgate, dup);
  };
  const cudaError_t e = keep == LORA_KEEP_BF16 ? grad(ffn_grad_kernel<kBf16, true>)
                        : F % kGroup == 0      ? grad(ffn_grad_kernel<kPacked, true>)
                                               : grad(ffn_grad_kernel<kPacked, false>);
  if (e != cudaSuccess) return LORA_ERR_CUDA;
  FfnArgs P{};
  P.m = int(M);
  P.n = int(K);
  P.nk = int(cdiv(F, kBK));
  // (a piece shorter than 4 blocks would keep the large tiles' epilogue from hiding under their MMAs)
  P.piece = std::max(4, int(cdiv(P.nk, kMaxPieces)));
  P.pieces = int(cdiv(P.nk, P.piece));
  P.out[0] = static_cast<__nv_bfloat16*>(dx);
  if ((s = launch<kDx>(P, Operands{{dgate, dup}, {w_gate, w_up}, M, F, F, K}, fit, st)) != LORA_OK || !dw) return s;
  FfnArgs Q{};
  Q.m = int(F);
  Q.n = int(K);
  Q.nk = int(cdiv(M, kBK));
  Q.out[0] = static_cast<__nv_bfloat16*>(dw_gate);
  Q.out[1] = static_cast<__nv_bfloat16*>(dw_up);
  return launch<kDw>(Q, Operands{{dgate, dup}, {x, x}, M, F, M, K}, fit, st);
}

}  // extern "C"
