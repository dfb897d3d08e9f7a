// layer_norm.cu -- layer norm over rows of N elements, forward and backward:
//   mean = sum(x) / N    var = sum((x - mean)^2) / N    rstd = 1 / sqrt(var + eps)
//   y  = xh w + b,  xh = (x - mean) rstd
//   dx = rstd (g - mean(g) - xh mean(g xh)),  g = dy w;    dw = sum_m dy xh;    db = sum_m dy
//
// All of it is bound by HBM: each element of x (and dy) is read once and held
// in registers while the row's sums are formed, each output written once. A row
// group of W warps owns a row; a thread holds 16 elements of it (8192 elements
// in a group of 16 warps; longer rows take the looped kernels at the end). W
// and each thread's columns follow from N alone, so a row's sums are added in
// the same order in any batch. The variance is the sum of squares about the
// mean, from registers: no cancellation, and no second read.
//
// The backward pass's column sums: a thread keeps dw and db of its 16 columns in
// registers over all rows its group visits (rows dealt round robin over the
// grid), the row groups of a CTA add up in shared memory, and each CTA leaves one
// partial row; a second kernel adds the partials in order. The number of CTAs
// depends on M and N only, so reruns give the same bits on any device.
#include "../csrc/common.cuh"
#include "../csrc/kernels.h"
#include "elems.cuh"
#include "mlp.h"

namespace mlp {
namespace {

using lora::grid_dependency_wait;
using lora::grid_dependents_launch;
using lora::launch_pdl;

constexpr int kPerThread = 16;                      // elements of a row a thread holds
constexpr int kMaxWarps = 16;                       // warps of a row group
constexpr int kHeldN = 32 * kPerThread * kMaxWarps; // longest row a group holds in registers
constexpr int kBlockWarps = 8;                      // warps of a CTA of short rows (several groups)
constexpr int kMaxParts = 304;                      // partial rows of dw and db: two CTAs on each of 152 SMs

inline int warps_per_row(int64_t n) { return int(cdiv(n, 32 * kPerThread)); }
inline int groups_per_block(int w) { return w >= kBlockWarps ? 1 : kBlockWarps / w; }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The sum of v over the W warps of a row group (named barrier 1 + group), in an order that W
// alone sets; every thread returns it. `red`: W floats of shared memory of the group, which the
// group touches in no other sum until all its threads have passed another barrier.
__device__ __forceinline__ float group_sum(float v, int W, int group, int wig, float* red) {
  v = warp_sum(v);
  if (W == 1) return v;
  if ((threadIdx.x & 31) == 0) red[wig] = v;
  lora::named_bar(1 + group, 32 * W);
  float s = red[0];
  for (int i = 1; i < W; ++i) s += red[i];
  return s;
}

template <int KIND, int VEC>
__global__ void __launch_bounds__(32 * kMaxWarps)
    ln_fwd_kernel(const void* __restrict__ x, const void* __restrict__ weight, const void* __restrict__ bias, int w_type,
                  float eps, int64_t M, int N, int W, void* __restrict__ y, float* __restrict__ mean_out,
                  float* __restrict__ rstd_out) {
  constexpr int NV = kPerThread / VEC;
  __shared__ float red[2][2 * kMaxWarps];
  grid_dependency_wait();
  grid_dependents_launch();
  const int warp = threadIdx.x >> 5, group = warp / W, wig = warp % W;
  const int t = wig * 32 + (threadIdx.x & 31);
  const int64_t row = int64_t(blockIdx.x) * (blockDim.x / (32 * W)) + group;
  if (row >= M) return;                      // whole groups: the other groups' barriers are their own
  Raw<KIND, VEC> raw[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * 32 * W + t) * VEC;
    if (c < N) raw[i].load(x, nullptr, row, N, c);
  }
  float v[NV][VEC];
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if ((i * 32 * W + t) * VEC < N) {
      raw[i].get(v[i]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += v[i][e];
    }
  }
  const float mean = __fdiv_rn(group_sum(s, W, group, wig, red[0] + group * W), float(N));
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if ((i * 32 * W + t) * VEC < N) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        v[i][e] -= mean;
        q = fmaf(v[i][e], v[i][e], q);
      }
    }
  }
  const float var = __fdiv_rn(group_sum(q, W, group, wig, red[1] + group * W), float(N));
  const float rstd = __frsqrt_rn(var + eps);
  if (t == 0) {
    mean_out[row] = mean;
    rstd_out[row] = rstd;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * 32 * W + t) * VEC;
    if (c < N) {
      float w[VEC], b[VEC], o[VEC];
      params_at<VEC>(weight, w_type, c, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) b[e] = 0.f;
      if (bias) params_at<VEC>(bias, w_type, c, b);
#pragma unroll
      for (int e = 0; e < VEC; ++e) o[e] = fmaf(v[i][e] * rstd, w[e], b[e]);
      store_vec<KIND, VEC>(y, row * N + c, o);
    }
  }
}

// XK: the kind of x (KIND, or packed). part: [gridDim.x][2][N] (dw, db), or [gridDim.x][N] without db.
template <int KIND, int XK, int VEC>
__global__ void __launch_bounds__(32 * kMaxWarps)
    ln_bwd_kernel(const void* __restrict__ dy, const void* __restrict__ x, const void* __restrict__ x_scales,
                  const void* __restrict__ weight, int w_type, const float* __restrict__ mean_in,
                  const float* __restrict__ rstd_in, int64_t M, int N, int W, void* __restrict__ dx,
                  float* __restrict__ part, int with_db) {
  constexpr int NV = kPerThread / VEC;
  __shared__ float red[2][2][2 * kMaxWarps];            // [row parity][sum]
  extern __shared__ float cols[];                       // [groups - 1][2][N]: the row groups' column sums
  grid_dependency_wait();
  grid_dependents_launch();
  const int warp = threadIdx.x >> 5, group = warp / W, wig = warp % W;
  const int ngroups = blockDim.x / (32 * W);
  const int t = wig * 32 + (threadIdx.x & 31);
  const int64_t x_ld = row_ld<XK>(N);
  const float inv_n = __fdiv_rn(1.f, float(N));
  float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * 32 * W + t) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[i][e] = dw[i][e] = db[i][e] = 0.f;
    if (c < N) params_at<VEC>(weight, w_type, c, w[i]);
  }
  int parity = 0;
  for (int64_t row = int64_t(blockIdx.x) * ngroups + group; row < M; row += int64_t(gridDim.x) * ngroups) {
    Raw<KIND, VEC> rdy[NV];
    Raw<XK, VEC> rx[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * 32 * W + t) * VEC;
      if (c < N) {
        rdy[i].load(dy, nullptr, row, N, c);
        rx[i].load(x, x_scales, row, x_ld, c);
      }
    }
    const float mean = mean_in[row], rstd = rstd_in[row];
    float xh[NV][VEC], g[NV][VEC];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if ((i * 32 * W + t) * VEC < N) {
        float d[VEC];
        rdy[i].get(d);
        rx[i].get(xh[i]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          xh[i][e] = (xh[i][e] - mean) * rstd;
          dw[i][e] = fmaf(d[e], xh[i][e], dw[i][e]);
          db[i][e] += d[e];
          g[i][e] = d[e] * w[i][e];
          s1 += g[i][e];
          s2 = fmaf(g[i][e], xh[i][e], s2);
        }
      }
    }
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if (W > 1) {
      float* r1 = red[parity][0] + group * W;
      float* r2 = red[parity][1] + group * W;
      if ((threadIdx.x & 31) == 0) {
        r1[wig] = s1;
        r2[wig] = s2;
      }
      // one barrier a row: the next row's sums use the other half of `red`, and the row after
      // that writes this half only after the next row's barrier
      lora::named_bar(1 + group, 32 * W);
      s1 = r1[0];
      s2 = r2[0];
      for (int i = 1; i < W; ++i) {
        s1 += r1[i];
        s2 += r2[i];
      }
      parity ^= 1;
    }
    const float c1 = s1 * inv_n, c2 = s2 * inv_n;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * 32 * W + t) * VEC;
      if (c < N) {
        float o[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = rstd * (g[i][e] - c1 - xh[i][e] * c2);
        store_vec<KIND, VEC>(dx, row * N + c, o);
      }
    }
  }
  // the row groups' column sums, added in group order
  if (ngroups > 1) {
    if (group > 0) {
      float* mine = cols + size_t(group - 1) * 2 * N;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int c = (i * 32 * W + t) * VEC + e;
          if (c < N) {
            mine[c] = dw[i][e];
            mine[N + c] = db[i][e];
          }
        }
    }
    __syncthreads();
  }
  if (group == 0) {
    float* out = part + size_t(blockIdx.x) * (with_db ? 2 : 1) * N;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int c = (i * 32 * W + t) * VEC + e;
        if (c < N) {
          float a = dw[i][e], b = db[i][e];
          for (int k = 1; k < ngroups; ++k) {
            a += cols[size_t(k - 1) * 2 * N + c];
            b += cols[size_t(k - 1) * 2 * N + N + c];
          }
          out[c] = a;
          if (with_db) out[N + c] = b;
        }
      }
  }
}

// ------------------------------------------------------ rows longer than kHeldN
// One CTA a row, looping over the row: the later passes read it again, from L2.
constexpr int kLongThreads = 512;

__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = red[0];
  for (int i = 1; i < kLongThreads / 32; ++i) s += red[i];
  return s;
}

template <int KIND, int VEC>
__global__ void __launch_bounds__(kLongThreads)
    ln_fwd_long_kernel(const void* __restrict__ x, const void* __restrict__ weight, const void* __restrict__ bias,
                       int w_type, float eps, int64_t M, int N, void* __restrict__ y, float* __restrict__ mean_out,
                       float* __restrict__ rstd_out) {
  __shared__ float red[kLongThreads / 32];
  grid_dependency_wait();
  grid_dependents_launch();
  for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
    float s = 0.f;
#pragma unroll 4
    for (int64_t c = int64_t(threadIdx.x) * VEC; c < N; c += kLongThreads * VEC) {
      Raw<KIND, VEC> r;
      float v[VEC];
      r.load(x, nullptr, row, N, int(c));
      r.get(v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += v[e];
    }
    const float mean = __fdiv_rn(block_sum(s, red), float(N));
    float q = 0.f;
#pragma unroll 4
    for (int64_t c = int64_t(threadIdx.x) * VEC; c < N; c += kLongThreads * VEC) {
      Raw<KIND, VEC> r;
      float v[VEC];
      r.load(x, nullptr, row, N, int(c));
      r.get(v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) q = fmaf(v[e] - mean, v[e] - mean, q);
    }
    const float rstd = __frsqrt_rn(__fdiv_rn(block_sum(q, red), float(N)) + eps);
    if (threadIdx.x == 0) {
      mean_out[row] = mean;
      rstd_out[row] = rstd;
    }
#pragma unroll 4
    for (int64_t c = int64_t(threadIdx.x) * VEC; c < N; c += kLongThreads * VEC) {
      Raw<KIND, VEC> r;
      float v[VEC], w[VEC], b[VEC];
      r.load(x, nullptr, row, N, int(c));
      r.get(v);
      params_at<VEC>(weight, w_type, int(c), w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) b[e] = 0.f;
      if (bias) params_at<VEC>(bias, w_type, int(c), b);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = fmaf((v[e] - mean) * rstd, w[e], b[e]);
      store_vec<KIND, VEC>(y, row * N + c, v);
    }
  }
}

template <int KIND, int XK, int VEC>
__global__ void __launch_bounds__(kLongThreads)
    ln_dx_long_kernel(const void* __restrict__ dy, const void* __restrict__ x, const void* __restrict__ x_scales,
                      const void* __restrict__ weight, int w_type, const float* __restrict__ mean_in,
                      const float* __restrict__ rstd_in, int64_t M, int N, void* __restrict__ dx) {
  __shared__ float red[kLongThreads / 32];
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t x_ld = row_ld<XK>(N);
  const float inv_n = __fdiv_rn(1.f, float(N));
  for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
    const float mean = mean_in[row], rstd = rstd_in[row];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll 4
    for (int64_t c = int64_t(threadIdx.x) * VEC; c < N; c += kLongThreads * VEC) {
      Raw<KIND, VEC> rd;
      Raw<XK, VEC> rx;
      float d[VEC], v[VEC], w[VEC];
      rd.load(dy, nullptr, row, N, int(c));
      rx.load(x, x_scales, row, x_ld, int(c));
      params_at<VEC>(weight, w_type, int(c), w);
      rd.get(d);
      rx.get(v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float g = d[e] * w[e];
        s1 += g;
        s2 = fmaf(g, (v[e] - mean) * rstd, s2);
      }
    }
    const float c1 = block_sum(s1, red) * inv_n, c2 = block_sum(s2, red) * inv_n;
#pragma unroll 4
    for (int64_t c = int64_t(threadIdx.x) * VEC; c < N; c += kLongThreads * VEC) {
      Raw<KIND, VEC> rd;
      Raw<XK, VEC> rx;
      float d[VEC], v[VEC], w[VEC];
      rd.load(dy, nullptr, row, N, int(c));
      rx.load(x, x_scales, row, x_ld, int(c));
      params_at<VEC>(weight, w_type, int(c), w);
      rd.get(d);
      rx.get(v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = rstd * (d[e] * w[e] - c1 - (v[e] - mean) * rstd * c2);
      store_vec<KIND, VEC>(dx, row * N + c, v);
    }
  }
}

// Column sums of long rows: a warp's 32 VEC columns by blockIdx.x, rows dealt round robin over
// blockIdx.y and the CTA's warps; the warps add up in shared memory, in order.
template <int KIND, int XK, int VEC>
__global__ void __launch_bounds__(32 * kBlockWarps)
    ln_cols_long_kernel(const void* __restrict__ dy, const void* __restrict__ x, const void* __restrict__ x_scales,
                        const float* __restrict__ mean_in, const float* __restrict__ rstd_in, int64_t M, int N,
                        float* __restrict__ part, int with_db) {
  __shared__ float sums[kBlockWarps][2][32 * VEC];
  grid_dependency_wait();
  grid_dependents_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c = (int64_t(blockIdx.x) * 32 + lane) * VEC;
  const int64_t x_ld = row_ld<XK>(N);
  float dw[VEC], db[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) dw[e] = db[e] = 0.f;
  if (c < N) {
#pragma unroll 4
    for (int64_t row = int64_t(blockIdx.y) * kBlockWarps + warp; row < M; row += int64_t(gridDim.y) * kBlockWarps) {
      Raw<KIND, VEC> rd;
      Raw<XK, VEC> rx;
      float d[VEC], v[VEC];
      rd.load(dy, nullptr, row, N, int(c));
      rx.load(x, x_scales, row, x_ld, int(c));
      const float mean = mean_in[row], rstd = rstd_in[row];
      rd.get(d);
      rx.get(v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        dw[e] = fmaf(d[e], (v[e] - mean) * rstd, dw[e]);
        db[e] += d[e];
      }
    }
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    sums[warp][0][lane * VEC + e] = dw[e];
    sums[warp][1][lane * VEC + e] = db[e];
  }
  __syncthreads();
  float* out = part + size_t(blockIdx.y) * (with_db ? 2 : 1) * N;
  for (int i = threadIdx.x; i < 32 * VEC; i += blockDim.x) {
    const int64_t col = int64_t(blockIdx.x) * 32 * VEC + i;
    if (col < N) {
      float a = 0.f, b = 0.f;
      for (int k = 0; k < kBlockWarps; ++k) {
        a += sums[k][0][i];
        b += sums[k][1][i];
      }
      out[col] = a;
      if (with_db) out[N + col] = b;
    }
  }
}

// dw and db from the partial rows [P][cols] (cols = 2 N with db): 32 columns a CTA, the partials
// dealt over its 8 warps, then the warps' sums in order.
__global__ void __launch_bounds__(256)
    ln_parts_kernel(const float* __restrict__ part, int P, int64_t cols, int64_t N, float* __restrict__ dw,
                    float* __restrict__ db) {
  __shared__ float sums[8][32];
  grid_dependency_wait();
  grid_dependents_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c = int64_t(blockIdx.x) * 32 + lane;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int p = warp; p < P; p += 8) s += __ldcg(part + size_t(p) * cols + c);
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < cols) {
    for (int k = 1; k < 8; ++k) s += sums[k][lane];
    if (c < N) dw[c] = s;
    else db[c - N] = s;
  }
}

// Partial rows of a backward pass: at most kMaxParts, and no more than there are row groups' rows.
int parts_of(int64_t M, int64_t N) {
  const int rows = N <= kHeldN ? groups_per_block(warps_per_row(N)) : kBlockWarps;
  const int64_t most = N <= kHeldN ? kMaxParts : 64;
  const int64_t p = cdiv(M, rows);
  return int(p < most ? p : most);
}

template <int KIND, int VEC>
cudaError_t fwd(const void* x, const void* w, const void* b, int w_type, float eps, int64_t M, int N, void* y,
                float* mean, float* rstd, cudaStream_t st) {
  if (N > kHeldN) {
    const int64_t grid = M < 152 * 4 ? M : 152 * 4;
    return launch_pdl(ln_fwd_long_kernel<KIND, VEC>, dim3(unsigned(grid)), dim3(kLongThreads), 0, st, x, w, b, w_type,
                      eps, M, N, y, mean, rstd);
  }
  const int W = warps_per_row(N), G = groups_per_block(W);
  return launch_pdl(ln_fwd_kernel<KIND, VEC>, dim3(unsigned(cdiv(M, G))), dim3(32 * W * G), 0, st, x, w, b, w_type, eps,
                    M, N, W, y, mean, rstd);
}

template <int KIND, int XK, int VEC>
cudaError_t bwd(const void* dy, const void* x, const void* xs, const void* w, int w_type, const float* mean,
                const float* rstd, int64_t M, int N, void* dx, float* part, int P, bool with_db, cudaStream_t st) {
  if (N > kHeldN) {
    const int64_t grid = M < 152 * 4 ? M : 152 * 4;
    cudaError_t e = launch_pdl(ln_dx_long_kernel<KIND, XK, VEC>, dim3(unsigned(grid)), dim3(kLongThreads), 0, st, dy, x,
                               xs, w, w_type, mean, rstd, M, N, dx);
    if (e != cudaSuccess) return e;
    return launch_pdl(ln_cols_long_kernel<KIND, XK, VEC>, dim3(unsigned(cdiv(N, 32 * VEC)), unsigned(P)),
                      dim3(32 * kBlockWarps), 0, st, dy, x, xs, mean, rstd, M, N, part, int(with_db));
  }
  const int W = warps_per_row(N), G = groups_per_block(W);
  const size_t smem = size_t(G - 1) * 2 * N * 4;   // at most 7 groups of 512 columns: 28 KB
  return launch_pdl(ln_bwd_kernel<KIND, XK, VEC>, dim3(unsigned(P)), dim3(32 * W * G), smem, st, dy, x, xs, w, w_type,
                    mean, rstd, M, N, W, dx, part, int(with_db));
}

}  // namespace
}  // namespace mlp

using namespace mlp;

extern "C" {

lora_status lora_layer_norm_fwd(const void* x, int x_type, const void* weight, const void* bias, int w_type, float eps,
                                int64_t M, int64_t N, void* y, float* mean, float* rstd, void* stream) {
  if (!size_ok(M) || !size_ok(N) || N < 1 || !type_ok(x_type) || !type_ok(w_type)) return LORA_ERR_SHAPE;
  if (M == 0) return LORA_OK;
  lora_status s = check_ptrs(x, weight, y, mean, rstd);
  if (s != LORA_OK) return s;
  if (bias && !aligned16(bias)) return LORA_ERR_ALIGN;
  int nsm = 0;
  if ((s = device_ready(&nsm)) != LORA_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int n = int(N);
  cudaError_t e;
  if (x_type == LORA_BF16)
    e = N % 8 == 0 ? fwd<kBf16, 8>(x, weight, bias, w_type, eps, M, n, y, mean, rstd, st)
                   : fwd<kBf16, 1>(x, weight, bias, w_type, eps, M, n, y, mean, rstd, st);
  else
    e = N % 4 == 0 ? fwd<kF32, 4>(x, weight, bias, w_type, eps, M, n, y, mean, rstd, st)
                   : fwd<kF32, 1>(x, weight, bias, w_type, eps, M, n, y, mean, rstd, st);
  return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

size_t lora_layer_norm_bwd_workspace_size(int64_t M, int64_t N) {
  if (!size_ok(M) || !size_ok(N) || N < 1) return 0;
  return round256(size_t(M ? parts_of(M, N) : 1) * 2 * size_t(N) * 4);
}

lora_status lora_layer_norm_bwd(const void* dy, int type, const void* x, const void* x_scales, const void* weight,
                                int w_type, const float* mean, const float* rstd, int64_t M, int64_t N, void* dx,
                                float* dw, float* db, void* workspace, size_t workspace_bytes, void* stream) {
  if (!size_ok(M) || !size_ok(N) || N < 1 || !type_ok(type) || !type_ok(w_type)) return LORA_ERR_SHAPE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  lora_status s;
  int nsm = 0;
  if (M == 0) {                                     // sums over no rows
    if ((s = check_ptrs(dw)) != LORA_OK) return s;
    if (db && !aligned16(db)) return LORA_ERR_ALIGN;
    if ((s = device_ready(&nsm)) != LORA_OK) return s;
    if (cudaMemsetAsync(dw, 0, size_t(N) * 4, st) != cudaSuccess) return LORA_ERR_CUDA;
    if (db && cudaMemsetAsync(db, 0, size_t(N) * 4, st) != cudaSuccess) return LORA_ERR_CUDA;
    return LORA_OK;
  }
  if ((s = check_ptrs(dy, x, weight, mean, rstd, dx, dw, workspace)) != LORA_OK) return s;
  if ((db && !aligned16(db)) || (x_scales && !aligned16(x_scales))) return LORA_ERR_ALIGN;
  if (workspace_bytes < lora_layer_norm_bwd_workspace_size(M, N)) return LORA_ERR_WORKSPACE;
  if ((s = device_ready(&nsm)) != LORA_OK) return s;
  float* part = static_cast<float*>(workspace);
  const int P = parts_of(M, N), n = int(N);
  const bool bf = type == LORA_BF16, vec = N % (bf ? 8 : 4) == 0, d = db != nullptr;
  auto go = [&](auto f) { return f(dy, x, x_scales, weight, w_type, mean, rstd, M, n, dx, part, P, d, st); };
  cudaError_t e;
  if (bf && vec) e = x_scales ? go(bwd<kBf16, kPacked, 8>) : go(bwd<kBf16, kBf16, 8>);
  else if (bf) e = x_scales ? go(bwd<kBf16, kPacked, 1>) : go(bwd<kBf16, kBf16, 1>);
  else if (vec) e = x_scales ? go(bwd<kF32, kPacked, 4>) : go(bwd<kF32, kF32, 4>);
  else e = x_scales ? go(bwd<kF32, kPacked, 1>) : go(bwd<kF32, kF32, 1>);
  if (e != cudaSuccess) return LORA_ERR_CUDA;
  const int64_t cols = (d ? 2 : 1) * N;
  e = launch_pdl(ln_parts_kernel, dim3(unsigned(cdiv(cols, 32))), dim3(256), 0, st, static_cast<const float*>(part), P,
                 cols, N, dw, db);
  return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

}  // extern "C"
