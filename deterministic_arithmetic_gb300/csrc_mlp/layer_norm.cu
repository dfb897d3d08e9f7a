// layer_norm.cu -- layer norm over rows of N elements, forward and backward:
//   mean = sum(x) / N    var = sum((x - mean)^2) / N    rstd = 1 / sqrt(var + eps)
//   y  = xh w + b,  xh = (x - mean) rstd
//   dx = rstd (g - mean(g) - xh mean(g xh)),  g = dy w;    dw = sum_m dy xh;    db = sum_m dy
//
// All of it is bound by HBM: each element of x (and dy) is read once, each output
// written once. A row group of W warps owns a row, a thread 16 columns of it (8192
// columns in 16 warps; longer rows take the looped kernels at the end). CTAs stay
// and take rows in turn. Every thread copies its own 16 elements of the rows to
// come into its own part of shared memory (cp.async, three rows deep) and reads
// back only what it copied itself, so the loads of several rows are in flight with
// no barrier and no registers spent on them; the row's sums take the loop's only
// barriers. Measured at 8192 x 4096 bf16: 23 us forward, 41 us backward (37 and the
// partials' sum). Before the column sums were stored four at a time (8 us of the backward
// pass) the ways to bring the rows were compared: loads straight into registers 43 and
// 65 us, bulk copies and mbarriers 31 and 49 (the copying thread's work a row held up its
// CTA's barriers), this one 23 and 49.
//
// The forward pass runs at the memory's rate (5.8 TB/s), and so does the backward pass on
// FP32 rows (6.1). On bf16 rows the backward pass is bound by a warp's chain a row: 361
// instructions for 512 columns, and the sums' shuffles, of which 16 warps on an SM (128
// registers a thread, 48 of them the weight and the column sums) issue one every second
// cycle. Twice the warps with 8 columns a thread took 24 us more and two rows to a barrier 7
// more: both add instructions to a row.
//
// W and each thread's columns follow from N alone, so a row's sums are added in
// the same order in any batch. The variance is the sum of squares about the mean,
// from values in registers: no cancellation, and no second read.
//
// The backward pass's column sums: a thread keeps dw and db of its 16 columns in
// registers over all rows its group visits (rows dealt round robin over the grid),
// the row groups of a CTA add up in shared memory, and each CTA leaves one partial
// row; a second kernel adds the partials in order. The number of CTAs depends on M
// and N only, so reruns give the same bits on any device.
#include <algorithm>

#include "../csrc/common.cuh"
#include "../csrc/kernels.h"
#include "elems.cuh"
#include "mlp.h"

namespace mlp {
namespace {

using namespace lora;

constexpr int kPerThread = 16;                      // columns of a row a thread owns
constexpr int kMaxWarps = 16;                       // warps of a row group
constexpr int kHeldN = 32 * kPerThread * kMaxWarps; // longest row a group owns
constexpr int kBlockWarps = 8;                      // warps of a CTA of short rows (several groups)
// The forward kernel is built for CTAs of up to 8, 12 and 16 warps, with the registers that this many
// CTAs on an SM leave a thread (5120 columns, bf16: 34.7 us with the 16-warp build, 27.0 with the 12).
constexpr int kMidWarps = 12;
constexpr int fwd_ctas(int warps) { return warps == 8 ? 3 : (warps == 12 ? 2 : 1); }
// Rows a thread has in hand, the current one and those to come. Three leave two CTAs of 256 threads (or
// one of 512) their shared memory in the backward pass on FP32 rows; more did nothing for bf16 rows either
// (8192 x 4096, forward and backward: 22.5 and 40.9 us with three, 23.0 and 41.3 with four, 24.2 and 42.5
// with six).
constexpr int kStages = 3;
constexpr int kSMs = 152, kMaxParts = 3 * kSMs;     // partial rows of dw and db (parts_of)

inline int warps_per_row(int64_t n) { return int(cdiv(n, 32 * kPerThread)); }
inline int groups_per_block(int w) { return w >= kBlockWarps ? 1 : kBlockWarps / w; }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A thread's 16 elements of a row: VEC at a time from column (i 32 W + t) VEC, of which the first nv
// vectors lie inside the row; the rest count as 0.
template <int VEC>
__device__ __forceinline__ int vectors_inside(int N, int W, int t) {
  const int left = N / VEC - t;                      // VEC > 1 divides N
  return left <= 0 ? 0 : min(kPerThread / VEC, (left + 32 * W - 1) / (32 * W));
}

template <int KIND>
constexpr int kElemBytes = KIND == kF32 ? 4 : (KIND == kBf16 ? 2 : 1);

// One vector of VEC elements, from memory or shared memory, as FP32.
template <int KIND, int VEC>
__device__ __forceinline__ void vec_at(const uint8_t* p, float* o) {
  if constexpr (KIND == kF32) {
    if constexpr (VEC >= 4) {
#pragma unroll
      for (int j = 0; j < VEC / 4; ++j) {
        const float4 q = reinterpret_cast<const float4*>(p)[j];
        o[4 * j] = q.x; o[4 * j + 1] = q.y; o[4 * j + 2] = q.z; o[4 * j + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] = reinterpret_cast<const float*>(p)[j];
    }
  } else if constexpr (KIND == kBf16) {
    if constexpr (VEC == 1) {
      o[0] = __uint_as_float(uint32_t(*reinterpret_cast<const uint16_t*>(p)) << 16);
    } else {
      uint32_t w[VEC / 2];
      if constexpr (VEC == 8) {
        const uint4 q = *reinterpret_cast<const uint4*>(p);
        w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
      } else if constexpr (VEC == 4) {
        const uint2 q = *reinterpret_cast<const uint2*>(p);
        w[0] = q.x; w[1] = q.y;
      } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
      }
#pragma unroll
      for (int j = 0; j < VEC / 2; ++j) {
        o[2 * j] = __uint_as_float(w[j] << 16);
        o[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
  } else if constexpr (VEC >= 4) {
    // codes as FP32: 2^23 + (code + 128) has the byte at the bottom, and the difference is exact
#pragma unroll
    for (int j = 0; j < VEC / 4; ++j) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(p)[j] ^ 0x80808080u;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[4 * j + e] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440u + e)) - 8388736.f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) o[j] = float(reinterpret_cast<const int8_t*>(p)[j]);
  }
}

// The rows of one tensor as a thread sees them. Vectors of 4, 8 or 16 bytes pass through the
// thread's slots in shared memory, kStages rows deep; smaller ones are read when they are needed.
template <int KIND, int VEC>
struct Feed {
  static constexpr int kBytes = kElemBytes<KIND> * VEC, NV = kPerThread / VEC;
  static constexpr bool kAsync = kBytes >= 4;
  static constexpr int kSlots = kAsync ? kStages * kPerThread * kElemBytes<KIND> : 0;   // bytes of shared memory a thread
  const uint8_t* src;               // the thread's first vector of the next row to copy (or to read)
  int64_t row_step;                 // bytes from a row of this group to its next
  uint32_t smem;                    // the thread's slots: [stage][vector][thread of the CTA]
  const uint8_t* slots;
  int vec_step;                     // bytes between the thread's vectors of a row
  __device__ __forceinline__ Feed(const void* base, int64_t ld, uint32_t row, uint32_t stride, int W, int t, uint8_t* area)
      : src(static_cast<const uint8_t*>(base) + (int64_t(row) * ld + t * VEC) * kElemBytes<KIND>),
        row_step(int64_t(stride) * ld * kElemBytes<KIND>), smem(smem_u32(area) + threadIdx.x * kBytes),
        slots(area + threadIdx.x * kBytes), vec_step(32 * W * kBytes) {}
  // Copies the next row's vectors into stage `st` (nothing when there is no such row).
  __device__ __forceinline__ void copy(int st, bool any, int nv) {
    if constexpr (kAsync) {
      if (any) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (i < nv) {
            const uint32_t dst = smem + (st * NV + i) * blockDim.x * kBytes;
            if constexpr (kBytes == 16)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src + i * vec_step) : "memory");
            else
              asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src + i * vec_step), "n"(kBytes) : "memory");
          }
        src += row_step;
      }
    }
  }
  // The current row's elements, from stage `st`.
  __device__ __forceinline__ void get(int st, int nv, float (&v)[kPerThread]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i < nv) {
        vec_at<KIND, VEC>(kAsync ? slots + (st * NV + i) * blockDim.x * kBytes : src + i * vec_step, &v[VEC * i]);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[VEC * i + e] = 0.f;
      }
    }
    if constexpr (!kAsync) src += row_step;
  }
};
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest kStages - 1 rows' copies of this thread have landed.
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory"); }

// The thread's 16 parameters.
template <int VEC>
__device__ __forceinline__ void params16(const void* p, int type, int nv, int W, int t, float (&v)[kPerThread]) {
#pragma unroll
  for (int i = 0; i < kPerThread / VEC; ++i) {
    const int c = (i * 32 * W + t) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[VEC * i + e] = 0.f;
    if (i < nv) {
      if (type == kBf16) vec_at<kBf16, VEC>(static_cast<const uint8_t*>(p) + 2 * c, &v[VEC * i]);
      else vec_at<kF32, VEC>(static_cast<const uint8_t*>(p) + 4 * c, &v[VEC * i]);
    }
  }
}
// Stores 16 elements to the row that starts at `row`, rounded once.
template <int KIND, int VEC>
__device__ __forceinline__ void store16(uint8_t* row, int nv, int W, int t, const float (&v)[kPerThread]) {
#pragma unroll
  for (int i = 0; i < kPerThread / VEC; ++i) {
    if (i >= nv) continue;
    float o[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[e] = v[VEC * i + e];
    store_vec<KIND, VEC>(row, (i * 32 * W + t) * VEC, o);
  }
}

// The thread's 16 column sums to and from a row of floats (16-byte aligned), four at a time where its
// columns lie so (8192 x 4096 bf16 backward: 49 us one at a time, a sector a lane and store; 41 so).
template <int VEC>
__device__ __forceinline__ void put_sums16(float* row, int nv, int W, int t, const float (&v)[kPerThread]) {
  constexpr int S = VEC >= 4 ? 4 : 1;
#pragma unroll
  for (int k = 0; k < kPerThread; k += S)
    if (k / VEC < nv) {
      float* at = row + (k / VEC * 32 * W + t) * VEC + k % VEC;
      if constexpr (S == 4) *reinterpret_cast<float4*>(at) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
      else *at = v[k];
    }
}
template <int VEC>
__device__ __forceinline__ void add_sums16(const float* row, int nv, int W, int t, float (&v)[kPerThread]) {
  constexpr int S = VEC >= 4 ? 4 : 1;
#pragma unroll
  for (int k = 0; k < kPerThread; k += S)
    if (k / VEC < nv) {
      const float* at = row + (k / VEC * 32 * W + t) * VEC + k % VEC;
      if constexpr (S == 4) {
        const float4 a = *reinterpret_cast<const float4*>(at);
        v[k] += a.x; v[k + 1] += a.y; v[k + 2] += a.z; v[k + 3] += a.w;
      } else {
        v[k] += *at;
      }
    }
}

// Four partial sums in step, then their tree.
struct Sum4 {
  float a[4] = {0.f, 0.f, 0.f, 0.f};
  __device__ __forceinline__ float total() const { return (a[0] + a[1]) + (a[2] + a[3]); }
};

// The sums of a row group's W warps (a warp's in every lane), in an order that W alone sets. `slots`:
// the group's slots_of(W) floats a sum (whole 16-byte reads; those past W are 0), written before and
// read behind one CTA barrier.
__host__ __device__ constexpr int slots_of(int W) { return (W + 3) & ~3; }
constexpr int kSlots = 32;                              // of a CTA: 8 groups of 4, or 1 of 16
__device__ __forceinline__ float group_sum(const float* slots, int W) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxWarps; i += 4) {
    if (i >= W) break;
    const float4 v = *reinterpret_cast<const float4*>(slots + i);
    s += (v.x + v.y) + (v.z + v.w);
  }
  return s;
}
__device__ __forceinline__ void clear_slots(float* slots, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) slots[i] = 0.f;
}


template <int KIND, int VEC, bool FULL, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, fwd_ctas(WARPS))
    ln_fwd_kernel(const void* __restrict__ x, const void* __restrict__ weight, const void* __restrict__ bias, int w_type,
                  float eps, uint32_t M, int N, int W, void* __restrict__ y, float* __restrict__ mean_out,
                  float* __restrict__ rstd_out) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float red[2][kSlots];
  clear_slots(&red[0][0], 2 * kSlots);
  const int warp = threadIdx.x >> 5, group = warp / W, groups = (blockDim.x >> 5) / W;
  const int t = (warp - group * W) * 32 + (threadIdx.x & 31);
  const int slot0 = group * slots_of(W), slot = slot0 + warp - group * W;
  const int nv = FULL ? kPerThread / VEC : vectors_inside<VEC>(N, W, t);
  const uint32_t stride = gridDim.x * groups;          // M + kStages * stride < 2^32
  uint32_t row = blockIdx.x * groups + group, ahead = row;
  __syncthreads();                   // the cleared slots
  grid_dependency_wait();
  grid_dependents_launch();
  Feed<KIND, VEC> feed(x, N, row, stride, W, t, smem);
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s, ahead += stride) {
    feed.copy(s, ahead < M, nv);
    copies_commit();
  }
  float w[kPerThread], b[kPerThread];
  params16<VEC>(weight, w_type, nv, W, t, w);
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) b[i] = 0.f;
  if (bias) params16<VEC>(bias, w_type, nv, W, t, b);
  const float inv_n = __fdiv_rn(1.f, float(N));
  uint8_t* out = static_cast<uint8_t*>(y) + int64_t(row) * N * kElemBytes<KIND>;
  const int64_t out_step = int64_t(stride) * N * kElemBytes<KIND>;
  for (int st = 0; row < M; row += stride, out += out_step, st = (st + 1) % kStages, ahead += stride) {
    feed.copy((st + kStages - 1) % kStages, ahead < M, nv);
    copies_commit();
    copies_wait();
    float v[kPerThread];
    Sum4 s, q;
    feed.get(st, nv, v);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) s.a[i & 3] += v[i];
    float sum = warp_sum(s.total());
    if (W > 1) {
      if ((threadIdx.x & 31) == 0) red[0][slot] = sum;
      named_bar(1 + group, 32 * W);
      sum = group_sum(&red[0][slot0], W);
    }
    const float mean = sum * inv_n;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) v[i] -= mean;
    if (nv < kPerThread / VEC) {     // an element outside the row counts for nothing
#pragma unroll
      for (int i = 0; i < kPerThread; ++i)
        if (i / VEC >= nv) v[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) q.a[i & 3] = fmaf(v[i], v[i], q.a[i & 3]);
    float sq = warp_sum(q.total());
    if (W > 1) {
      // two barriers a row: each sum's slots are written again only behind the other's barrier
      if ((threadIdx.x & 31) == 0) red[1][slot] = sq;
      named_bar(1 + group, 32 * W);
      sq = group_sum(&red[1][slot0], W);
    }
    const float rstd = rsqrtf(fmaf(sq, inv_n, eps));
    if (t == 0) {
      mean_out[row] = mean;
      rstd_out[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) v[i] = fmaf(v[i] * rstd, w[i], b[i]);
    store16<KIND, VEC>(out, nv, W, t, v);
  }
}

// XK: the kind of x (KIND, or packed). part: [gridDim.x][ld], a row the sums of dw, then (from N) of db.
template <int KIND, int XK, int VEC, bool FULL, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, WARPS == kMaxWarps ? 1 : 2)
    ln_bwd_kernel(const void* __restrict__ dy, const void* __restrict__ x, const void* __restrict__ x_scales,
                  const void* __restrict__ weight, int w_type, const float* __restrict__ mean_in,
                  const float* __restrict__ rstd_in, uint32_t M, int N, int W, void* __restrict__ dx,
                  float* __restrict__ part, int64_t ld, int with_db) {
  constexpr int NV = kPerThread / VEC;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float red[2][2][kSlots];     // [row parity][sum]
  clear_slots(&red[0][0][0], 4 * kSlots);
  const int warp = threadIdx.x >> 5, group = warp / W, groups = (blockDim.x >> 5) / W;
  const int t = (warp - group * W) * 32 + (threadIdx.x & 31);
  const int slot0 = group * slots_of(W), slot = slot0 + warp - group * W;
  const int nv = FULL ? NV : vectors_inside<VEC>(N, W, t);
  const uint32_t stride = gridDim.x * groups;          // M + kStages * stride < 2^32
  uint32_t row = blockIdx.x * groups + group, ahead = row;
  __syncthreads();                   // the cleared slots
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t x_ld = row_ld<XK>(N);
  Feed<KIND, VEC> feed_dy(dy, N, row, stride, W, t, smem);
  Feed<XK, VEC> feed_x(x, x_ld, row, stride, W, t, smem + Feed<KIND, VEC>::kSlots * blockDim.x);
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s, ahead += stride) {
    feed_dy.copy(s, ahead < M, nv);
    feed_x.copy(s, ahead < M, nv);
    copies_commit();
  }
  const float inv_n = __fdiv_rn(1.f, float(N));
  float w[kPerThread], dw[kPerThread], db[kPerThread];
  params16<VEC>(weight, w_type, nv, W, t, w);
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) dw[i] = db[i] = 0.f;
  // what a row needs besides its elements is loaded a row ahead
  float next_mean = 0.f, next_rstd = 0.f;
  // The scale bytes of a warp's vectors: a thread's own of each, or, where a vector is 1 or 2 elements and
  // the warp's 16 groups therefore more than its loads are worth, a group a lane.
  constexpr bool kShared = XK == kPacked && VEC <= 2;
  const int lane = threadIdx.x & 31, group0 = (lane / VEC * W + (t >> 5)) * VEC + lane % VEC;
  uint8_t next_scale[kShared ? 1 : NV];
  auto look_ahead = [&](uint32_t r) {
    if (r >= M) return;
    next_mean = mean_in[r];
    next_rstd = rstd_in[r];
    if constexpr (XK == kPacked) {
      const uint8_t* sc = static_cast<const uint8_t*>(x_scales) + int64_t(r) * (x_ld >> 5);
      if constexpr (kShared) {
        next_scale[0] = lane < kPerThread && group0 < int(x_ld >> 5) ? sc[group0] : uint8_t(0);
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (i < nv) next_scale[i] = sc[((i * 32 * W + t) * VEC) >> 5];
      }
    }
  };
  look_ahead(row);
  uint8_t* out = static_cast<uint8_t*>(dx) + int64_t(row) * N * kElemBytes<KIND>;
  const int64_t out_step = int64_t(stride) * N * kElemBytes<KIND>;
  int parity = 0;
  for (int st = 0; row < M; row += stride, out += out_step, st = (st + 1) % kStages, ahead += stride) {
    const bool any = ahead < M;
    feed_dy.copy((st + kStages - 1) % kStages, any, nv);
    feed_x.copy((st + kStages - 1) % kStages, any, nv);
    copies_commit();
    const float mean = next_mean, rstd = next_rstd;
    float step[NV];
    if constexpr (kShared) {
      const float own = scale_step(next_scale[0]);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float s = __shfl_sync(0xffffffffu, own, i * VEC + lane * VEC / 32);
        step[i] = i < nv ? s : 0.f;
      }
    } else if constexpr (XK == kPacked) {
#pragma unroll
      for (int i = 0; i < NV; ++i) step[i] = i < nv ? scale_step(next_scale[i]) : 0.f;
    }
    look_ahead(row + stride);
    copies_wait();
    float g[kPerThread], xh[kPerThread];
    Sum4 s1, s2;
    feed_dy.get(st, nv, g);
    feed_x.get(st, nv, xh);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {               // elements outside the row have dy = 0
      if constexpr (XK == kPacked) xh[i] *= step[i / VEC];
      xh[i] = (xh[i] - mean) * rstd;
      dw[i] = fmaf(g[i], xh[i], dw[i]);
      db[i] += g[i];
      g[i] *= w[i];
      s1.a[i & 3] += g[i];
      s2.a[i & 3] = fmaf(g[i], xh[i], s2.a[i & 3]);
    }
    float g_sum = warp_sum(s1.total()), gx_sum = warp_sum(s2.total());
    if (W > 1) {
      // one barrier a row: the next one's sums use the other half of `red`, and the one after that
      // writes this half only behind the next one's barrier
      if ((threadIdx.x & 31) == 0) red[parity][0][slot] = g_sum, red[parity][1][slot] = gx_sum;
      named_bar(1 + group, 32 * W);
      g_sum = group_sum(&red[parity][0][slot0], W);
      gx_sum = group_sum(&red[parity][1][slot0], W);
      parity ^= 1;
    }
    // dx = rstd g - rstd c1 - xh rstd c2
    const float c1 = -rstd * (g_sum * inv_n), c2 = -rstd * (gx_sum * inv_n);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) g[i] = fmaf(xh[i], c2, fmaf(g[i], rstd, c1));
    store16<KIND, VEC>(out, nv, W, t, g);
  }
  // the row groups' column sums, added in group order; the slots' memory holds them
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  float* cols = reinterpret_cast<float*>(smem);
  if (group > 0) {
    put_sums16<VEC>(cols + size_t(group - 1) * 2 * N, nv, W, t, dw);
    put_sums16<VEC>(cols + size_t(group - 1) * 2 * N + N, nv, W, t, db);
  }
  __syncthreads();
  if (group == 0) {
    for (int k = 1; k < groups; ++k) {
      add_sums16<VEC>(cols + size_t(k - 1) * 2 * N, nv, W, t, dw);
      add_sums16<VEC>(cols + size_t(k - 1) * 2 * N + N, nv, W, t, db);
    }
    float* sums = part + int64_t(blockIdx.x) * ld;
    put_sums16<VEC>(sums, nv, W, t, dw);
    if (with_db) put_sums16<VEC>(sums + N, nv, W, t, db);
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
    const float rstd = rsqrtf(__fdiv_rn(block_sum(q, red), float(N)) + eps);
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
                        float* __restrict__ part, int64_t ld, int with_db) {
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
  float* out = part + int64_t(blockIdx.y) * ld;
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

// dw and db from the partial rows [P][ld]: 64 columns a CTA, the partials dealt over its 16 warps,
// then the warps' sums in order.
__global__ void __launch_bounds__(512)
    ln_parts_kernel(const float* __restrict__ part, int P, int64_t ld, int64_t cols, int64_t N, float* __restrict__ dw,
                    float* __restrict__ db) {
  __shared__ float2 sums[16][32];
  grid_dependency_wait();
  grid_dependents_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c = int64_t(blockIdx.x) * 64 + 2 * lane;
  float2 s = make_float2(0.f, 0.f);
  if (c < cols) {                                    // ld is even: the pair lies inside the row
    constexpr int kDeep = (kMaxParts + 15) / 16;
    float2 v[kDeep];                                 // all loads in flight together
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      const int p = warp + 16 * i;
      v[i] = p < P ? __ldcg(reinterpret_cast<const float2*>(part + int64_t(p) * ld + c)) : make_float2(0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < kDeep; ++i) s.x += v[i].x, s.y += v[i].y;
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (threadIdx.x < 64) {
    const int64_t col = int64_t(blockIdx.x) * 64 + threadIdx.x;
    if (col < cols) {
      float a = 0.f;
      for (int k = 0; k < 16; ++k) a += reinterpret_cast<const float*>(&sums[k][0])[threadIdx.x];
      if (col < N) dw[col] = a;
      else db[col - N] = a;
    }
  }
}

template <class K>
cudaError_t set_smem(K* kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}
// Shared memory of the slots of a CTA of `threads`, and (backward) of the row groups' column sums.
template <int KIND, int VEC>
int fwd_smem(int threads) { return threads * Feed<KIND, VEC>::kSlots; }
template <int KIND, int XK, int VEC>
int bwd_smem(int threads) {
  const int slots = threads * (Feed<KIND, VEC>::kSlots + Feed<XK, VEC>::kSlots);
  const int sums = (kBlockWarps - 1) * 2 * 32 * kPerThread * 4;       // at most 7 groups of 512 columns
  return slots > sums ? slots : sums;
}

// Partial rows of a backward pass, one a CTA: as many CTAs as the 152 SMs hold at once of 128 registers
// a thread (three of 160 threads, two of 256, one above), and no more than there are rows for.
constexpr int kLongParts = 64;
int parts_of(int64_t M, int64_t N) {
  if (N > kHeldN) return int(std::min<int64_t>(cdiv(M, kBlockWarps), kLongParts));
  const int W = warps_per_row(N), G = groups_per_block(W), held = 512 / (32 * W * G);
  return int(std::min<int64_t>(cdiv(M, G), kSMs * std::max(1, std::min(held, kMaxParts / kSMs))));
}
int64_t part_ld(int64_t N) { return (2 * N + 3) & ~int64_t(3); }

template <int KIND, int VEC>
cudaError_t fwd(const void* x, const void* w, const void* b, int w_type, float eps, int64_t M, int64_t N, void* y,
                float* mean, float* rstd, int nsm, cudaStream_t st) {
  if (N > kHeldN) {
    const int64_t grid = M < nsm * 4 ? M : nsm * 4;
    return launch_pdl(ln_fwd_long_kernel<KIND, VEC>, dim3(unsigned(grid)), dim3(kLongThreads), 0, st, x, w, b, w_type,
                      eps, M, int(N), y, mean, rstd);
  }
  const int W = warps_per_row(N), G = groups_per_block(W), threads = 32 * W * G;
  const int built = threads <= 32 * kBlockWarps ? kBlockWarps : (threads <= 32 * kMidWarps ? kMidWarps : kMaxWarps);
  // what an SM holds at once: 80 registers a thread (128 in the 16-warp build)
  const int64_t work = cdiv(M, G), most = int64_t(nsm) * std::max(1, (built == kMaxWarps ? 512 : 800) / threads);
  const dim3 grid(unsigned(work < most ? work : most));
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(threads), fwd_smem<KIND, VEC>(threads), st, x, w, b, w_type, eps, uint32_t(M),
                      int(N), W, y, mean, rstd);
  };
  // rows that fill their threads exactly take kernels without tests of the row's end (8192 x 4096 bf16: 22.5
  // against 24.1 us, backward 40.6 against 43.9)
  constexpr bool vec = VEC > 2;
  const bool full = vec && N == 32 * kPerThread * W;
  if (built == kBlockWarps)
    return full ? go(ln_fwd_kernel<KIND, VEC, vec, kBlockWarps>) : go(ln_fwd_kernel<KIND, VEC, false, kBlockWarps>);
  if (built == kMidWarps)
    return full ? go(ln_fwd_kernel<KIND, VEC, vec, kMidWarps>) : go(ln_fwd_kernel<KIND, VEC, false, kMidWarps>);
  return full ? go(ln_fwd_kernel<KIND, VEC, vec, kMaxWarps>) : go(ln_fwd_kernel<KIND, VEC, false, kMaxWarps>);
}

template <int KIND, int XK, int VEC>
cudaError_t bwd(const void* dy, const void* x, const void* xs, const void* w, int w_type, const float* mean,
                const float* rstd, int64_t M, int64_t N, void* dx, float* part, bool with_db, int nsm, int* parts,
                cudaStream_t st) {
  const int64_t ld = part_ld(N);
  *parts = parts_of(M, N);
  if (N > kHeldN) {
    const int64_t grid = M < nsm * 4 ? M : nsm * 4;
    const cudaError_t err = launch_pdl(ln_dx_long_kernel<KIND, XK, VEC>, dim3(unsigned(grid)), dim3(kLongThreads), 0, st,
                                       dy, x, xs, w, w_type, mean, rstd, M, int(N), dx);
    if (err != cudaSuccess) return err;
    return launch_pdl(ln_cols_long_kernel<KIND, XK, VEC>, dim3(unsigned(cdiv(N, 32 * VEC)), unsigned(*parts)),
                      dim3(32 * kBlockWarps), 0, st, dy, x, xs, mean, rstd, M, int(N), part, ld, int(with_db));
  }
  const int W = warps_per_row(N), G = groups_per_block(W), threads = 32 * W * G;
  const dim3 grid = dim3(unsigned(*parts));
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(threads), bwd_smem<KIND, XK, VEC>(threads), st, dy, x, xs, w, w_type, mean, rstd,
                      uint32_t(M), int(N), W, dx, part, ld, int(with_db));
  };
  constexpr bool vec = VEC > 2;
  const bool full = vec && N == 32 * kPerThread * W;
  if (threads <= 32 * kBlockWarps)
    return full ? go(ln_bwd_kernel<KIND, XK, VEC, vec, kBlockWarps>) : go(ln_bwd_kernel<KIND, XK, VEC, false, kBlockWarps>);
  return full ? go(ln_bwd_kernel<KIND, XK, VEC, vec, kMaxWarps>) : go(ln_bwd_kernel<KIND, XK, VEC, false, kMaxWarps>);
}

template <int KIND, int VEC, bool FULL>
cudaError_t prepare_as() {
  cudaError_t e = cudaSuccess;
  auto fwd_ok = [&](auto kernel, int warps) { return (e = set_smem(kernel, fwd_smem<KIND, VEC>(32 * warps))) == cudaSuccess; };
  auto bwd_ok = [&](auto kernel, auto packed, int warps) {
    return (e = set_smem(kernel, bwd_smem<KIND, KIND, VEC>(32 * warps))) == cudaSuccess &&
           (e = set_smem(packed, bwd_smem<KIND, kPacked, VEC>(32 * warps))) == cudaSuccess;
  };
  fwd_ok(ln_fwd_kernel<KIND, VEC, FULL, kBlockWarps>, kBlockWarps) &&
      fwd_ok(ln_fwd_kernel<KIND, VEC, FULL, kMidWarps>, kMidWarps) &&
      fwd_ok(ln_fwd_kernel<KIND, VEC, FULL, kMaxWarps>, kMaxWarps) &&
      bwd_ok(ln_bwd_kernel<KIND, KIND, VEC, FULL, kBlockWarps>, ln_bwd_kernel<KIND, kPacked, VEC, FULL, kBlockWarps>, kBlockWarps) &&
      bwd_ok(ln_bwd_kernel<KIND, KIND, VEC, FULL, kMaxWarps>, ln_bwd_kernel<KIND, kPacked, VEC, FULL, kMaxWarps>, kMaxWarps);
  return e;
}
template <int KIND, int VEC>
cudaError_t prepare() {
  const cudaError_t e = prepare_as<KIND, VEC, false>();
  return e == cudaSuccess && VEC > 2 ? prepare_as<KIND, VEC, (VEC > 2)>() : e;
}

}  // namespace

cudaError_t prepare_layer_norm() {
  cudaError_t e;
  if ((e = prepare<kBf16, 8>()) != cudaSuccess || (e = prepare<kBf16, 2>()) != cudaSuccess ||
      (e = prepare<kBf16, 1>()) != cudaSuccess || (e = prepare<kF32, 4>()) != cudaSuccess)
    return e;
  return prepare<kF32, 1>();
}

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
  auto go = [&](auto f) { return f(x, weight, bias, w_type, eps, M, N, y, mean, rstd, nsm, st); };
  const cudaError_t e = x_type == LORA_F32 ? (N % 4 == 0 ? go(fwd<kF32, 4>) : go(fwd<kF32, 1>))
                        : N % 8 == 0       ? go(fwd<kBf16, 8>)
                        : N % 2 == 0       ? go(fwd<kBf16, 2>)
                                           : go(fwd<kBf16, 1>);
  return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

size_t lora_layer_norm_bwd_workspace_size(int64_t M, int64_t N) {
  if (!size_ok(M) || !size_ok(N) || N < 1) return 0;
  return round256(size_t(M ? parts_of(M, N) : 1) * size_t(part_ld(N)) * 4);
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
  const bool d = db != nullptr;
  int P = 0;
  auto go = [&](auto f) { return f(dy, x, x_scales, weight, w_type, mean, rstd, M, N, dx, part, d, nsm, &P, st); };
  cudaError_t e;
  if (type == LORA_F32 && N % 4 == 0) e = x_scales ? go(bwd<kF32, kPacked, 4>) : go(bwd<kF32, kF32, 4>);
  else if (type == LORA_F32) e = x_scales ? go(bwd<kF32, kPacked, 1>) : go(bwd<kF32, kF32, 1>);
  else if (N % 8 == 0) e = x_scales ? go(bwd<kBf16, kPacked, 8>) : go(bwd<kBf16, kBf16, 8>);
  else if (N % 2 == 0) e = x_scales ? go(bwd<kBf16, kPacked, 2>) : go(bwd<kBf16, kBf16, 2>);
  else e = x_scales ? go(bwd<kBf16, kPacked, 1>) : go(bwd<kBf16, kBf16, 1>);
  if (e != cudaSuccess) return LORA_ERR_CUDA;
  const int64_t cols = (d ? 2 : 1) * N;
  e = launch_pdl(ln_parts_kernel, dim3(unsigned(cdiv(cols, 64))), dim3(512), 0, st, static_cast<const float*>(part), P,
                 part_ld(N), cols, N, dw, db);
  return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

}  // extern "C"
