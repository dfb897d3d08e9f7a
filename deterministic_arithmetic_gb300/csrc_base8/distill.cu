// distill.cu -- the loss against a teacher's top logits, forward and backward (lora_distill_topk_* of
// include/lora_base8.h).
//
// A row of logits is read once a pass. The forward pass holds a running maximum and the sum of exponentials
// relative to it, of everything that is no entry of the teacher's; the row's few entries are read on their own, and
// their part joined at the end. So the mass of the rest is a sum, and no difference. Bound by HBM.
//
// A row is cut into groups of 256 elements, dealt in turn to 64 places (8 of a CTA's 8 warps each); each
// thread of a place holds a maximum and a sum of its own, and the places' are joined in a fixed order. A batch of
// few rows has its rows' places spread over the CTAs of a cluster: the places, and so the bits, stay the same.
#include "../csrc/common.cuh"
#include "../csrc/kernels.h"
#include "../csrc_mlp/elems.cuh"
#include "base8.h"
#include "block8.cuh"

namespace mlp {
namespace {

using namespace lora;

constexpr int kThreads = 256, kWarps = 8, kGroupElems = 256, kPlaces = 8;
constexpr int kMaxTop = 1024;
constexpr float kLog2e = 1.4426950408889634f, kInf = __builtin_huge_valf();

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What a thread holds of a group of 256 elements of its warp: 8 of them, in pieces of VEC consecutive ones, 32 VEC apart. VEC
// is what rows of V elements allow (16 bytes where whole vectors fit a row).
template <int KIND, int VEC>
struct Held {
  static constexpr int kWords = KIND == kF32 ? 8 : 4;
  uint32_t w[kWords];
  static __device__ __forceinline__ int at(int e, int lane) { return (e / VEC) * 32 * VEC + lane * VEC + e % VEC; }
  // Elements of the group at p, of which `n` exist; the others are -infinity.
  __device__ __forceinline__ void load(const void* p, int64_t base, int n, int lane) {
    if constexpr (KIND == kBf16 && VEC == 8) {
      if (8 * lane < n) {
        const uint4 t = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + base + 8 * lane);
        w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
      } else {
        w[0] = w[1] = w[2] = w[3] = 0xFF80FF80u;
      }
    } else if constexpr (KIND == kBf16 && VEC == 2) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = 64 * j + 2 * lane < n
                   ? *reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p) + base + 64 * j + 2 * lane)
                   : 0xFF80FF80u;
    } else if constexpr (KIND == kBf16) {
      const uint16_t* q = static_cast<const uint16_t*>(p) + base + lane;
      uint32_t h[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = 32 * j + lane < n ? q[32 * j] : 0xFF80u;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = h[2 * j] | (h[2 * j + 1] << 16);
    } else if constexpr (VEC == 4) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float4 t = make_float4(-kInf, -kInf, -kInf, -kInf);
        if (128 * j + 4 * lane < n) t = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + base + 128 * j + 4 * lane);
        w[4 * j] = __float_as_uint(t.x); w[4 * j + 1] = __float_as_uint(t.y);
        w[4 * j + 2] = __float_as_uint(t.z); w[4 * j + 3] = __float_as_uint(t.w);
      }
    } else {
      const float* q = static_cast<const float*>(p) + base + lane;
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(32 * j + lane < n ? q[32 * j] : -kInf);
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if constexpr (KIND == kF32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
  // Element e becomes -infinity.
  __device__ __forceinline__ void drop(int e) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (KIND == kF32) {
        if (i == e) w[i] = 0xFF800000u;
      } else {
        const uint32_t hit = i == e / 2 ? (e & 1 ? 0xFFFF0000u : 0xFFFFu) : 0u;
        w[i] = (w[i] & ~hit) | (0xFF80FF80u & hit);
      }
    }
  }
  // The largest (NaN passed over); of bf16 values by pairs.
  __device__ __forceinline__ float largest() const {
    if constexpr (KIND == kF32) {
      float m = __uint_as_float(w[0]);
#pragma unroll
      for (int i = 1; i < 8; ++i) m = fmaxf(m, __uint_as_float(w[i]));
      return m;
    } else {
      const auto pair = [](uint32_t v) { return *reinterpret_cast<const __nv_bfloat162*>(&v); };
      const __nv_bfloat162 m = __hmax2(__hmax2(pair(w[0]), pair(w[1])), __hmax2(pair(w[2]), pair(w[3])));
      return fmaxf(__low2float(m), __high2float(m));
    }
  }
  // The values, rounded once, to the same elements.
  static __device__ __forceinline__ void store(void* p, int64_t base, int n, int lane, const float (&v)[8]) {
    if constexpr (KIND == kBf16 && VEC == 8) {
      if (8 * lane < n) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + base + 8 * lane) = pack_bf16x8(v);
    } else if constexpr (KIND == kBf16 && VEC == 2) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (64 * j + 2 * lane < n)
          *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p) + base + 64 * j + 2 * lane) = bf16x2_bits(v[2 * j], v[2 * j + 1]);
    } else if constexpr (KIND == kBf16) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (32 * j + lane < n) static_cast<__nv_bfloat16*>(p)[base + 32 * j + lane] = __float2bfloat16_rn(v[j]);
    } else if constexpr (VEC == 4) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (128 * j + 4 * lane < n)
          *reinterpret_cast<float4*>(static_cast<float*>(p) + base + 128 * j + 4 * lane) =
              make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (32 * j + lane < n) static_cast<float*>(p)[base + 32 * j + lane] = v[j];
    }
  }
  // Of the lane and element that hold the group's element o.
  static __device__ __forceinline__ int lane_of(int o) { return (o / VEC) & 31; }
  static __device__ __forceinline__ int elem_of(int o) { return o / (32 * VEC) * VEC + o % VEC; }
};

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

struct DistillArgs {
  const void *z, *ids, *teacher;
  const float *teacher_lse, *weight, *dloss;
  int id8, teacher_type;           // ids in 64 bits; the teacher's type
  int64_t M;
  int V, top, groups;              // groups of 256 elements of a row
  float temperature;
  float *loss, *probs, *stats;
  void* dz;
  float* scales;
  int seg;                         // backward: groups of a CTA
};

// An id as its place in the vocabulary, -1 where it has none.
__device__ __forceinline__ int id_at(const DistillArgs& P, int64_t i) {
  if (P.id8) {
    const int64_t v = __ldg(static_cast<const long long*>(P.ids) + i);
    return v >= 0 && v < P.V ? int(v) : -1;
  }
  const int v = __ldg(static_cast<const int*>(P.ids) + i);
  return v >= 0 && v < P.V ? v : -1;
}
__device__ __forceinline__ float logit_at(const DistillArgs& P, int kind, int64_t i) { return param_at(P.z, kind, i); }

// The entries of a row by group: head[g] the first of group g, next[i] the one after entry i, -1 at the end. The
// order within a group is no fixed one; nothing depends on it.
struct Lists {
  int *head, *next, *id;           // shared memory: groups, top, top
};

// The sum (maximum) over a warp, in a fixed order; every lane has it.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Sums of exponentials relative to a maximum: value = sum * 2^((max - reference) * c). An empty one has max
// -infinity and sum 0; one with +infinity or NaN gives NaN.
struct Part {
  float m, s;
};
__device__ __forceinline__ float rescale(float s, float from, float to, float c) {
  return from == -kInf && s == 0.f ? 0.f : s * ex2((from - to) * c);
}

// ----------------------------------------------------------------- forward
// CL: CTAs of a row's cluster. Of the 8 places of a thread, CTA r has those congruent to r.
template <int KIND, int VEC, int CL>
__global__ void __launch_bounds__(kThreads, KIND == kF32 ? 2 : 3) distill_fwd_kernel(const __grid_constant__ DistillArgs P) {
  constexpr int kOwn = kPlaces / CL;               // places of a thread of this CTA
  constexpr int kLoads = KIND == kF32 ? 4 : 8;     // groups of a warp in flight
  extern __shared__ int smem[];
  __shared__ Part sent[CL > 1 ? kPlaces : 1][CL > 1 ? kThreads : 1];    // what the cluster's CTAs send to the first
  __shared__ Part warps[kWarps];
  const Lists L{smem, smem + P.groups, smem + P.groups + P.top};
  float* tl = reinterpret_cast<float*>(L.id + P.top);      // the entries' teacher logits; -infinity where dropped
  float* zl = tl + P.top;                                  // and student logits
  const int lane = int(lane_id()), warp = int(warp_id()), tid = int(threadIdx.x);
  const int rank = CL > 1 ? int(cluster_rank()) : 0;
  const int64_t row = blockIdx.x / CL;
  grid_dependency_wait();
  grid_dependents_launch();
  const float weight = P.weight ? __ldg(P.weight + row) : 1.f;
  if (weight == 0.f) {                             // the same in every CTA of the cluster
    if (rank == 0) {
      for (int i = tid; i < P.top; i += kThreads) P.probs[row * P.top + i] = -1.f;
      if (tid < 4) P.stats[row * 4 + tid] = 0.f;
      if (tid == 0) P.loss[row] = 0.f;
    }
    return;
  }
  // The groups of a warp in one sequence q: place q % kOwn of round q / kOwn. As one is taken in, the one kLoads on is sent for; the
  // first are on their way while the entries' lists are made.
  const int64_t base = row * P.V;
  const int rounds = (P.groups + kPlaces * kWarps - 1) / (kPlaces * kWarps), whole = P.V / (kPlaces * kWarps * kGroupElems);
  const auto group = [&](int q) { return q / kOwn * (kPlaces * kWarps) + (CL * (q % kOwn) + rank) * kWarps + warp; };
  Held<KIND, VEC> held[kLoads];
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    const int g = group(k);
    held[k].load(P.z, base + int64_t(g) * kGroupElems, P.V - g * kGroupElems, lane);
  }
  for (int g = tid; g < P.groups; g += kThreads) L.head[g] = -1;
  __syncthreads();
  for (int i = tid; i < P.top; i += kThreads) {
    const int64_t at = row * P.top + i;
    int id = id_at(P, at);
    const float t = param_at(P.teacher, P.teacher_type, at);
    if (t == -kInf) id = -1;
    L.id[i] = id;
    tl[i] = id < 0 ? -kInf : t;
    if (id >= 0) {
      L.next[i] = atomicExch(&L.head[id / kGroupElems], i);
      if (rank == 0) zl[i] = logit_at(P, KIND, row * P.V + id);
    }
  }
  if constexpr (CL > 1) cluster_sync_all();        // (every CTA of the cluster runs: its shared memory may be written)
  else __syncthreads();
  // of several entries of one id the first counts
  if (rank == 0)
    for (int i = tid; i < P.top; i += kThreads) {
      const int id = L.id[i];
      if (id < 0) continue;
      for (int j = L.head[id / kGroupElems]; j >= 0; j = L.next[j])
        if (j < i && L.id[j] == id) {
          tl[i] = -kInf;
          break;
        }
    }

  const float c = kLog2e / P.temperature;
  Part own[kOwn];
#pragma unroll
  for (int j = 0; j < kOwn; ++j) own[j] = {-kInf, 0.f};
  constexpr int kBatch = kOwn > kLoads ? kOwn : kLoads;
  const auto take = [&](Held<KIND, VEC>& v, Part& p, int g) {
    for (int i = L.head[g]; i >= 0; i = L.next[i]) {           // entries are no part of the rest
      const int o = L.id[i] - g * kGroupElems;
      if (Held<KIND, VEC>::lane_of(o) == lane) v.drop(Held<KIND, VEC>::elem_of(o));
    }
    const float m = v.largest();
    if (m > p.m) {
      p.s = rescale(p.s, p.m, m, c);
      p.m = m;
    }
    const float ref = p.m == -kInf ? 0.f : p.m;               // nothing but -infinity so far: all terms are 0
    float x[8];
    v.get(x);
    float2 y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      y[e] = mul2(add2(make_float2(x[2 * e], x[2 * e + 1]), make_float2(-ref, -ref)), make_float2(c, c));
      y[e] = make_float2(ex2(y[e].x), ex2(y[e].y));
    }
    const float2 t = add2(add2(y[0], y[1]), add2(y[2], y[3]));
    p.s += t.x + t.y;
  };
  int q0 = 0;
  for (; (q0 + kBatch + kLoads) <= whole * kOwn; q0 += kBatch) {       // whole groups only, the ones sent for too
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      Held<KIND, VEC>& v = held[k % kLoads];
      take(v, own[k % kOwn], group(q0 + k));
      v.load(P.z, base + int64_t(group(q0 + k + kLoads)) * kGroupElems, kGroupElems, lane);
    }
  }
#pragma unroll 1
  for (; q0 < rounds * kOwn; q0 += kBatch) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int g = group(q0 + k), next = group(q0 + k + kLoads);
      Held<KIND, VEC>& v = held[k % kLoads];
      if (g < P.groups) take(v, own[k % kOwn], g);
      v.load(P.z, base + int64_t(next) * kGroupElems, P.V - next * kGroupElems, lane);
    }
  }

  // the thread's places, in order; then the warp's lanes, the warps
  Part all[kPlaces];
  if constexpr (CL > 1) {
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      const uint32_t at = peer_addr(smem_u32(&sent[CL * j + rank][tid]), 0);
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(own[j].m), "f"(own[j].s) : "memory");
    }
    cluster_sync_all();
    if (rank != 0) return;
#pragma unroll
    for (int j = 0; j < kPlaces; ++j) all[j] = sent[j][tid];
  } else {
#pragma unroll
    for (int j = 0; j < kPlaces; ++j) all[j] = own[j];
  }
  Part t = all[0];
#pragma unroll
  for (int j = 1; j < kPlaces; ++j) t.m = fmaxf(t.m, all[j].m);
  t.m = warp_max(t.m);
  t.s = 0.f;
#pragma unroll
  for (int j = 0; j < kPlaces; ++j) t.s += rescale(all[j].s, all[j].m, t.m, c);
  t.s = warp_sum(t.s);
  if (lane == 0) warps[warp] = t;
  __syncthreads();
  if (warp != 0) return;

  // ---- the row's end, one warp. The rest of the vocabulary:
  Part rest = warps[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) rest.m = fmaxf(rest.m, warps[w].m);
  rest.s = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) rest.s += rescale(warps[w].s, warps[w].m, rest.m, c);
  // the entries': maxima, then sums
  float zm = -kInf, tm = -kInf;
  bool any = false;
  for (int i = lane; i < P.top; i += 32)
    if (tl[i] != -kInf) {
      any = true;
      zm = fmaxf(zm, zl[i]);
      tm = fmaxf(tm, tl[i]);
    }
  any = __any_sync(0xffffffffu, any);
  zm = warp_max(zm);
  tm = warp_max(tm);
  const float m = fmaxf(rest.m, zm);
  float s_top = 0.f, s_teacher = 0.f;
  for (int i = lane; i < P.top; i += 32)
    if (tl[i] != -kInf) {
      s_top += ex2((zl[i] - m) * c);
      s_teacher += ex2((tl[i] - tm) * c);
    }
  s_top = warp_sum(s_top);
  s_teacher = warp_sum(s_teacher);
  const float s_rest = rescale(rest.s, rest.m, m, c), s = s_rest + s_top;
  // log p - log q = (t - z) / T - (norm - log sum exp(z / T)): a difference of an entry's own two logits, and one of the
  // row's, taken in 64 bits. The terms of a small divergence cancel, and so keep their digits.
  const float inv_t = 1.f / P.temperature, log_s = logf(s);
  const float lse = P.teacher_lse ? __ldg(P.teacher_lse + row) : 0.f, log_t = logf(s_teacher);
  const double it = 1.0 / double(P.temperature);
  const float gap = float((P.teacher_lse ? double(lse) : double(tm) * it + double(log_t)) - (double(m) * it + double(log_s)));
  const float it_lo = float(it - double(inv_t));
  float sum_p = 0.f, loss = 0.f;
  for (int i = lane; i < P.top; i += 32) {
    const float ti = tl[i];
    float p = -1.f;
    if (ti != -kInf) {
      // t / T - lse by an exact product and its rest; (t - the largest t) / T - log of the sum
      const float h = ti * inv_t, rest_h = fmaf(ti, inv_t, -h) + ti * it_lo;
      p = expf(P.teacher_lse ? (h - lse) + rest_h : (ti - tm) * inv_t - log_t);
      sum_p += p;
      if (p != 0.f) loss += p * ((ti - zl[i]) * inv_t - gap);
    }
    P.probs[row * P.top + i] = p;
  }
  sum_p = warp_sum(sum_p);
  loss = warp_sum(loss);
  if (lane == 0) {
    float keep = 1.f;
    if (P.teacher_lse) {
      const float r = sum_p >= 1.f ? 0.f : 1.f - sum_p, ratio = s_top / s_rest;   // log rho = -log(1 + ratio)
      if (r != 0.f) loss += r * (log1pf(-sum_p) + log1pf(ratio));                 // (NaN too)
      if (s_rest != 0.f) keep = 1.f - r * (1.f + ratio);
    }
    P.loss[row] = any ? weight * loss : 0.f;
    *reinterpret_cast<float4*>(P.stats + row * 4) =
        any ? make_float4(m, log2f(s), keep, weight) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

// ---------------------------------------------------------------- backward
// A CTA takes P.seg groups of a row; each element is written by the thread that read it. OUT8: in 8-bit blocks.
template <int KIND, int VEC, bool OUT8>
__global__ void __launch_bounds__(kThreads, KIND == kF32 ? 2 : 3) distill_bwd_kernel(const __grid_constant__ DistillArgs P) {
  constexpr int kLoads = KIND == kF32 ? 4 : 8;
  extern __shared__ int smem[];
  const Lists L{smem, smem + P.seg, smem + P.seg + P.top};
  float* pl = reinterpret_cast<float*>(L.id + P.top);
  const int lane = int(lane_id()), warp = int(warp_id()), tid = int(threadIdx.x);
  const int segs = (P.groups + P.seg - 1) / P.seg;
  const int64_t row = blockIdx.x / segs;
  const int g0 = int(blockIdx.x - row * segs) * P.seg, g1 = min(P.groups, g0 + P.seg);
  grid_dependency_wait();
  grid_dependents_launch();
  const float4 st = __ldg(reinterpret_cast<const float4*>(P.stats + row * 4));
  const float g = __ldg(P.dloss + row) * st.w / P.temperature;
  const bool zero = g == 0.f;
  for (int i = tid; i < g1 - g0; i += kThreads) L.head[i] = -1;
  __syncthreads();
  for (int i = tid; i < P.top && !zero; i += kThreads) {
    const int64_t at = row * P.top + i;
    const int id = id_at(P, at);
    const float p = __ldg(P.probs + at);
    if (id >= 0 && !(p < 0.f) && id / kGroupElems >= g0 && id / kGroupElems < g1) {
      L.id[i] = id;
      pl[i] = p;
      L.next[i] = atomicExch(&L.head[id / kGroupElems - g0], i);
    }
  }
  __syncthreads();
  // q = 2^((x - m) c - log2 sum): the difference first, which is exact where q is large
  const float c = kLog2e / P.temperature, m = st.x, log_s = -st.y, gr = g * st.z;
  const int64_t base = row * P.V, ld = code_ld(P.V);
  const int cblocks = (P.V + kBlock - 1) / kBlock;
  for (int gb = g0 + warp; gb < g1; gb += kWarps * kLoads) {
    Held<KIND, VEC> held[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const int gi = gb + kWarps * k;
      if (gi < g1 && !zero) held[k].load(P.z, base + int64_t(gi) * kGroupElems, P.V - gi * kGroupElems, lane);
    }
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const int gi = gb + kWarps * k, n = P.V - gi * kGroupElems;
      if (gi >= g1) break;
      float v[8];
      if (zero) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
      } else {
        float x[8];
        held[k].get(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = ex2(fmaf(x[e] - m, c, log_s));
          v[e] = x[e] * gr;
        }
        for (int i = L.head[gi - g0]; i >= 0; i = L.next[i]) {
          const int o = L.id[i] - gi * kGroupElems, e0 = Held<KIND, VEC>::elem_of(o);
          if (Held<KIND, VEC>::lane_of(o) == lane) {
            const float pg = pl[i] * g;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (e == e0) v[e] = fmaf(x[e], g, -pg);
          }
        }
      }
      if constexpr (!OUT8) {
        Held<KIND, VEC>::store(P.dz, base + int64_t(gi) * kGroupElems, n, lane, v);
      } else {
        // the two blocks of the group: of 8 consecutive elements a lane, 16 lanes each; else the first and last four
        // of every lane. (What lies past column V is no value: 0, and written up to the codes' row length.)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (Held<KIND, VEC>::at(e, lane) >= n) v[e] = 0.f;
        uint32_t a[2] = {0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e) a[VEC == 8 ? 0 : e / 4] = max(a[VEC == 8 ? 0 : e / 4], abs_bits(v[e]));
        if constexpr (VEC == 8) {
#pragma unroll
          for (int o = 8; o; o >>= 1) a[0] = max(a[0], __shfl_xor_sync(0xffffffffu, a[0], o));
        } else {
          a[0] = __reduce_max_sync(0xffffffffu, a[0]);
          a[1] = __reduce_max_sync(0xffffffffu, a[1]);
        }
        uint8_t* out = static_cast<uint8_t*>(P.dz) + row * ld + int64_t(gi) * kGroupElems;
        const int nld = int(ld) - gi * kGroupElems;
        float* sc = P.scales + row * cblocks + 2 * gi;
        if constexpr (VEC == 8) {
          const BlockScale s = block_scale(a[0]);
          if (8 * lane < nld) *reinterpret_cast<uint2*>(out + 8 * lane) = codes8(v, s.inv);
          if ((lane & 15) == 0 && 8 * lane < n) sc[lane >> 4] = s.scale;
        } else {
          const BlockScale s[2] = {block_scale(a[0]), block_scale(a[1])};
#pragma unroll
          for (int h = 0; h < 8; h += VEC) {
            const int at = Held<KIND, VEC>::at(h, lane);
            const float inv = s[h / 4].inv;
            if (at >= nld) continue;
            if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(out + at) = codes4(v[h], v[h + 1], v[h + 2], v[h + 3], inv);
            else if constexpr (VEC == 2) *reinterpret_cast<uint16_t*>(out + at) = uint16_t(codes2(v[h], v[h + 1], inv));
            else out[at] = uint8_t(codes2(v[h], 0.f, inv));
          }
          if (lane < 2 && 128 * lane < n) sc[lane] = lane == 0 ? s[0].scale : s[1].scale;
        }
      }
    }
  }
}

bool args_ok(int type, int id_bytes, float temperature, int64_t M, int64_t V, int64_t top) {
  return type_ok(type) && (id_bytes == 4 || id_bytes == 8) && temperature > 0.f && temperature < kInf && M >= 0 &&
         M < (int64_t(1) << 28) && V >= 1 && V < (int64_t(1) << 22) && top >= 1 && top <= kMaxTop;
}

// Shared memory of a vocabulary's and a row's lists may pass the 48 KB that a launch has without asking.
constexpr size_t kMostSmem = (16384 + 4 * kMaxTop) * 4;

template <int KIND, int VEC>
cudaError_t launch_fwd(DistillArgs& P, int cl, cudaStream_t st) {
  const size_t smem = size_t(P.groups + 4 * P.top) * 4;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(P.M * cl));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {unsigned(cl), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = cl > 1 ? 2 : 1;
  if (cl == 8) return cudaLaunchKernelEx(&cfg, distill_fwd_kernel<KIND, VEC, 8>, P);
  if (cl == 2) return cudaLaunchKernelEx(&cfg, distill_fwd_kernel<KIND, VEC, 2>, P);
  return cudaLaunchKernelEx(&cfg, distill_fwd_kernel<KIND, VEC, 1>, P);
}
template <int KIND, int VEC>
cudaError_t launch_bwd(DistillArgs& P, bool out8, cudaStream_t st) {
  const size_t smem = size_t(P.seg + 3 * P.top) * 4;
  const dim3 grid(unsigned(P.M * cdiv(P.groups, P.seg)));
  return out8 ? launch_pdl(distill_bwd_kernel<KIND, VEC, true>, grid, dim3(kThreads), smem, st, P)
              : launch_pdl(distill_bwd_kernel<KIND, VEC, false>, grid, dim3(kThreads), smem, st, P);
}
template <int KIND, int VEC>
cudaError_t prepare() {
  cudaError_t e = cudaSuccess;
  auto set = [&](auto kernel) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMostSmem));
  };
  set(distill_fwd_kernel<KIND, VEC, 1>);
  set(distill_fwd_kernel<KIND, VEC, 2>);
  set(distill_fwd_kernel<KIND, VEC, 8>);
  set(distill_bwd_kernel<KIND, VEC, false>);
  set(distill_bwd_kernel<KIND, VEC, true>);
  return e;
}

// By the widest vector that fits every row.
template <class F>
cudaError_t by_vector(int type, int64_t V, F&& f) {
  using std::integral_constant;
  if (type == LORA_F32)
    return V % 4 == 0 ? f(integral_constant<int, kF32>{}, integral_constant<int, 4>{})
                      : f(integral_constant<int, kF32>{}, integral_constant<int, 1>{});
  return V % 8 == 0   ? f(integral_constant<int, kBf16>{}, integral_constant<int, 8>{})
         : V % 2 == 0 ? f(integral_constant<int, kBf16>{}, integral_constant<int, 2>{})
                      : f(integral_constant<int, kBf16>{}, integral_constant<int, 1>{});
}

}  // namespace

cudaError_t prepare_distill() {
  cudaError_t e;
  if ((e = prepare<kBf16, 8>()) != cudaSuccess || (e = prepare<kBf16, 2>()) != cudaSuccess ||
      (e = prepare<kBf16, 1>()) != cudaSuccess || (e = prepare<kF32, 4>()) != cudaSuccess)
    return e;
  return prepare<kF32, 1>();
}

}  // namespace mlp

using namespace mlp;

extern "C" {

lora_status lora_distill_topk_fwd(const void* logits, int type, const void* ids, int id_bytes, const void* teacher,
                                  int teacher_type, const float* teacher_lse, const float* weight, float temperature,
                                  int64_t M, int64_t V, int64_t top, float* loss, float* probs, float* stats,
                                  void* stream) {
  if (!args_ok(type, id_bytes, temperature, M, V, top) || !type_ok(teacher_type)) return LORA_ERR_SHAPE;
  if (M == 0) return LORA_OK;
  lora_status s = check_ptrs(logits, ids, teacher, static_cast<const void*>(loss), static_cast<const void*>(probs),
                             static_cast<const void*>(stats));
  if (s == LORA_OK && teacher_lse) s = check_ptrs(teacher_lse);
  if (s == LORA_OK && weight) s = check_ptrs(weight);
  if (s != LORA_OK) return s;
  int nsm = 0;
  if ((s = device_ready(&nsm)) != LORA_OK) return s;
  DistillArgs P{};
  P.z = logits;
  P.ids = ids;
  P.id8 = id_bytes == 8;
  P.teacher = teacher;
  P.teacher_type = teacher_type;
  P.teacher_lse = teacher_lse;
  P.weight = weight;
  P.temperature = temperature;
  P.M = M;
  P.V = int(V);
  P.top = int(top);
  P.groups = int(cdiv(V, kGroupElems));
  P.loss = loss;
  P.probs = probs;
  P.stats = stats;
  // few rows: a row's groups over the CTAs of a cluster, while each of their warps has one
  const int cl = M * 4 <= nsm && P.groups >= 4 * kWarps ? 8 : (M <= 2 * nsm && P.groups >= 2 * kWarps ? 2 : 1);
  const cudaError_t e = by_vector(type, V, [&](auto kind, auto vec) {
    return launch_fwd<kind.value, vec.value>(P, cl, static_cast<cudaStream_t>(stream));
  });
  return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

lora_status lora_distill_topk_bwd(const float* dloss, const void* logits, int type, const void* ids, int id_bytes,
                                  const float* probs, const float* stats, float temperature, int64_t M, int64_t V,
                                  int64_t top, void* dlogits, float* scales, void* stream) {
  if (!args_ok(type, id_bytes, temperature, M, V, top)) return LORA_ERR_SHAPE;
  if (M == 0) return LORA_OK;
  lora_status s = check_ptrs(static_cast<const void*>(dloss), logits, ids, static_cast<const void*>(probs),
                             static_cast<const void*>(stats), static_cast<const void*>(dlogits));
  if (s == LORA_OK && scales) s = check_ptrs(scales);
  if (s != LORA_OK) return s;
  DistillArgs P{};
  P.z = logits;
  P.ids = ids;
  P.id8 = id_bytes == 8;
  P.dloss = dloss;
  P.temperature = temperature;
  P.M = M;
  P.V = int(V);
  P.top = int(top);
  P.groups = int(cdiv(V, kGroupElems));
  P.probs = const_cast<float*>(probs);
  P.stats = const_cast<float*>(stats);
  P.dz = dlogits;
  P.scales = scales;
  P.seg = 64;
  if (M * cdiv(P.groups, P.seg) >= (int64_t(1) << 31)) return LORA_ERR_SHAPE;
  int nsm = 0;
  if ((s = device_ready(&nsm)) != LORA_OK) return s;
  const cudaError_t e = by_vector(type, V, [&](auto kind, auto vec) {
    return launch_bwd<kind.value, vec.value>(P, scales != nullptr, static_cast<cudaStream_t>(stream));
  });
  return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

}  // extern "C"
