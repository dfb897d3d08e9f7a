// distill.cu -- the loss against a teacher's top logits, forward and backward (lora_distill_topk_* of
// include/lora_base8.h).
//
// A row of logits is read once a pass. The forward pass holds a running maximum and the sum of exponentials
// relative to it, of everything that is no entry of the teacher's; the row's few entries are read on their own, and
// their part joined at the end. So the mass of the rest is a sum, and no difference. Long rows are
// bound by HBM (4096 x 131072 bf16 170 us forward, 5.9 TB/s; 303 backward, 6.9), short ones by the warp of a row's entries.
//
// A row is cut into groups of 256 elements, dealt in turn to the places of eight warps (1, 2 or 4 each, by the row's length
// alone); each thread of a place holds a maximum and a sum of its own, and the places' are joined in a fixed order. A batch of
// few rows has its rows' places spread over the CTAs of a cluster: the places, and so the bits, stay the same.
#include "../csrc/common.cuh"
#include "../csrc/kernels.h"
#include "../csrc_mlp/elems.cuh"
#include "base8.h"
#include "block8.cuh"
#include "distill.h"

#include <algorithm>
#include <cfloat>
#include <type_traits>

namespace mlp {
namespace {

using namespace lora;

constexpr int kThreads = 256, kWarps = 8, kGroupElems = 256, kPlaces = 4;
constexpr int kMaxTop = 1024;
constexpr float kLog2e = 1.4426950408889634f, kInf = __builtin_huge_valf();

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 8 bf16 elements from element `first` on (in pairs) of the 16 in u.
__device__ __forceinline__ void shifted(uint32_t (&u)[8], int first, uint32_t (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 6; ++i) u[i] = first & 4 ? u[i + 2] : u[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) u[i] = first & 2 ? u[i + 1] : u[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(u[i], u[i + 1], first & 1 ? 16 : 0);
}

// What a thread holds of a group of 256 elements of its warp: 8 of them, in pieces of VEC consecutive ones, 32 VEC apart:
// one of 8 (bf16), two of 4 (fp32), or (fp32 rows of odd lengths) single ones. SHIFT: bf16 rows whose length is no multiple of
// 8 start at any element; their pieces are put together from the two 16-byte vectors that hold them (loads of 2 bytes took
// 4096 x 50257 forward 201 us where this took 166; by pairs, from words, 232; 115 since, in sets of four).
template <int KIND, int VEC, bool SHIFT>
struct Held {
  static_assert(KIND == kF32 ? !SHIFT : VEC == 8, "");
  static constexpr int kWords = KIND == kF32 ? 8 : 4;
  uint32_t w[SHIFT ? 8 : kWords];                  // SHIFT: the two vectors, until settle()
  static __device__ __forceinline__ int at(int e, int lane) { return (e / VEC) * 32 * VEC + lane * VEC + e % VEC; }
  // The lane's first byte of a group that starts at element `base` (SHIFT: of the vector that holds it).
  static __device__ __forceinline__ const uint8_t* place(const void* p, int64_t base, int off, int lane) {
    constexpr int kBytes = KIND == kF32 ? 4 : 2;
    return static_cast<const uint8_t*>(p) + (base - off + lane * VEC) * kBytes;
  }
  // Elements of the group whose lane's place is `at`, of which n exist (the others stay what they were). off: the row's first
  // element % 8. edge: nothing need lie behind the row's end.
  __device__ __forceinline__ void load_whole(const uint8_t* at, int off) {
    if constexpr (KIND == kBf16) {
      uint4 t = *reinterpret_cast<const uint4*>(at);
      w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
      if constexpr (SHIFT) {
        if (off) {
          t = *reinterpret_cast<const uint4*>(at + 16);
          w[4] = t.x; w[5] = t.y; w[6] = t.z; w[7] = t.w;
        }
      }
    } else if constexpr (VEC == 4) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 t = *reinterpret_cast<const float4*>(at + 512 * j);
        w[4 * j] = __float_as_uint(t.x); w[4 * j + 1] = __float_as_uint(t.y);
        w[4 * j + 2] = __float_as_uint(t.z); w[4 * j + 3] = __float_as_uint(t.w);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = *reinterpret_cast<const uint32_t*>(at + 128 * j);
    }
  }
  __device__ __forceinline__ void load(const uint8_t* at, int off, int n, bool edge, int lane) {
    if constexpr (KIND == kBf16 && !SHIFT) {
      if (8 * lane < n) {
        const uint4 t = *reinterpret_cast<const uint4*>(at);
        w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
      }
    } else if constexpr (KIND == kBf16) {
      // elements of the row from the first and from the second vector's start on
      const int n0 = n + off - 8 * lane, n1 = n0 - 8;
      if (edge) {
        if (n0 > off) some(at, n0, w);
        if (off && n1 > 0) some(at + 16, n1, w + 4);
        return;
      }
      if (n0 > off) {
        const uint4 t = *reinterpret_cast<const uint4*>(at);
        w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
      }
      if (off && n1 > 0) {
        const uint4 t = *reinterpret_cast<const uint4*>(at + 16);
        w[4] = t.x; w[5] = t.y; w[6] = t.z; w[7] = t.w;
      }
    } else if constexpr (VEC == 4) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (128 * j + 4 * lane < n) {
          const float4 t = *reinterpret_cast<const float4*>(at + 512 * j);
          w[4 * j] = __float_as_uint(t.x); w[4 * j + 1] = __float_as_uint(t.y);
          w[4 * j + 2] = __float_as_uint(t.z); w[4 * j + 3] = __float_as_uint(t.w);
        }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (32 * j + lane < n) w[j] = *reinterpret_cast<const uint32_t*>(at + 128 * j);
    }
  }
  // The first n elements of a vector that need not lie in the tensor whole.
  static __device__ __forceinline__ void some(const uint8_t* at, int n, uint32_t* w) {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(at);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (2 * i < n ? uint32_t(q[2 * i]) : 0u) | (2 * i + 1 < n ? uint32_t(q[2 * i + 1]) << 16 : 0u);
  }
  // Makes the elements themselves of what load() brought.
  __device__ __forceinline__ void settle(int off) {
    if constexpr (SHIFT) {
      uint32_t t[4];
      shifted(w, off, t);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = t[i];
    }
  }
  // -infinity where the row has no more elements.
  __device__ __forceinline__ void end(int n, int lane) {
    if constexpr (KIND == kF32) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at(e, lane) >= n) w[e] = 0xFF800000u;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (at(2 * i, lane) >= n) w[i] = 0xFF80FF80u;
        else if (at(2 * i + 1, lane) >= n) w[i] = (w[i] & 0xFFFFu) | 0xFF800000u;
      }
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
  // The group's element o (0 to 255) becomes -infinity, where the lane has it.
  __device__ __forceinline__ void drop(uint32_t o, uint32_t lane) {
    if constexpr (KIND == kF32) {
      const uint32_t e = (o / VEC % 32 == lane) ? o / (32 * VEC) * VEC + o % VEC : 8u;
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = e == uint32_t(i) ? 0xFF800000u : w[i];
    } else {
      const uint32_t half = o / 8 == lane ? (o & 1 ? 0xFFFF0000u : 0xFFFFu) : 0u, word = o / 2 % 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t hit = word == uint32_t(i) ? half : 0u;
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
    static_assert(!SHIFT && VEC > 1, "");
    if constexpr (KIND == kBf16) {
      if (8 * lane < n) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + base + 8 * lane) = pack_bf16x8(v);
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (128 * j + 4 * lane < n)
          *reinterpret_cast<float4*>(static_cast<float*>(p) + base + 128 * j + 4 * lane) =
              make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
  }
  // load() and store() of a row that starts `lead` elements behind a 16-byte boundary, and whose groups are cut from there: `from`
  // is the row's element (its group's first ones may lie before it) that the group starts at, `row` the row's first.
  __device__ __forceinline__ void load_led(const void* p, int64_t row, int from, int V, bool edge, int lane) {
    static_assert(!SHIFT && VEC > 1, "");
#pragma unroll
    for (int j = 0; j < 8 / VEC; ++j) {
      const int i = from + at(VEC * j, lane);
      uint32_t* to = w + 4 * j;
      if (i >= V) continue;
      if (i + VEC <= V || !edge) {
        const uint4 t = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + (row + i) * (16 / VEC));
        to[0] = t.x; to[1] = t.y; to[2] = t.z; to[3] = t.w;
      } else if constexpr (KIND == kBf16) {
        some(static_cast<const uint8_t*>(p) + (row + i) * 2, V - i, to);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) to[e] = i + e < V ? static_cast<const uint32_t*>(p)[row + i + e] : 0u;
      }
    }
  }
  static __device__ __forceinline__ void store_led(void* p, int64_t row, int from, int V, int lane, const float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8 / VEC; ++j) {
      const int i = from + at(VEC * j, lane);
      if (i >= V) continue;
      if (i >= 0 && i + VEC <= V) {
        if constexpr (KIND == kBf16) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + row + i) = pack_bf16x8(v);
        else *reinterpret_cast<float4*>(static_cast<float*>(p) + row + i) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (i + e >= 0 && i + e < V) {
            if constexpr (KIND == kBf16) static_cast<__nv_bfloat16*>(p)[row + i + e] = __float2bfloat16_rn(v[e]);
            else static_cast<float*>(p)[row + i + e] = v[4 * j + e];
          }
      }
    }
  }
  // Which of the lane's elements is the group's element o; 8: none.
  static __device__ __forceinline__ uint32_t elem_of(uint32_t o, uint32_t lane) {
    return o / VEC % 32 == lane ? o / (32 * VEC) * VEC + o % VEC : 8u;
  }
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

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

struct DistillArgs {
  const void *z, *ids, *teacher;
  const float *teacher_lse, *weight, *dloss;
  int id8, teacher_type;           // ids in 64 bits; the teacher's type
  int64_t M;
  int V, top, groups, places;      // groups of 256 elements of a row; forward: places of a warp
  float temperature;
  float inv_t, inv_t_lo, c;        // forward: 1 / temperature as the sum of two; log2(e) / temperature
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

// Whether a vector that holds elements of the row may reach past the tensor's end.
__device__ __forceinline__ bool at_edge(const DistillArgs& P, int64_t row) { return (P.M - 1 - row) * P.V < 8; }

// The entries of a row by group: head[g] the first of group g, link[i] the one after entry i, -1 at the end, and its id (-1 where
// it is none). The order within a group is no fixed one; nothing depends on it.
struct Lists {
  int* head;                       // shared memory: groups
  int2* link;                      // top of (the next one, id)
};

__host__ __device__ constexpr int even(int n) { return (n + 1) & ~1; }

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

// CTAs of an SM: bf16 3, 4 and 5 194, 177 and 289 us at 4096 x 131072 (five spill), fp32 2, 3 and 4 172, 167 and 176 at 2048 x
// 131072.
template <int KIND>
constexpr int kMinCtas = KIND == kF32 ? 3 : 4;

// ----------------------------------------------------------------- forward
// A CTA has eight warps that stream its rows, and a ninth for their entries: it makes the lists of the next row and ends the one
// before while the others stream. (With all warps at a row's entries first and one at its end, a row of 4096 x 131072 took
// 5 us beside its 18 of streaming.) The loads run on from row to row.
constexpr int kFwdThreads = kThreads + 32;
constexpr uint32_t kBarLists = 1, kBarParts = 3;   // named barriers, two of each: rows in turn

__device__ __forceinline__ void bar_arrive(uint32_t id) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(kFwdThreads) : "memory"); }

// What the ninth warp makes of a row's entries.
struct Row {
  Lists lists;
  float *t, *z;                    // the entries' teacher logits, -infinity where dropped; and student logits
};

// A number as the sum of two floats, of which the second has what the first has not.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
// v / T so (1 / T given so); a mask's lowest value may pass the range, and has no rest.
__device__ __forceinline__ Two over_t(float v, Two inv_t) {
  const float h = v * inv_t.hi;
  return {h, fabsf(h) < kInf ? fmaf(v, inv_t.hi, -h) + v * inv_t.lo : 0.f};
}
__device__ const float2 kRoots[32] = {             // 2^(j / 32)
    {0x1p+0f, 0.f}, {0x1.059b0ep+0f, -0x1.9d4f52p-25f}, {0x1.0b5586p+0f, 0x1.9f3122p-25f}, {0x1.11301ep+0f, -0x1.fdb496p-25f},
    {0x1.172b84p+0f, -0x1.c15742p-27f}, {0x1.1d4874p+0f, -0x1.d2e8cap-25f}, {0x1.2387a6p+0f, 0x1.ceac48p-25f}, {0x1.29e9ep+0f, -0x1.5c0424p-25f},
    {0x1.306fep+0f, 0x1.4636e2p-25f}, {0x1.371a74p+0f, -0x1.18aac6p-25f}, {0x1.3dea64p+0f, 0x1.824684p-25f}, {0x1.44e086p+0f, 0x1.8624b4p-30f},
    {0x1.4bfdaep+0f, -0x1.593abcp-25f}, {0x1.5342b6p+0f, -0x1.2c561p-25f}, {0x1.5ab07ep+0f, -0x1.5bd5ecp-27f}, {0x1.6247ecp+0f, -0x1.f8b55p-25f},
    {0x1.6a09e6p+0f, 0x1.9fcef4p-26f}, {0x1.71f75ep+0f, 0x1.1d8beep-25f}, {0x1.7a1148p+0f, -0x1.829fdp-25f}, {0x1.82589ap+0f, -0x1.accc7cp-26f},
    {0x1.8ace54p+0f, 0x1.15506ep-27f}, {0x1.93737cp+0f, -0x1.e64744p-25f}, {0x1.9c4918p+0f, 0x1.51f848p-27f}, {0x1.a5503cp+0f, -0x1.b83b54p-25f},
    {0x1.ae89fap+0f, -0x1.a94b14p-26f}, {0x1.b7f77p+0f, -0x1.a09438p-25f}, {0x1.c199bep+0f, -0x1.3d56b2p-27f}, {0x1.cb720ep+0f, -0x1.8837ccp-27f},
    {0x1.d5818ep+0f, -0x1.822dbcp-27f}, {0x1.dfc974p+0f, -0x1.908c94p-25f}, {0x1.ea4afap+0f, 0x1.52486cp-27f}, {0x1.f50766p+0f, -0x1.246ebp-26f}};
// p = e^(t / T - lse) in units of 2^-50, right to 2^-44 of 1 (a p of e^-64 or less is 0, of more than e is e). By a table and the series of
// e^g (P. T. P. Tang, 1989): t / T - lse = j log 2 / 32 + g, with log 2 / 32 in three parts, j times the first of which is exact.
__device__ __forceinline__ int64_t whole_p(float t, float lse, Two inv_t, const float2* roots) {
  const Two v = over_t(t, inv_t);
  const bool some = v.hi > lse - 64.f;
  Two a = two_sum(some ? fminf(v.hi, lse + 1.f) : lse - 64.f, -lse);
  a.lo += some ? v.lo : 0.f;
  const float j = rintf(a.hi * 46.166241f), h = j * 0x1.0bfbe8p-20f;
  const int k = int(j);
  const float2 root = roots[k & 31];
  const Two f = two_sum(fmaf(-j, 0x1.62ep-6f, a.hi), -h);
  const float g = f.hi, gl = f.lo + fmaf(-j, 0x1.cf79acp-45f, a.lo - fmaf(j, 0x1.0bfbe8p-20f, -h));
  const float q = g * g, ql = fmaf(g, g, -q), u = fmaf(0.5f, q, g), ul = fmaf(0.5f, q, g - u);
  const float c = q * g * fmaf(g, fmaf(g, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f);
  const float w = ul + fmaf(0.5f, ql, gl + fmaf(u, gl, c));                             // e^g - 1 = u + w
  const float x = root.x * u, xl = fmaf(root.x, u, -x), p = __fadd_rn(root.x, x);
  const float pl = (x - (p - root.x)) + (xl + fmaf(root.y, u, fmaf(root.x, w, root.y)));
  const float scale = __uint_as_float(uint32_t(127 + 50 + (k >> 5)) << 23);
  return __float2ll_rn(p * scale) + __float2int_rn(pl * scale);
}

// The lists, of all lanes. Logits only where they are wanted (the cluster's first CTA).
__device__ __forceinline__ void make_lists(const DistillArgs& P, const Row& r, int kind, int64_t row, bool logits, int lane) {
  const Lists& L = r.lists;
  for (int g = lane; g < P.groups; g += 32) L.head[g] = -1;
  __syncwarp();
  // Entries of a lane whose loads are on their way together: this warp's time a row bounds rows of few logits (4096 x 32000 with 256
  // entries, one, two and four: 166, 142 and 133 us; with 16 entries 56.3, 56.3 and 58.2).
  constexpr int kMany = 2;
  for (int i0 = lane; i0 < P.top; i0 += 32 * kMany) {
    int id[kMany];
    float t[kMany], z[kMany];
#pragma unroll
    for (int k = 0; k < kMany; ++k) {
      const int64_t at = row * P.top + min(i0 + 32 * k, P.top - 1);
      id[k] = id_at(P, at);
      t[k] = param_at(P.teacher, P.teacher_type, at);
    }
#pragma unroll
    for (int k = 0; k < kMany; ++k) {
      if (t[k] == -kInf) id[k] = -1;
      z[k] = id[k] >= 0 && logits ? param_at(P.z, kind, row * P.V + id[k]) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kMany; ++k) {
      const int i = i0 + 32 * k;
      if (i >= P.top) break;
      r.t[i] = id[k] < 0 ? -kInf : t[k];
      L.link[i] = make_int2(id[k] < 0 ? -1 : atomicExch(&L.head[id[k] / kGroupElems], i), id[k]);
      r.z[i] = z[k];
    }
  }
  __syncwarp();
  // of several entries of one id the first counts
  for (int i = lane; i < P.top; i += 32) {
    const int id = L.link[i].y;
    if (id < 0) continue;
    for (int j = L.head[id / kGroupElems]; j >= 0; j = L.link[j].x)
      if (j < i && L.link[j].y == id) {
        r.t[i] = -kInf;
        break;
      }
  }
  __syncwarp();
}

// 1 - sum p of a row's entries, of the whole warp, where the floats' sum of p is near 1: the listed logits may have all the teacher's
// mass but 10^-6, of which p and sums in floats leave nothing. The sum is one of whole numbers, and so exact. (Of a teacher of
// 64 entries that has only such rows, 8192 x 2000 89 -> 98 us, 4096 x 32000 63 -> 69, x 131072 177 -> 177. In doubles, of which GB300
// makes two operations an SM and cycle, 115, 77 and 182; in every row, while the student's logits are on their way, 107, 72 and 181.)
__device__ __forceinline__ float rest_of_teacher(const DistillArgs& P, const float* t, float lse, const float2* roots, int lane) {
  int64_t sum = 0;
#pragma unroll 1
  for (int i = lane; i < P.top; i += 32) sum += whole_p(t[i], lse, {P.inv_t, P.inv_t_lo}, roots);    // (-infinity: no entry)
  constexpr int kHalf = 25;
  const uint32_t high = __reduce_add_sync(0xffffffffu, uint32_t(sum >> kHalf));
  const uint32_t low = __reduce_add_sync(0xffffffffu, uint32_t(sum) & ((1u << kHalf) - 1));
  const int64_t left = (int64_t(1) << 50) - ((int64_t(high) << kHalf) + low);
  return fmaf(float(int(left >> 24)), 0x1p-26f, float(int(left & 0xFFFFFF)) * 0x1p-50f);
}

// The end of a row with teacher_lse whose pieces are far apart, or whose listed entries have all the teacher's mass or nearly.
//
// A rest below 2^-32 of the row's sum may lose itself beside the entries': log rho is taken from the rest's own maximum. And what the
// backward pass takes, 1 - r / rho, from r / rho = 2^32 on (the 1 is no part of that) is held by its logarithm, as -2^32 log2: r rho_j of
// an element is then one exponential of log2(r / rho) and the element's exponent, where q_j alone may be too small for a float.
// Of a logarithm of 2^12 a float's rounding is 1e-4 of the gradient: below that rho counts as 0 there. (Halves: the
// difference of two of the type's values may pass its largest.)
//
// A teacher that lists all its mass leaves 0 only up to the roundings of its log-sum-exp, in half ulps of 1: up to 64 of a sum of
// exponentials, and |lse| for each rounding on the way, of t / T, of the largest, of the result. Where rho counts as 0 so much is no
// mass: its logarithm would be all of the loss (1e-7 of a mask's lowest value). (1/2 at most: lse may be infinite.)
constexpr float kSmall = 0.0625f, kFarRest = 0x1p-32f, kFarOver = 0x1p32f, kFarKeep = -0x1p37f, kFarMost = 4096.f;
__device__ __forceinline__ void end_rare(const DistillArgs& P, const float* t, Part rest, float m, float s, float s_rest, float s_top,
                                         float sum_p, float loss, float lse, const float2* roots, int64_t row, float weight, int lane) {
  const float c = P.c;
  float left = 1.f - sum_p, log_left = 0.f, log2_p = 0.f, keep = 1.f;
  if (left > -1.f && left < kSmall) left = rest_of_teacher(P, t, lse, roots, lane);
  if (lane != 0) return;
  if (left > 0.f) {
    log_left = left < kSmall ? logf(left) : log1pf(-sum_p);
  } else {                                         // the gradient is sum_p q - p
    log2_p = left > -1.f ? kLog2e * log1pf(-left) : log2f(sum_p);
    left = 0.f;
  }
  if (s_rest < s * kFarRest) {
    const float fall = 0.5f * rest.m - 0.5f * m;
    const float log2_rho = rest.s == 0.f ? -kInf : 2.f * (fall * c) + (log2f(rest.s) - log2f(s));
    const bool none = log2_rho < -kFarMost;
    if (none && left <= fminf(0.5f, fmaf(8.f, fabsf(lse), 64.f) * 0x1p-24f)) left = 0.f;
    if (left != 0.f) {
      const float over = log2f(left) - log2_rho;                                         // log2(r / rho)
      loss += rest.s == 0.f ? kInf : left * (log_left - (2.f * (fall * P.inv_t) + (logf(rest.s) - logf(s))));
      keep = none ? 1.f : (over < 32.f ? 1.f - exp2f(over) : -kFarOver * over);
    }
  } else if (left != 0.f) {
    const float ratio = s_top / s_rest;            // log rho = -log(1 + ratio)
    loss += left * (log_left + log1pf(ratio));
    if (s_rest != 0.f) keep = 1.f - left * (1.f + ratio);
  }
  P.loss[row] = weight * loss;
  *reinterpret_cast<float4*>(P.stats + row * 4) = make_float4(m, log2f(s) - log2_p, keep, weight);
}

// The row's end, from the eight warps' parts: of one warp.
__device__ __forceinline__ void end_row(const DistillArgs& P, const Row& r, const Part* warps, const float2* roots, int64_t row, float weight,
                                        int lane) {
  const float c = P.c;
  // the rest of the vocabulary
  Part rest = warps[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) rest.m = fmaxf(rest.m, warps[w].m);
  rest.s = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) rest.s += rescale(warps[w].s, warps[w].m, rest.m, c);
  // the entries': maxima, then sums
  float zm = -kInf, tm = -kInf;
  bool any = false;
#pragma unroll 2
  for (int i = lane; i < P.top; i += 32)
    if (r.t[i] != -kInf) {
      any = true;
      zm = fmaxf(zm, r.z[i]);
      tm = fmaxf(tm, r.t[i]);
    }
  any = __any_sync(0xffffffffu, any);
  zm = warp_max(zm);
  tm = warp_max(tm);
  // (without the teacher's mass of the rest nobody asks for the student's: the stream then has the entries too)
  const float m = fmaxf(rest.m, zm);
  float s_top = 0.f, s_teacher = 0.f;
#pragma unroll 2
  for (int i = lane; i < P.top; i += 32)
    if (r.t[i] != -kInf) {
      s_top += ex2((r.z[i] - m) * c);
      s_teacher += ex2((r.t[i] - tm) * c);
    }
  s_top = warp_sum(s_top);
  s_teacher = warp_sum(s_teacher);
  const float s_rest = rescale(rest.s, rest.m, m, c), s = P.teacher_lse ? s_rest + s_top : s_rest;
  // log p - log q = (t - z) / T - (norm - log sum exp(z / T)): a difference of an entry's own two logits, and one of the
  // row's. The terms of a small divergence cancel, and so keep their digits: what a product or 1 / T leaves is carried along.
  const float inv_t = P.inv_t;
  const float log_s = logf(s), log_t = logf(s_teacher), lse = P.teacher_lse ? __ldg(P.teacher_lse + row) : 0.f;
  const Two m_t = over_t(m, {P.inv_t, P.inv_t_lo});
  const float gap = P.teacher_lse ? ((lse - m_t.hi) - m_t.lo) - log_s : fmaf(tm - m, inv_t, log_t - log_s);
  // Logits far from the teacher's (a row whose mask leaves only the type's lowest value) lose the digits of t in t - z:
  // there, log p and log q each from its own maximum.
  const bool near = fabsf(gap) < 64.f;
  float sum_p = 0.f, loss = 0.f;
#pragma unroll 2
  for (int i = lane; i < P.top; i += 32) {
    const float ti = r.t[i];
    float p = -1.f;
    if (ti != -kInf) {
      const Two v = over_t(ti, {P.inv_t, P.inv_t_lo});
      const float log_p = P.teacher_lse ? (v.hi - lse) + v.lo : (ti - tm) * inv_t - log_t;
      p = expf(log_p);
      sum_p += p;
      if (p != 0.f) loss += p * (near ? (ti - r.z[i]) * inv_t - gap : log_p - ((r.z[i] - m) * inv_t - log_s));
    }
    P.probs[row * P.top + i] = p;
  }
  sum_p = warp_sum(sum_p);
  loss = warp_sum(loss);
  if (__builtin_expect(P.teacher_lse && any && (1.f - sum_p < kSmall || s_rest < s * kFarRest), 0)) {
    end_rare(P, r.t, rest, m, s, s_rest, s_top, sum_p, loss, lse, roots, row, weight, lane);
  } else if (lane == 0) {
    float keep = 1.f;
    if (P.teacher_lse) {
      const float left = 1.f - sum_p, ratio = s_top / s_rest;                            // log rho = -log(1 + ratio)
      loss += left * (log1pf(-sum_p) + log1pf(ratio));
      if (s_rest != 0.f) keep = 1.f - left * (1.f + ratio);
    }
    P.loss[row] = any ? weight * loss : 0.f;
    *reinterpret_cast<float4*>(P.stats + row * 4) =
        any ? make_float4(m, log2f(s), keep, weight) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

// The sum of 2^((x - m) c) over a group, for maxima far from 0, where the products x c have no digits behind the point.
template <class H>
__device__ __noinline__ float far_sum(H v, float m, float c) {
  float x[8], sum = 0.f;
  v.get(x);
#pragma unroll
  for (int e = 0; e < 8; ++e) sum += ex2((x[e] - m) * c);
  return sum;
}

// Groups of a set. (SHIFT holds twice the words of a group: sets of eight, two CTAs an SM, took 4096 x 50257 154 us, sets of four 115.)
constexpr int set_of(int kind, bool shift) { return kind == kF32 || shift ? 4 : 8; }

// CL: CTAs of a row's cluster. Of a thread's places, CTA r has those congruent to r.
//
// A place's groups are taken in a set of eight (fp32: four) rounds at a time: one maximum, and at most one rescaling of the sum, for
// a thread's 64 (32) elements. (Group by group, a thread's instructions were more of the time than its loads.)
template <int KIND, int VEC, bool SHIFT, int CL>
__global__ void __launch_bounds__(kFwdThreads, kMinCtas<KIND>) distill_fwd_kernel(const __grid_constant__ DistillArgs P) {
  constexpr int kSet = set_of(KIND, SHIFT);
  using H = Held<KIND, VEC, SHIFT>;
  extern __shared__ int smem[];
  __shared__ Part sent[kPlaces][kThreads];         // the threads' places; in a cluster's first CTA all of them
  __shared__ Part parts[2][kWarps];
  __shared__ int64_t rows[2];                      // the rows in turn; -1: no more
  __shared__ float2 roots[32];                     // kRoots, for the ninth warp
  const int lane = int(lane_id()), warp = int(warp_id()), tid = int(threadIdx.x);
  const int rank = CL > 1 ? int(cluster_rank()) : 0;
  const auto entries = [&](int b) {
    int2* at = reinterpret_cast<int2*>(smem + b * (even(P.groups) + 4 * P.top));
    float* t = reinterpret_cast<float*>(at + P.top);
    return Row{{reinterpret_cast<int*>(t + 2 * P.top), at}, t, t + P.top};
  };
  grid_dependency_wait();
  grid_dependents_launch();
  if constexpr (CL > 1) cluster_sync_all();        // every CTA of the cluster runs: its shared memory may be written

  if (warp == kWarps) {
    // ---------------------------------------------------------- the entries
    if (P.teacher_lse) roots[lane] = kRoots[lane];
    __syncwarp();
    int64_t next = blockIdx.x / CL, was = -1;
    float weight = 0.f, w_next = P.weight ? __ldg(P.weight + next) : 1.f;
    const int64_t step = gridDim.x / CL;
    for (int b = 0;; b ^= 1) {
      // the next row that is read, its lists; what the ones passed over leave
      int64_t row = -1;
      float w = 0.f;
      for (; row < 0 && next < P.M; next += step) {
        w = w_next;
        if (P.weight && next + step < P.M) w_next = __ldg(P.weight + next + step);
        if (w != 0.f) {
          row = next;
        } else if (rank == 0) {
          for (int i = lane; i < P.top; i += 32) P.probs[next * P.top + i] = -1.f;
          if (lane < 4) P.stats[next * 4 + lane] = 0.f;
          if (lane == 0) P.loss[next] = 0.f;
        }
      }
      if (row >= 0) make_lists(P, entries(b), KIND, row, rank == 0, lane);
      if (lane == 0) rows[b] = row;
      __syncwarp();
      bar_arrive(kBarLists + b);
      if (was >= 0) {
        if constexpr (CL > 1) cluster_sync_all();  // (a cluster has one row)
        if (rank == 0) {
          named_bar(kBarParts + (b ^ 1), kFwdThreads);
          end_row(P, entries(b ^ 1), parts[b ^ 1], roots, was, weight, lane);
        }
      }
      if (row < 0) return;
      was = row;
      weight = w;
    }
  }

  // ---------------------------------------------------------------- the stream
  // A set of groups is sent for, taken in, and the next one sent for, of the next row when this one has no more: warps wait in
  // turn.
  const float c = P.c;
  constexpr int kBytes = KIND == kF32 ? 4 : 2;
  const int stride = P.places * kWarps, round = stride * kGroupElems;      // groups and elements of a round
  const int sets = (P.groups + stride * kSet - 1) / (stride * kSet);       // of a place
  const int places = P.places / CL;                // of this CTA
  const auto first_of = [&](int j) { return ((CL * j + rank) * kWarps + warp) * kGroupElems; };
  const auto offset = [&](int64_t row) { return SHIFT ? int(row * P.V & 7) : 0; };
  // what is sent for next: row `to`, its place and rounds; nothing when to is -1
  int64_t to = -1;
  int to_b = 1, to_j = places, to_q = 0, to_left = 0, to_off = 0;
  const uint8_t* to_at = nullptr;
  bool to_edge = false, more = true;
  const auto send = [&](H (&h)[kSet]) {
    if (to_j == places && more) {                  // the next row; its lists are there
      to_b ^= 1;
      named_bar(kBarLists + to_b, kFwdThreads);
      to = rows[to_b];
      more = to >= 0;
      to_j = 0;
      to_off = offset(to);
      to_edge = at_edge(P, to);
      to_left = P.V - first_of(0);
      to_at = H::place(P.z, to * P.V + first_of(0), to_off, lane);
    }
    if (!more) return;
    if (to_left >= (kSet - 1) * round + kGroupElems + 8) {     // (the second vector of an unaligned group's last lane, too)
#pragma unroll
      for (int i = 0; i < kSet; ++i) h[i].load_whole(to_at + int64_t(i * round) * kBytes, to_off);
    } else {
#pragma unroll
      for (int i = 0; i < kSet; ++i) h[i].load(to_at + int64_t(i * round) * kBytes, to_off, to_left - i * round, to_edge, lane);
    }
    if (++to_q < sets) {
      to_at += int64_t(kSet * round) * kBytes;
      to_left -= kSet * round;
    } else {
      to_q = 0;
      ++to_j;
      to_left = P.V - first_of(to_j);
      to_at = H::place(P.z, to * P.V + first_of(to_j), to_off, lane);
    }
  };
  H h[kSet];
  send(h);
  int64_t row = to;
  if (row < 0) return;
  // what is taken in next
  int b = 0, j = 0, q = 0, left = P.V - first_of(0), off = offset(row);
  Part p{-kInf, 0.f};
  // Takes a set in; true when that was the end of the row.
  const auto take = [&]() {
    if (left > 0) {
      const Lists L = entries(b).lists;
      const int* head = L.head + (P.V - left) / kGroupElems;
      // (half a set where the rest of it has no elements)
      const bool all = left > kSet / 2 * round;
#pragma unroll
      for (int i = 0; i < kSet; ++i) {
        if (i >= kSet / 2 && !all) break;
        h[i].settle(off);
      }
      if (left < (kSet - 1) * round + kGroupElems) {
#pragma unroll
        for (int i = 0; i < kSet; ++i)
          if (left - i * round < kGroupElems) h[i].end(left - i * round, lane);
      }
      if (P.teacher_lse) {                         // the entries are no part of the rest
#pragma unroll
        for (int i = 0; i < kSet; ++i) {
          if (left <= i * round) break;
          const int first = P.V - left + i * round;
          for (int e = head[i * stride]; e >= 0;) {
            const int2 link = L.link[e];
            h[i].drop(uint32_t(link.y - first), uint32_t(lane));
            e = link.x;
          }
        }
      }
      float m = h[0].largest();
#pragma unroll
      for (int i = 1; i < kSet; ++i) m = fmaxf(m, h[i].largest());           // (-infinity where there are none)
      if (m > p.m) {
        p.s = rescale(p.s, p.m, m, c);
        p.m = m;
      }
      // 2^((x - m) c) = 2^(x c - r) 2^(r - m c) with r = m c rounded to an integer: one fma an element
      const float ref = p.m == -kInf ? 0.f : p.m, mc = ref * c;            // (nothing but -infinity so far: all terms are 0)
      if (__any_sync(0xffffffffu, !(fabsf(mc) < 65536.f))) {
#pragma unroll
        for (int i = 0; i < kSet; ++i)
          if (left > i * round) p.s += far_sum(h[i], ref, c);
      } else {
        const float r = rintf(mc);
        float2 sum = make_float2(0.f, 0.f);
        const auto add = [&](int i) {
          float x[8];
          h[i].get(x);
          float2 y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[e] = fma2(make_float2(x[2 * e], x[2 * e + 1]), make_float2(c, c), make_float2(-r, -r));
            y[e] = make_float2(ex2(y[e].x), ex2(y[e].y));
          }
          sum = add2(sum, add2(add2(y[0], y[1]), add2(y[2], y[3])));
        };
#pragma unroll
        for (int i = 0; i < kSet / 2; ++i) add(i);
        if (all) {
#pragma unroll
          for (int i = kSet / 2; i < kSet; ++i) add(i);
        }
        p.s += (sum.x + sum.y) * ex2(fmaf(-ref, c, r));
      }
    }
    if (++q < sets) {
      left -= kSet * round;
      return false;
    }
    // the place is done
    if constexpr (CL > 1)
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(peer_addr(smem_u32(&sent[CL * j + rank][tid]), 0)), "f"(p.m), "f"(p.s) : "memory");
    else
      sent[j][tid] = p;
    p = {-kInf, 0.f};
    q = 0;
    ++j;
    left = P.V - first_of(j);
    if (j < places) return false;
    // and the row: the thread's places, in order; then the warp's lanes
    if constexpr (CL > 1) {
      cluster_sync_all();
      if (rank != 0) return true;
    }
    Part all[kPlaces];
#pragma unroll
    for (int i = 0; i < kPlaces; ++i) all[i] = i < P.places ? sent[i][tid] : Part{-kInf, 0.f};
    Part t = all[0];
#pragma unroll
    for (int i = 1; i < kPlaces; ++i) t.m = fmaxf(t.m, all[i].m);
    t.m = warp_max(t.m);
    t.s = 0.f;
#pragma unroll
    for (int i = 0; i < kPlaces; ++i) t.s += rescale(all[i].s, all[i].m, t.m, c);
    t.s = warp_sum(t.s);
    if (lane == 0) parts[b][warp] = t;
    __syncwarp();
    bar_arrive(kBarParts + b);
    return true;
  };
  while (true) {
    const bool ended = take();
    if (CL > 1 && ended) return;                   // (a cluster has one row)
    send(h);
    if (!ended) continue;
    row = to;
    if (row < 0) return;
    off = to_off;
    b ^= 1;
    j = 0;
    left = P.V - first_of(0);
  }
}

// ---------------------------------------------------------------- backward
// A CTA takes P.seg groups of a row; each element is written by the thread that read it. OUT8: in 8-bit blocks. Bound by HBM (in
// blocks, by the instructions of a group too). fp32, two CTAs an SM and three: 2048 x 131072 in blocks 341 and 221 us.
template <int KIND, int VEC, bool SHIFT, bool OUT8>
__global__ void __launch_bounds__(kThreads, KIND == kF32 ? 3 : (OUT8 ? 4 : 5)) distill_bwd_kernel(const __grid_constant__ DistillArgs P) {
  constexpr int kLoads = 4;                        // groups of a warp in flight
  // Rows that vectors do not fit, element by element: cut into groups from a 16-byte boundary on (4096 x 50257 bf16 226 -> 143 us,
  // 2048 x 50257 fp32 148 -> 131). The blocks of OUT8 start with their row.
  constexpr bool LED = !OUT8 && (SHIFT || VEC == 1);
  using H = Held<KIND, LED ? (KIND == kF32 ? 4 : 8) : VEC, SHIFT && !LED>;
  extern __shared__ int smem[];
  const Lists L{smem + 3 * P.top + (P.top & 1), reinterpret_cast<int2*>(smem)};
  float* pl = reinterpret_cast<float*>(smem + 2 * P.top);
  const int lane = int(lane_id()), warp = int(warp_id()), tid = int(threadIdx.x);
  const int segs = (P.groups + P.seg - 1) / P.seg;
  const int64_t row = blockIdx.x / segs;
  const int g0 = int(blockIdx.x - row * segs) * P.seg, g1 = min(P.groups, g0 + P.seg);
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t base = row * P.V, ld = code_ld(P.V);
  const int first = SHIFT && !LED ? int(base & 7) : 0, lead = LED ? int(base & (KIND == kF32 ? 3 : 7)) : 0;
  const bool edge = at_edge(P, row);
  const float4 st = __ldg(reinterpret_cast<const float4*>(P.stats + row * 4));
  const float g = __ldg(P.dloss + row) * st.w / P.temperature;
  const bool zero = g == 0.f || st.w == 0.f;       // (of weight 0 whatever dloss is)
  for (int i = tid; i < g1 - g0; i += kThreads) L.head[i] = -1;
  __syncthreads();
  for (int i = tid; i < P.top && !zero; i += kThreads) {
    const int64_t at = row * P.top + i;
    const int id = id_at(P, at);
    const float p = __ldg(P.probs + at);
    const int at_group = (id + lead) / kGroupElems;
    if (id >= 0 && !(p < 0.f) && at_group >= g0 && at_group < g1) {
      pl[i] = p;
      L.link[i] = make_int2(atomicExch(&L.head[at_group - g0], i), id);
    }
  }
  __syncthreads();
  // q = 2^((x - m) c - log2 sum): the difference first, which is exact where q is large
  const float c = kLog2e / P.temperature, m = st.x, log_s = -st.y, gr = g * st.z;
  // FAR: a row whose rest has the gradient -r rho_j, by way of log2(r / rho) (end_rare). A loop of its own: with a branch in this
  // one, 4096 x 50257 bf16 took 138 us instead of 127.
  const auto groups = [&](auto far) {
    constexpr bool FAR = far.value;
    const int cblocks = (P.V + kBlock - 1) / kBlock;
    for (int gb = g0 + warp; gb < g1; gb += kWarps * kLoads) {
      H held[kLoads];
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int gi = gb + kWarps * k;
        if (gi >= g1 || zero) continue;
        if constexpr (LED) held[k].load_led(P.z, base, gi * kGroupElems - lead, P.V, edge, lane);
        else held[k].load(H::place(P.z, base + int64_t(gi) * kGroupElems, first, lane), first, P.V - gi * kGroupElems, edge, lane);
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
          held[k].settle(first);
          held[k].get(x);                            // (what lies past the row's end is not stored)
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float2 y = fma2(add2(make_float2(x[e], x[e + 1]), make_float2(-m, -m)), make_float2(c, c), make_float2(log_s, log_s));
            x[e] = ex2(y.x);
            x[e + 1] = ex2(y.y);
            const float2 t = mul2(make_float2(x[e], x[e + 1]), make_float2(gr, gr));
            v[e] = t.x;
            v[e + 1] = t.y;
          }
          if constexpr (FAR) {
            const float lift = st.z * (-1.f / kFarOver);
            held[k].get(v);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = -g * ex2(fmaf(v[e] - m, c, log_s + lift));
          }
          for (int i = L.head[gi - g0]; i >= 0;) {
            const int2 link = L.link[i];
            const uint32_t mine = H::elem_of(uint32_t(link.y + lead - gi * kGroupElems), uint32_t(lane));
            const float pg = pl[i] * g;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = mine == uint32_t(e) ? fmaf(x[e], g, -pg) : v[e];
            i = link.x;
          }
        }
        if constexpr (LED) {
          H::store_led(P.dz, base, gi * kGroupElems - lead, P.V, lane, v);
        } else if constexpr (!OUT8) {
          H::store(P.dz, base + int64_t(gi) * kGroupElems, n, lane, v);
        } else {
          // the two blocks of the group: of 8 consecutive elements a lane, 16 lanes each; else the first and last four
          // of every lane. (What lies past column V is no value: 0, and written up to the codes' row length.)
          if (n < kGroupElems) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (H::at(e, lane) >= n) v[e] = 0.f;
          }
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
              const int at = H::at(h, lane);
              const float inv = s[h / 4].inv;
              if (at >= nld) continue;
              if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(out + at) = codes4(v[h], v[h + 1], v[h + 2], v[h + 3], inv);
              else out[at] = uint8_t(codes2(v[h], 0.f, inv));
            }
            if (lane < 2 && 128 * lane < n) sc[lane] = lane == 0 ? s[0].scale : s[1].scale;
          }
        }
      }
    }
  };
  if (st.z <= kFarKeep) groups(std::true_type{});
  else groups(std::false_type{});
}

bool args_ok(int type, int id_bytes, float temperature, int64_t M, int64_t V, int64_t top) {
  return type_ok(type) && (id_bytes == 4 || id_bytes == 8) && temperature >= FLT_MIN && temperature < kInf && M >= 0 &&
         M < (int64_t(1) << 28) && V >= 1 && V < (int64_t(1) << 22) && top >= 1 && top <= kMaxTop;
}

// Shared memory of a vocabulary's and a row's lists may pass the 48 KB that a launch has without asking.
constexpr size_t kMostSmem = 2 * (16384 + 4 * kMaxTop) * 4;

template <int KIND, int VEC, bool SHIFT>
cudaError_t launch_fwd(DistillArgs& P, int cl, int nsm, cudaStream_t st) {
  const size_t smem = size_t(cl > 1 ? 1 : 2) * (even(P.groups) + 4 * P.top) * 4;
  // as many CTAs as are resident (the lists of a long vocabulary leave room for fewer)
  const int64_t room = std::max<int64_t>(1, 227 * 1024 / int64_t(smem + sizeof(Part) * kPlaces * kThreads + 2048));
  const int64_t ctas = nsm * std::min<int64_t>(kMinCtas<KIND>, room);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(cl > 1 ? P.M * cl : std::min<int64_t>(P.M, ctas)));
  cfg.blockDim = dim3(kFwdThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {unsigned(cl), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = cl > 1 ? 2 : 1;
  if (cl == 4) return cudaLaunchKernelEx(&cfg, distill_fwd_kernel<KIND, VEC, SHIFT, 4>, P);
  if (cl == 2) return cudaLaunchKernelEx(&cfg, distill_fwd_kernel<KIND, VEC, SHIFT, 2>, P);
  return cudaLaunchKernelEx(&cfg, distill_fwd_kernel<KIND, VEC, SHIFT, 1>, P);
}
template <int KIND, int VEC, bool SHIFT>
cudaError_t launch_bwd(DistillArgs& P, bool out8, cudaStream_t st) {
  // (a row that starts behind a 16-byte boundary may reach one group further)
  if (!out8 && (SHIFT || VEC == 1)) P.groups = int(cdiv(P.V + (KIND == kF32 ? 3 : 7), kGroupElems));
  const size_t smem = size_t(P.seg + 3 * P.top + 1) * 4;
  const dim3 grid(unsigned(P.M * cdiv(P.groups, P.seg)));
  return out8 ? launch_pdl(distill_bwd_kernel<KIND, VEC, SHIFT, true>, grid, dim3(kThreads), smem, st, P)
              : launch_pdl(distill_bwd_kernel<KIND, VEC, SHIFT, false>, grid, dim3(kThreads), smem, st, P);
}
template <int KIND, int VEC, bool SHIFT>
cudaError_t prepare() {
  cudaError_t e = cudaSuccess;
  auto set = [&](auto kernel) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMostSmem));
  };
  set(distill_fwd_kernel<KIND, VEC, SHIFT, 1>);
  set(distill_fwd_kernel<KIND, VEC, SHIFT, 2>);
  set(distill_fwd_kernel<KIND, VEC, SHIFT, 4>);
  set(distill_bwd_kernel<KIND, VEC, SHIFT, false>);
  set(distill_bwd_kernel<KIND, VEC, SHIFT, true>);
  return e;
}

// By what the rows' length allows.
template <class F>
cudaError_t by_length(int type, int64_t V, F&& f) {
  using std::integral_constant;
  const auto as = [&](auto kind, auto vec, auto shift) { return f(kind, vec, shift); };
  if (type == LORA_F32)
    return V % 4 == 0 ? as(integral_constant<int, kF32>{}, integral_constant<int, 4>{}, std::false_type{})
                      : as(integral_constant<int, kF32>{}, integral_constant<int, 1>{}, std::false_type{});
  return V % 8 == 0 ? as(integral_constant<int, kBf16>{}, integral_constant<int, 8>{}, std::false_type{})
                    : as(integral_constant<int, kBf16>{}, integral_constant<int, 8>{}, std::true_type{});
}

}  // namespace

cudaError_t prepare_distill() {
  cudaError_t e;
  if ((e = prepare<kBf16, 8, false>()) != cudaSuccess || (e = prepare<kBf16, 8, true>()) != cudaSuccess ||
      (e = prepare<kF32, 4, false>()) != cudaSuccess)
    return e;
  return prepare<kF32, 1, false>();
}

}  // namespace mlp

using namespace mlp;

extern "C" {

lora_status lora_distill_topk_fwd(const void* logits, int type, const void* ids, int id_bytes, const void* teacher,
                                  int teacher_type, const float* teacher_lse, const float* weight, float temperature,
                                  int64_t M, int64_t V, int64_t top, float* loss, float* probs, float* stats,
                                  void* stream) {
  return lora_distill_topk_fwd_wide(logits, type, ids, id_bytes, teacher, teacher_type, teacher_lse, weight, temperature, M, V,
                                    top, loss, probs, stats, stream);
}

lora_status lora_distill_topk_fwd_wide(const void* logits, int type, const void* ids, int id_bytes, const void* teacher,
                                       int teacher_type, const float* teacher_lse, const float* weight, double temperature,
                                       int64_t M, int64_t V, int64_t top, float* loss, float* probs, float* stats,
                                       void* stream) {
  const float t = float(temperature);
  if (!args_ok(type, id_bytes, t, M, V, top) || !type_ok(teacher_type)) return LORA_ERR_SHAPE;
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
  P.temperature = t;
  P.inv_t = 1.f / t;
  P.inv_t_lo = float(1.0 / temperature - double(P.inv_t));
  P.c = kLog2e / t;
  P.M = M;
  P.V = int(V);
  P.top = int(top);
  P.groups = int(cdiv(V, kGroupElems));
  P.loss = loss;
  P.probs = probs;
  P.stats = stats;
  // Of the row's length alone: one place while a row is short, two, or four where that leaves no warp more half sets. Of many
  // rows fewer places are faster, of few rows more (4096 x 32000 by 1, 2, 4, 8: 61.5, 61.1, 97.7 and 176 us; 4096 x 50256 96, 101, 110
  // and 178, one row of 50257 15.6, 9.6, 9.8 and 8.4; 4096 x 131072 179, 179, 181 and 187, one row 16.5, 10.8, 8.2 and 8.1; 4096 x
  // 151936 219, 222, 253 and 333).
  const int half = kWarps * set_of(type == LORA_F32 ? kF32 : kBf16, V % 8 != 0) / 2;
  const auto halves = [&](int places) { return places * cdiv(P.groups, places * half); };
  P.places = P.groups <= 96 ? 1 : (P.groups >= 448 && halves(4) == halves(1) ? 4 : 2);
  // few rows: a row's places over the CTAs of a cluster
  int cl = 1;
  while (cl < P.places && M * cl * 2 <= 2 * nsm) cl *= 2;
  const cudaError_t e = by_length(type, V, [&](auto kind, auto vec, auto shift) {
    return launch_fwd<kind.value, vec.value, shift.value>(P, cl, nsm, static_cast<cudaStream_t>(stream));
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
  int nsm = 0;
  if ((s = device_ready(&nsm)) != LORA_OK) return s;
  // A CTA's start (its row's statistics, the lists) is the dearer the fewer groups it has: as many as leave every SM some rounds of
  // CTAs (64 and this: 4096 x 131072 bf16 336 and 303 us, in blocks 400 and 319; 64 x 50257 fp32 7.1 and 5.1).
  P.seg = 256;
  while (P.seg > 64 && M * cdiv(P.groups, P.seg) < 12 * nsm) P.seg /= 2;
  if (M * cdiv(P.groups, P.seg) < 2 * nsm) P.seg = 32;
  if (M * (cdiv(P.groups, P.seg) + 1) >= (int64_t(1) << 31)) return LORA_ERR_SHAPE;
  const cudaError_t e = by_length(type, V, [&](auto kind, auto vec, auto shift) {
    return launch_bwd<kind.value, vec.value, shift.value>(P, scales != nullptr, static_cast<cudaStream_t>(stream));
  });
  return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

}  // extern "C"
