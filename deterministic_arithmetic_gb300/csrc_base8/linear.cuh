// linear.cuh -- the tensor-core kernel of the products with weights in 8-bit blocks: e4m3 operands by TMA
// into swizzled shared memory, tcgen05 MMAs (kind::f8f6f4) into FP32 accumulators in TMEM.
//   kLinFwd  y = x w^T     both operands lie along the reduction (K-major)
//   kLinBwd  dx = dy w     the weight's rows lie across it (MN-major): one copy of the codes serves both passes
//
// A block of 128 of the reduction has a scale of its own for each row and each 128 columns, so its sum is
// an accumulator of its own: four MMAs of depth 32 from a cleared start, which the epilogue warps then
// multiply by the scales' product and add to the output's FP32 sum in registers, one fma an element, blocks in
// order. An output's bits depend on its row, its column and the reduction's length only: not on the
// tile it falls into, nor on the batch.
//
// Large products (8192 x 4096 -> 4096 101 us, 2720 TFLOP/s; 4096 x 17408 -> 5120 279) are bound by a chain: TMEM holds two
// accumulators of a 256-column tile, and each is filled, told, read and given back; the tensor pipe is 65 % busy. Few rows are bound by
// an SM's loads, 45 bytes a ns, and by the k-blocks' order (1 x 5120 -> 17408 17.8 us of 13.2 that the memory needs): hence tiles of 32
// to 256 columns, by which more SMs load.
#pragma once

#include "../csrc_mlp/gemm.cuh"
#include "linear.h"

namespace mlp {

constexpr int kLinBK = 128;                        // depth of a k-block: a block of the scales
constexpr int kLinArea = 208 * 1024;               // the operand ring and, behind it, the epilogue warps' boxes
// A box: 32 rows of 64 bytes that TMA stores or (delta's) loads. Tiles of 256 columns have four of each warp, five with delta,
// which leaves the ring four of its 32 KB stages; six are no faster (8192 x 4096 -> 4096: 101 and 100 us). Smaller tiles
// have one; there the MMAs' reads past a short batch's rows of A (whose products nobody reads) end in them.
constexpr int kBox = 32 * 64, kBoxesPlain = 4, kBoxesDelta = 5;
constexpr int lin_boxes(int W, bool delta) { return W < 256 ? 1 : (delta ? kBoxesDelta : kBoxesPlain); }
constexpr int lin_ring(int W, bool delta) { return kLinArea - kEpiWarps * lin_boxes(W, delta) * kBox; }
constexpr int kLinStages = 16;
constexpr int kLinSlots = 4;                       // accumulator slots at most
// Behind that the ring of scales: groups of four k-blocks, a k-block's products of a row's scale and that of each of the (at
// most two) column blocks that a tile touches, [block of columns][row].
constexpr int kScaleGroup = 4, kScaleGroups = 4, kScaleBytes = 2 * kBM * 4;       // (of a k-block)
constexpr int kLinScales = kScaleGroups * kScaleGroup * kScaleBytes;
constexpr int kLinBars = 2 * kLinStages + 2 * kLinSlots + 2 * kScaleGroups + kEpiWarps * 2 + 2;
constexpr size_t kLinSmem = kLinArea + kLinScales + 1024 + kLinBars * 8 + 16;
static_assert(kLinSmem < 227 * 1024, "shared memory of a CTA");

// Four warps to load, issue and idle, eight for the epilogue. Of 256-column tiles an epilogue thread holds 128 sums:
// it takes registers that the first four warps give up (shares of 40 and 232 of the launch's 168 a thread).
constexpr int kLinThreads = 384, kLinRegs = 168, kLinRegsFew = 40, kLinRegsMany = 232;
static_assert(128 * kLinRegsFew + 256 * kLinRegsMany <= kLinThreads * kLinRegs, "the shares fit the launch's registers");

// The bounded waits of waits.cuh, without a call: a kernel that shares out its registers can hold none. And without
// acquires and releases at cluster scope: what the barriers of this kernel stand for is written by copies and tensor cores,
// never by a peer's stores. (Acquiring at that scope throws the SM's L1 away, and a release waits for the thread's loads: of a
// pair's 4096 x 17408 -> 5120, 943 us with both, 411 with neither.)
__device__ __forceinline__ bool lin_done(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0u;
}
// The same of a barrier that says who may use an accumulator. Across a pair the arrival may be the peer's, so the test is one at
// cluster scope; relaxed, for nothing but TMEM hangs on it, and that the threads' tcgen05 fences order: in turn, the tensor
// operation and its wait, fence before, arrival; test, fence after, tensor operation.
template <int CG>
__device__ __forceinline__ bool lin_done_acc(uint32_t bar, uint32_t parity) {
  if constexpr (CG == 1) return lin_done(bar, parity);
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0u;
}
// The whole warp arrives once. Predicated, no branch: where lanes part, the code behind may run once for each part (a
// pair's 4096 x 17408 -> 5120 took 552 us instead of 314 with a warp split so).
__device__ __forceinline__ void lin_arrive(uint32_t bar, bool one) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar), "r"(uint32_t(one))
      : "memory");
}
__device__ __forceinline__ void lin_arrive_peer(uint32_t cluster_addr, bool one) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(cluster_addr), "r"(uint32_t(one))
      : "memory");
}
// Where a wait that runs out reports (common.cuh's Abort, with what only that needs left where it lies).
struct LinAbort {
  uint32_t flag;                   // shared memory
  uint32_t* status;                // a kernel parameter
  __device__ __forceinline__ bool raised() const {
    uint32_t v;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(flag) : "memory");
    return v != 0u;
  }
};
// A wait of the whole warp, which stays together; the same answer in every lane. `quarter`: of the limit (the test hook).
// CG 2: lin_done_acc's, of a pair.
template <int CG = 1>
__device__ __forceinline__ bool lin_wait_longer(uint32_t bar, uint32_t parity, LinAbort ab, uint32_t site, bool teardown = false,
                                                bool quarter = false) {
  const auto test = [&]() {
    if constexpr (CG == 1) return mbar_test(bar, parity);
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0u;
  };
  // (the clock takes longer to read than most waits last: not before some tries)
  for (uint32_t it = 1; it <= 1024u; ++it) {
    if (__all_sync(0xffffffffu, test())) return true;
  }
  const uint32_t us = ab.status[3];
  uint64_t limit = teardown ? kDrainLimitNs : (us ? uint64_t(us) * 1000ull : kWaitLimitNs);
  if (quarter) limit /= 4;
  const uint64_t t0 = global_ns();
  while (true) {
    const bool done = test(), out = global_ns() - t0 > limit;
    if (__all_sync(0xffffffffu, done)) return true;
    if (__any_sync(0xffffffffu, !teardown && ab.raised())) return false;
    if (__any_sync(0xffffffffu, out)) {
      asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(ab.flag), "r"(1u) : "memory");
      if (lane_id() == 0) atomicCAS(ab.status, 0u, (site << 8) | kDevTimeout);   // the first code stays
      __syncwarp();
      return false;
    }
  }
}
__device__ __forceinline__ bool lin_wait(uint32_t bar, uint32_t parity, LinAbort ab, uint32_t site) {
  return __builtin_expect(__all_sync(0xffffffffu, lin_done(bar, parity)), 1) || lin_wait_longer(bar, parity, ab, site);
}
template <int CG>
__device__ __forceinline__ bool lin_wait_acc(uint32_t bar, uint32_t parity, LinAbort ab, uint32_t site) {
  return __builtin_expect(__all_sync(0xffffffffu, lin_done_acc<CG>(bar, parity)), 1) || lin_wait_longer<CG>(bar, parity, ab, site);
}
__device__ __forceinline__ void lin_drain(uint32_t bar, uint32_t parity, LinAbort ab, uint32_t site) {
  if (!__all_sync(0xffffffffu, lin_done(bar, parity))) lin_wait_longer(bar, parity, ab, site, true);
}

// D (+)= A B^T. Of the operands' descriptors the low words differ from MMA to MMA, the high ones never.
template <int CG, int ACCUMULATE>
__device__ __forceinline__ void mma_f8(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "mov.b64 a, {%1, %2};\n\t"
        "mov.b64 b, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "n"(ACCUMULATE)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "mov.b64 a, {%1, %2};\n\t"
        "mov.b64 b, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "n"(ACCUMULATE)
        : "memory");
}
// Instruction descriptor: e4m3 A and B (0), FP32 D, A K-major, B K-major or (b_mn) MN-major.
__device__ __forceinline__ uint32_t idesc_f8(int M, int N, int b_mn) {
  return (1u << 4) | (uint32_t(b_mn) << 16) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// a += s * (x, y), each one fma, as a pair.
__device__ __forceinline__ void add_scaled(float2& a, float s, uint32_t x, uint32_t y) {
  asm("{\n\t.reg .b64 a, v, s;\n\t"
      "mov.b64 a, {%0, %1};\n\t"
      "mov.b64 v, {%2, %3};\n\t"
      "mov.b64 s, {%4, %4};\n\t"
      "fma.rn.f32x2 a, s, v, a;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a.x), "+f"(a.y)
      : "r"(x), "r"(y), "f"(s));
}
template <int N>
__device__ __forceinline__ void tmem_ldn(uint32_t taddr, uint32_t (&r)[N]) {
  static_assert(N == 16 || N == 32, "");
  if constexpr (N == 32) tmem_ld32(taddr, r);
  else tmem_ld16(taddr, r);
}

// Columns of a copied piece of MN-major B, which is its swizzle span; an MMA takes whole pieces.
constexpr int lin_chunk(int W) { return W < 128 ? W : 128; }

// The tile of a unit: groups of up to 16 row tiles, row tiles fastest (gemm.cuh).
struct LinUnit {
  int tm, col, bn;
};
template <int CG>
__device__ __forceinline__ LinUnit lin_unit(const LinArgs& P, int u) {
  const int group = u / (16 * P.tiles_n), m0 = 16 * group;
  const int gm = min(16, P.tiles_m - m0);
  const int r = u - 16 * group * P.tiles_n;
  return {m0 + r % gm, (r / gm) * P.bn, P.bn};
}

// 32 rows by 16 columns of the warp (lane l holds row row0 + l's), plus delta, to the output, by way of the warp's
// 2 KB of shared memory: 4 lanes a row then read and write whole sectors. 16-byte pieces of a row are permuted by the
// row's bits 1 and 2, so that neither way meets a bank twice. Rows past m and columns past `end` are left alone.
__device__ __forceinline__ void lin_store16(const LinArgs& P, uint32_t box, int64_t row0, int col, int end, const float2* acc,
                                            uint32_t lane) {
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(box + lane * 64 + ((j ^ (lane >> 1 & 3)) << 4)),
                 "f"(acc[2 * j].x), "f"(acc[2 * j].y), "f"(acc[2 * j + 1].x), "f"(acc[2 * j + 1].y)
                 : "memory");
  __syncwarp();
  const int c = col + 4 * int(lane & 3);
  const bool whole = P.vec && c < end;             // the row's columns are whole vectors: so are c's
  float4 d[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row0 + 8 * i + int(lane >> 2);
    d[i] = whole && P.delta && row < P.m ? __ldcs(reinterpret_cast<const float4*>(P.delta + row * P.n + c))
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + int(lane >> 2);
    const int64_t row = row0 + r;
    float v[4];
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                 : "r"(box + r * 64 + (((lane & 3) ^ (r >> 1 & 3)) << 4))
                 : "memory");
    if (row >= P.m || c >= end) continue;
    const int64_t at = row * P.n + c;
    if (whole) {
      v[0] += d[i].x; v[1] += d[i].y; v[2] += d[i].z; v[3] += d[i].w;
      if (P.out_f32)
        *reinterpret_cast<float4*>(static_cast<float*>(P.out) + at) = make_float4(v[0], v[1], v[2], v[3]);
      else
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(P.out) + at) =
            make_uint2(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < end) {
          const float y = P.delta ? v[e] + P.delta[at + e] : v[e];
          if (P.out_f32) static_cast<float*>(P.out)[at + e] = y;
          else static_cast<__nv_bfloat16*>(P.out)[at + e] = __float2bfloat16_rn(y);
        }
    }
  }
}

// W: columns of an accumulator (bn rounded up to a power of two); DEEP: k-blocks of a stage, each with an
// accumulator of its own in the slot. JOINS: tiles of 256 columns whose delta comes by boxes (one more thing that the
// epilogue's registers would hold).
template <int MODE, int CG, int W, int DEEP, bool JOINS>
__global__ void __launch_bounds__(kLinThreads, 1) linear_kernel(const __grid_constant__ LinArgs P, uint32_t* status) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem_raw + (base - raw) + kLinArea + kLinScales);
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kLinStages + s); };
  auto tfull = [&](int b) { return bar0 + 8u * (2 * kLinStages + b); };
  auto tempty = [&](int b) { return bar0 + 8u * (2 * kLinStages + kLinSlots + b); };
  auto sfull = [&](int g) { return bar0 + 8u * (2 * kLinStages + 2 * kLinSlots + g); };
  auto sempty = [&](int g) { return bar0 + 8u * (2 * kLinStages + 2 * kLinSlots + kScaleGroups + g); };
  const uint32_t scales = base + kLinArea;
  // delta's boxes of half i of an epilogue warp's columns have come
  auto came = [&](int w, int i) { return bar0 + 8u * (2 * kLinStages + 2 * kLinSlots + 2 * kScaleGroups + 2 * w + i); };
  const uint32_t drain = bar0 + 8u * (kLinBars - 2), never = drain + 8u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kLinBars);
  constexpr int kSlotCols = W * DEEP;              // of TMEM: a stage's accumulators
  constexpr int kSlots = 512 / kSlotCols < kLinSlots ? 512 / kSlotCols : kLinSlots;
  static_assert(kSlots >= 2 && (W >= 32 && W <= 256), "TMEM columns");
  static_assert(CG == 1 || W == 256, "pairs take tiles of 256 columns");

  const uint32_t warp = warp_id(), lane = lane_id();
  const int rank = CG == 2 ? int(cluster_rank()) : 0;       // of a pair: 0 issues the MMAs
  const int stages = P.stages, stage_bytes = DEEP * P.block_bytes;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kLinStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < kSlots; ++b) {
      mbar_init(tfull(b), 1);
      mbar_init(tempty(b), kEpiWarps + (CG == 2 && rank == 0 ? 1 : 0));
    }
    for (int g = 0; g < kScaleGroups; ++g) {
      mbar_init(sfull(g), 1);
      mbar_init(sempty(g), kEpiWarps);
    }
    for (int i = 0; i < kEpiWarps * 2; ++i) mbar_init(came(0, i), 1);
    mbar_init(drain, 1);
    mbar_init(never, 1);
    tmem_slot[1] = 0u;                             // the abort flag
    mbar_fence_init();
    prefetch_map(&P.a);
    prefetch_map(&P.b);
    if (W == 256 && P.boxes) prefetch_map(&P.o);
  }
  // (a pair meets before its joint TMEM allocation and after its freeing, as in gemm.cuh)
  __syncwarp();
  if constexpr (CG == 2) cluster_sync_all();
  if (warp == 1) acc_alloc<CG>(smem_u32(tmem_slot));
  __syncwarp();
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  grid_dependents_launch();
  const LinAbort ab{drain + 20u, status};
  const int first = blockIdx.x / CG, step = gridDim.x / CG;
  // a copied piece of MN-major B: kChunk columns of 128 rows of the weight, its swizzle span
  constexpr int kChunk = lin_chunk(W);

  if (warp < 4) {
  if constexpr (W == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLinRegsFew));
  if (warp == 0) {
    // ------------------------------------------------------------ producer (gemm.cuh's)
    const bool one = elect_one();
    if (stall_requested(status, kKindLinear + MODE)) lin_wait_longer(never, 0u, ab, kSiteLinear + 1, false, true);   // test hook
    __syncwarp();
    // (of one row of tiles each byte of the weight is read once: 1 x 5120 <- 17408 25.7 -> 24.4 us)
    const uint64_t pa = P.tiles_n > 1 ? policy_evict_last() : policy_normal();
    const uint64_t pb = P.tiles_m > 1 ? policy_normal() : policy_evict_first();
    const uint32_t full0 = CG == 2 ? peer_addr(full(0), 0) : full(0);
    int idx = 0;
    uint32_t phase = 0, issued = 0;
    bool ready = true;
    for (int u = first; u < P.total; u += step) {
      const LinUnit w = lin_unit<CG>(P, u);
      const int row0 = (w.tm * CG + rank) * kBM;           // this CTA's rows of A
      const int col0 = w.col + rank * (w.bn / 2);          // and columns (of a pair, half of the tile's)
      for (int kb = 0; kb < P.nk; kb += DEEP) {
        if (!__all_sync(0xffffffffu, ready) && !lin_wait(empty(idx), phase ^ 1u, ab, kSiteLinear + 2)) goto given_up;
        const uint32_t st0 = base + uint32_t(idx) * stage_bytes, bar = full0 + 8u * idx, here = full(idx);
        if (++idx == stages) idx = 0, phase ^= 1u;
        ready = lin_done(empty(idx), phase ^ 1u);
        ++issued;
        if (one) {
          if (rank == 0) mbar_expect_tx(here, uint32_t(CG * (DEEP == 1 ? 1 : min(DEEP, P.nk - kb)) * P.block_bytes));
#pragma unroll
          for (int k = 0; k < DEEP; ++k) {
            if (k > 0 && kb + k >= P.nk) break;
            const uint32_t st = st0 + k * P.block_bytes, sb = st + P.a_bytes;
            const int k0 = (kb + k) * kLinBK;
            load2d<CG>(st, &P.a, bar, k0, row0, pa);
            if constexpr (MODE == kLinFwd) {
              load2d<CG>(sb, &P.b, bar, k0, col0, pb);
            } else {
#pragma unroll 1
              for (int j = 0; j < P.bn / CG; j += kChunk) load2d<CG>(sb + j * kLinBK, &P.b, bar, col0 + j, k0, pb);
            }
          }
        }
        __syncwarp();
      }
    }
  given_up:
    // nothing may reach this CTA's shared memory once it has gone (gemm.cuh)
    for (uint32_t s = 0; s < uint32_t(stages) && s < issued; ++s) {
      const uint32_t parity = ((issued - 1u - s) / stages) & 1u;       // of the stage's last use
      if (rank == 0) lin_drain(full(s), parity, ab, kSiteLinear + 3);
      if (!ab.raised()) lin_wait(empty(s), parity, ab, kSiteLinear + 8);
    }
    if (ab.raised())
      for (const uint64_t t0 = global_ns(); global_ns() - t0 < kDrainLimitNs;) {
      }
    __syncwarp();
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer
    if (rank == 0) {
      // K-major operands step 32 bytes inside the swizzle span per 32 of the reduction; MN-major ones 32 rows.
      constexpr uint32_t kSpan = MODE == kLinFwd ? 128 : kChunk, a_step = 32u, b_step = MODE == kLinFwd ? 32u : 32u * kSpan;
      const uint64_t a0 = smem_desc(base, 16u, 1024u, kLayoutSW128);
      const uint64_t b0 = smem_desc(base + P.a_bytes, MODE == kLinFwd ? 16u : kLinBK * kSpan, 8u * kSpan, layout_for_span(kSpan));
      const uint32_t a_lo = uint32_t(a0), a_hi = uint32_t(a0 >> 32), b_lo = uint32_t(b0), b_hi = uint32_t(b0 >> 32);
      const uint32_t idesc = idesc_f8(CG * kBM, P.bn, MODE == kLinBwd);
      const bool one = elect_one();
      int idx = 0, buf = 0;
      uint32_t phase = 0, tphase = 0;
      // Whether stage idx has landed and slot buf has been read: tested as soon as the one before is issued. (This warp's own
      // steps are what bounds the large tiles.)
      bool landed = false, free = true, ok = true;
      for (int u = first; u < P.total; u += step) {
        for (int kb = 0; kb < P.nk; kb += DEEP) {
          if (!__all_sync(0xffffffffu, landed)) ok = lin_wait(full(idx), phase, ab, kSiteLinear + 5);
          if (!ok) break;
          const uint32_t off = uint32_t(idx) * stage_bytes, used = empty(idx);
          if (++idx == stages) idx = 0, phase ^= 1u;
          if (!__all_sync(0xffffffffu, free)) ok = lin_wait_acc<CG>(tempty(buf), tphase ^ 1u, ab, kSiteLinear + 4);
          if (!ok) break;
          tc_fence_after();
          if (one) {
            const uint32_t d = tmem + buf * kSlotCols;
#pragma unroll
            for (int k = 0; k < DEEP; ++k) {
              if (k > 0 && kb + k >= P.nk) break;
              const uint32_t a = a_lo + ((off + k * P.block_bytes) >> 4), b = b_lo + ((off + k * P.block_bytes) >> 4);
              mma_f8<CG, 0>(d + k * W, a, a_hi, b, b_hi, idesc);
#pragma unroll
              for (int j = 1; j < kLinBK / 32; ++j)
                mma_f8<CG, 1>(d + k * W, a + (j * a_step >> 4), a_hi, b + (j * b_step >> 4), b_hi, idesc);
            }
            commit<CG>(tfull(buf));
            commit<CG>(used);
          }
          __syncwarp();
          if (++buf == kSlots) buf = 0, tphase ^= 1u;
          free = lin_done_acc<CG>(tempty(buf), tphase ^ 1u);
          landed = lin_done(full(idx), phase);
        }
      }
      if (one) commit_here<CG>(drain);
      __syncwarp();
      lin_drain(drain, 0u, ab, kSiteLinear + 6);
    } else {
      // of a pair's second CTA: tells the first, once for all of its epilogue warps, that they have read a slot (arrivals across
      // the pair are slow: an arrival of each warp, 332 us and 293 at 4096 x 17408 -> 5120)
      int buf = 0;
      uint32_t tphase = 0;
      bool ok = true;
      for (int u = first; u < P.total; u += step)
        for (int i = 0; i < P.nk && ok; ++i) {
          ok = lin_wait_acc<CG>(tempty(buf), tphase, ab, kSiteLinear + 11);
          tc_fence_after();                        // (passes the warps' order on)
          tc_fence_before();
          lin_arrive_peer(peer_addr(tempty(buf), 0), ok && lane == 0);
          if (++buf == kSlots) buf = 0, tphase ^= 1u;
        }
    }
  } else {
    // ------------------------------------------------------ scales, two warps
    // Their groups in turn. (Loaded by the epilogue's warps themselves, the scales' latency was most of a k-block's time: of a
    // pair's 4096 x 17408 -> 5120, 411 us so, 337 with these warps.)
    uint32_t n = 0;                                // groups so far, of both warps
    bool ok = true;
    for (int u = first; u < P.total; u += step) {
      const LinUnit w = lin_unit<CG>(P, u);
      const int64_t row0 = int64_t(w.tm * CG + rank) * kBM + lane;
      const float* sb[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) sb[e] = P.sb + min(w.col / 128 + e, (P.n - 1) / 128) * P.sb_out;
      for (int kb = 0; kb < P.nk && ok; kb += kScaleGroup, ++n) {
        if ((n & 1u) != (warp & 1u)) continue;
        const uint32_t g = n % kScaleGroups;
        ok = lin_wait(sempty(g), (n / kScaleGroups & 1u) ^ 1u, ab, kSiteLinear + 9);
        if (!ok) break;
        const uint32_t at = scales + g * kScaleGroup * kScaleBytes + lane * 4;
#pragma unroll 1
        for (int h = 0; h < kScaleGroup; h += 2) {
          float a[2][4], b[2][2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const bool in = kb + h + k < P.nk;
#pragma unroll
            for (int j = 0; j < 4; ++j) a[k][j] = in ? __ldg(P.sa + min(row0 + 32 * j, int64_t(P.m) - 1) * P.nk + kb + h + k) : 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) b[k][e] = in ? __ldg(sb[e] + (kb + h + k) * P.sb_red) : 0.f;
          }
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + (h + k) * kScaleBytes + e * kBM * 4 + j * 128), "f"(a[k][j] * b[k][e])
                             : "memory");
        }
        __syncwarp();
        lin_arrive(sfull(g), lane == 0);
      }
    }
  }
  } else {
    // ------------------------------------------------------------ epilogue
    if constexpr (W == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kLinRegsMany));
    // A warp has its quarter of the rows and half of the tile's columns, in chunks of C.
    constexpr int C = W >= 64 ? 32 : 16, kChunks = W / 2 / C;
    constexpr int kScales = W == 256 ? 1 : 2;                      // scales of a lane's row, of the warp's columns, a k-block
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lanes = uint32_t(q * 32) << 16;
    const int off = half * (W / 2);                                // its first column in the tile
    auto column = [&](int i) { return off + i; };                  // and its i-th
    auto scale_of = [](int i) { return i * kScales / (W / 2); };   // which of the scales that has
    int buf = 0;
    uint32_t tphase = 0, n = 0;                    // groups of scales so far
    // No wait has run out. Once one has, no more of delta is loaded: a barrier that was told of boxes is told no second time.
    bool ok = true;
    const uint32_t box0 = base + lin_ring(W, JOINS) + (warp - 4) * lin_boxes(W, JOINS) * kBox;
    uint32_t dphase = 0;
    for (int u = first; u < P.total; u += step) {
      const LinUnit w = lin_unit<CG>(P, u);
      const int64_t row0 = int64_t(w.tm * CG + rank) * kBM + q * 32;
      const bool rows = row0 < P.m;
      uint32_t block[kScales];                     // where in a k-block's scales
#pragma unroll
      for (int e = 0; e < kScales; ++e)
        block[e] = uint32_t((w.col + column(e * (W / 2) / kScales)) / 128 - w.col / 128) * (kBM * 4) + (q * 32 + lane) * 4;
      auto boxed = [&](int i) { return rows && w.col + column(16 * i) < P.n; };
      // delta's box i (16 columns), into a place; TMA fills what lies past its ends with zeros. The boxes of a half of the tile
      // complete one barrier, which is told how many there are.
      auto load_delta = [&](int i, int place, int half) {
        if (lane == 0)
          tma_load(box0 + place * kBox, &P.d, came(warp - 4, half), w.col + column(16 * i), int(row0), policy_normal());
      };
      auto expect = [&](int half) {
        int boxes = 0;
        for (int i = 4 * half; i < 4 * half + 4; ++i) boxes += boxed(i);
        if (lane == 0) mbar_expect_tx(came(warp - 4, half), boxes * kBox);
      };
      if constexpr (JOINS) {
        if (ok && boxed(0)) {
          if (lane == 0) tma_store_wait_read<0>();   // the tile before has left the places
          __syncwarp();
          expect(0);
#pragma unroll 1
          for (int i = 0; i < 4; ++i)
            if (boxed(i)) load_delta(i, i, 0);
          if (boxed(4)) {
            expect(1);
            load_delta(4, 4, 1);
#pragma unroll 1
            for (int i = 5; i < 8; ++i)
              if (boxed(i) && lane == 0) tma_prefetch_l2(&P.d, w.col + column(16 * i), int(row0));
          }
        }
      }
      float2 acc[kChunks * C / 2];
      if constexpr (!JOINS) ok = true;               // (kept across tiles, it costs the large ones 2 %)
#pragma unroll
      for (int i = 0; i < kChunks * C / 2; ++i) acc[i] = make_float2(0.f, 0.f);
      for (int kb0 = 0; kb0 < P.nk; kb0 += kScaleGroup, ++n) {
        const uint32_t g = n % kScaleGroups, sg = scales + g * kScaleGroup * kScaleBytes;
        ok = lin_wait(sfull(g), n / kScaleGroups & 1u, ab, kSiteLinear + 10) && ok;
#pragma unroll(DEEP)                               // (code that does not fit the instruction caches costs more)
        for (int k = 0; k < kScaleGroup; ++k) {
          if (kb0 + k >= P.nk) break;
          float s[kScales];
#pragma unroll
          for (int e = 0; e < kScales; ++e)
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(s[e]) : "r"(sg + k * kScaleBytes + block[e]) : "memory");
          const bool last = k % DEEP == DEEP - 1 || kb0 + k == P.nk - 1;       // of its slot
          if (k % DEEP == 0) {
            ok = lin_wait_acc<CG>(tfull(buf), tphase, ab, kSiteLinear + 7) && ok;
            tc_fence_after();
          }
          auto leave = [&]() {
            tc_fence_before();
            __syncwarp();
            lin_arrive(tempty(buf), ok && lane == 0);
            if (++buf == kSlots) buf = 0, tphase ^= 1u;
          };
          if (ok && rows) {
            // a chunk is on its way while the one before is added; the slot is given back when the last has come
            const uint32_t at = tmem + buf * kSlotCols + (k % DEEP) * W + lanes + off;
            uint32_t r[kChunks > 1 ? 2 : 1][C];
            tmem_ldn(at, r[0]);
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
              uint32_t(&v)[C] = r[kChunks > 1 ? i & 1 : 0];
              tmem_ld_wait();
              reg_fence(v);
              if (i + 1 < kChunks) tmem_ldn(at + (i + 1) * C, r[(i + 1) & 1]);
              else if (last) leave();
#pragma unroll
              for (int e = 0; e < C; e += 2) add_scaled(acc[(i * C + e) / 2], s[scale_of(i * C + e)], v[e], v[e + 1]);
            }
          } else if (last) {
            leave();
          }
        }
        __syncwarp();
        lin_arrive(sempty(g), ok && lane == 0);
      }
      if (W == 256 && P.boxes) {
        // The warp's 128 columns, in boxes of 32 (bf16) or 16 (fp32). A box holds 32 rows of 64 bytes, whose 16-byte pieces are
        // permuted by the row's bits 1 and 2; a lane reads and writes its own row's.
        const uint32_t mine = box0 + lane * 64, turn = lane >> 1 & 3;
        auto put = [&](int i, uint32_t box) {      // 16 columns from the i-th 16 on
          const float2* a = acc + 8 * i;
          if (P.out_f32) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(mine + box * kBox + ((j ^ turn) << 4)), "f"(a[2 * j].x),
                           "f"(a[2 * j].y), "f"(a[2 * j + 1].x), "f"(a[2 * j + 1].y)
                           : "memory");
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(mine + box * kBox + (((2 * (i & 1) + j) ^ turn) << 4)),
                           "r"(bf16x2_bits(a[4 * j].x, a[4 * j].y)), "r"(bf16x2_bits(a[4 * j + 1].x, a[4 * j + 1].y)),
                           "r"(bf16x2_bits(a[4 * j + 2].x, a[4 * j + 2].y)), "r"(bf16x2_bits(a[4 * j + 3].x, a[4 * j + 3].y))
                           : "memory");
          }
        };
        auto send = [&](int i, uint32_t box) {     // lane 0: a box whose first column is the i-th 16's
          if (ok && boxed(i)) tma_store(&P.o, box0 + box * kBox, w.col + column(16 * i), int(row0), policy_normal());
        };
        auto join = [&](int i, uint32_t place) {   // delta's box i
          float2* a = acc + 8 * i;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float4 v;
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                         : "r"(mine + place * kBox + ((j ^ turn) << 4))
                         : "memory");
            a[2 * j].x += v.x; a[2 * j].y += v.y; a[2 * j + 1].x += v.z; a[2 * j + 1].y += v.w;
          }
        };
        auto handed = [&]() {                      // the boxes are written
          fence_proxy_async();
          __syncwarp();
        };
        if (!boxed(0)) {
          // (nothing of the tile is the warp's)
        } else if constexpr (JOINS) {
          // First half: delta's boxes have come during the k-blocks. The results go over them, and what is free again takes
          // the second half's boxes (all but one: that came with the first).
          ok = lin_wait(came(warp - 4, 0), dphase & 1u, ab, kSiteLinear + 12) && ok;
          dphase ^= 1u;
#pragma unroll
          for (int i = 0; i < 4; ++i) join(i, i);
          __syncwarp();
          if (!P.out_f32 && ok && boxed(4)) {
            if (boxed(5)) load_delta(5, 2, 1);
            if (boxed(6)) load_delta(6, 3, 1);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) put(i, P.out_f32 ? i : i / 2);
          handed();
          if (lane == 0) {
            for (int i = 0; i < 4; i += P.out_f32 ? 1 : 2) send(i, P.out_f32 ? i : i / 2);
            tma_store_commit();
            tma_store_wait_read<0>();
          }
          __syncwarp();
          if (ok && boxed(4)) {
            if (P.out_f32) {
              if (boxed(5)) load_delta(5, 2, 1);
              if (boxed(6)) load_delta(6, 3, 1);
            }
            if (boxed(7)) load_delta(7, 0, 1);
          }
          if (boxed(4)) {
            ok = lin_wait(came(warp - 4, 1), dphase >> 1 & 1u, ab, kSiteLinear + 12) && ok;
            dphase ^= 2u;
            join(4, 4);
            join(5, 2);
            join(6, 3);
            join(7, 0);
            put(4, 4);
            put(5, P.out_f32 ? 2 : 4);
            put(6, P.out_f32 ? 3 : 2);
            put(7, P.out_f32 ? 0 : 2);
            handed();
            if (lane == 0) {
              send(4, 4);
              if (P.out_f32) send(5, 2);
              send(6, P.out_f32 ? 3 : 2);
              if (P.out_f32) send(7, 0);
              tma_store_commit();
            }
          }
        } else {
          // (bf16: all at once; fp32 fills the four boxes twice)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h == 0 || P.out_f32) {
              if (lane == 0) tma_store_wait_read<0>();
              __syncwarp();
            }
#pragma unroll
            for (int i = 4 * h; i < 4 * h + 4; ++i) put(i, P.out_f32 ? i & 3 : i / 2);
            if (h == 1 || P.out_f32) {
              handed();
              if (lane == 0) {
                const int step = P.out_f32 ? 1 : 2;
                for (int i = P.out_f32 ? 4 * h : 0; i < 4 * h + 4; i += step) send(i, P.out_f32 ? i & 3 : i / 2);
                tma_store_commit();
              }
            }
          }
        }
      } else if (ok && rows) {
        const int end = min(P.n, w.col + w.bn);
#pragma unroll
        for (int i = 0; i < kChunks * C; i += 16)
          if (column(i) < w.bn) lin_store16(P, box0, row0, w.col + column(i), end, acc + i / 2, lane);
      }
    }
    if (W == 256 && lane == 0) tma_store_wait_all<0>();
  }

  __syncwarp();
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync_all();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    acc_free<CG>(tmem);
  }
  __syncwarp();
  if constexpr (CG == 2) cluster_sync_all();
}

}  // namespace mlp
