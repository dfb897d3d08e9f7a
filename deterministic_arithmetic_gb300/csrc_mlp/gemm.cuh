// gemm.cuh -- the tensor-core kernel of the gated feed-forward block: bf16 operands by TMA into
// 128-byte-swizzled shared memory, tcgen05 MMAs into FP32 accumulators in TMEM, three products:
//   kFwd  G = x Wg^T and U = x Wu^T over the same x tile, and in the epilogue h = act(G + Dg) (U + Du),
//         with G + Dg and U + Du kept in bf16 or in 8 bits when asked for
//   kDx   dx = dG Wg + dU Wu
//   kDw   dWg = dG^T x and dWu = dU^T x
//
// An accumulator takes its reduction in order, 16 products at a time, from a cleared start, and how a
// reduction is cut depends on its length alone: an output's bits do not depend on the tile it falls into,
// nor on how many rows the batch has. FP32 accumulation; each output is rounded to bf16 once, in the
// epilogue.
//
// 4096 x 5120 x 17408: 767 us forward (1.90 PFLOP/s), 856 dx, 760 dW on a cool device. Bound by the tensor
// pipe (77 to 82 % active at 2048 x 4096 x 8192) and, back to back, by the device's power: the clock falls
// to some 1.6 GHz, and plain library products of the sizes take 830 to 860 us. One token (5120 -> 17408): 57 us, the
// weights' 356 MB at 6.2 TB/s.
//
// CG = 2 works in pairs of CTAs (a cluster of two neighbouring SMs, cta_group::2): a 256 x 256 tile,
// each CTA holding 128 rows of A, half of B's columns and the accumulator of its rows, so that each
// operand byte in shared memory feeds twice the products of a CTA alone. The pair's first CTA
// issues the MMAs of both; copies of both arrive at its barriers. CG = 1 is a CTA alone with 128
// rows and bn columns, for batches and outputs too small to give every pair a tile.
//
// dx's reductions are the longest (both of F), and its outputs the smallest. So each product is taken in
// up to four pieces, an accumulator each, and the pieces are added in order: every variant adds the same
// ones, so the bits are the same. SPLIT (kDx, CG = 1) is a cluster a tile:
//   2   a product a CTA: the first sends its pieces' sum to the second, which holds its own pieces in four
//       accumulators and adds them to that
//   8   a piece a CTA, for outputs of very few tiles: every CTA sends 16 rows of its accumulator to each of
//       the others, and adds and stores 16 rows itself
//
// Persistent CTAs (pairs) take tiles in turn. Warp 0 loads, warp 1 issues the MMAs, warps 2 to 9 read the
// accumulator and write the tile (a warp its quarter of the lanes, the two halves of the warps
// alternate 32-column chunks); two accumulators of 256 TMEM columns let a tile's epilogue run under
// the next tile's MMAs.
#pragma once

#include "../csrc/common.cuh"
#include "../csrc/kernels.h"
#include "elems.cuh"
#include "gated_ffn.h"
#include "mlp.h"
#include "pack8.cuh"
#include "waits.cuh"

namespace mlp {

using namespace lora;

constexpr int kABytes = kBM * kBK * 2;             // 16 KB
constexpr int kMaxStages = 16;
constexpr int kRingBytes = 192 * 1024;             // the operand ring
// Behind it: a stage of a small batch holds fewer than 128 rows of A, and the MMAs' reads of the other
// rows (whose products nobody reads) run on into what follows, in the last stage to here.
// The same place holds the boxes that dW's epilogue writes out (two of 2 KB a warp), and ends with what a
// split's CTAs send one another.
constexpr int kEpiWarps = 8;
constexpr int kBoxBytes = 32 * 32 * 2, kRingSlack = kEpiWarps * 2 * kBoxBytes;
static_assert(kRingSlack >= kABytes, "the reads past a short A stay inside");
constexpr int kGemmThreads = 32 * (2 + kEpiWarps);
constexpr int kMaxPieces = 4;                      // of a product of dx
constexpr int kMaxAccs = 4;                        // accumulators in the 512 columns of TMEM
constexpr size_t kGemmSmem = kRingBytes + kRingSlack + 1024 + (2 * kMaxStages + 2 * kMaxAccs + 3) * 8 + 16;
static_assert(kGemmSmem < 227 * 1024, "shared memory of a CTA");

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
      "%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// ------------------------------------------------------------ pairs of CTAs
// The same operations as common.cuh's, for cta_group::2. `bar` of a copy is the address of the first
// CTA's barrier (peer_addr), dst the caller's own shared memory.
template <int CG>
__device__ __forceinline__ void load2d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y, uint64_t policy) {
  if constexpr (CG == 1) {
    tma_load(dst, m, bar, x, y, policy);
  } else {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "l"(policy)
        : "memory");
  }
}
// A box of a block_map: 64-column blocks from block z, rows from y.
template <int CG>
__device__ __forceinline__ void load3d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int y, int z, uint64_t policy) {
  if constexpr (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(0), "r"(y), "r"(z), "l"(policy)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(0), "r"(y), "r"(z), "l"(policy)
        : "memory");
}
__device__ __forceinline__ uint64_t policy_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (CG == 1) {
    mma_bf16(d, a, b, idesc, accumulate);
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}
// Arrive on `bar` (with CG = 2: on that barrier of both CTAs) once the MMAs issued so far are done.
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (CG == 1) {
    mma_commit(bar);
  } else {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(uint16_t(3))
        : "memory");
  }
}
// The same on the caller's barrier alone.
template <int CG>
__device__ __forceinline__ void commit_here(uint32_t bar) {
  if constexpr (CG == 1)
    mma_commit(bar);
  else
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
template <int CG>
__device__ __forceinline__ void acc_alloc(uint32_t slot) {
  if constexpr (CG == 1) {
    tmem_alloc(slot, 512);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void acc_free(uint32_t taddr) {
  if constexpr (CG == 1)
    tmem_dealloc(taddr, 512);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(512) : "memory");
}

// act(y) = y p and its slope p + y p (1 - p) z', with p = 1 / (1 + exp(-z)): z = y for silu; for gelu in
// its tanh form 0.5 y (1 + tanh(s)) = y / (1 + exp(-2 s)), z = 2 s = sqrt(8 / pi) (y + 0.044715 y^3).
// The fast exponential and division, a few units of FP32's last place (the exponential's grow with |z|):
// every result is rounded to bf16 or to a step of 8 bits, some 2^-9 of it, right after.
__device__ __forceinline__ float act_p(int act, float y) {
  const float z = act == LORA_ACT_SILU ? y : 1.5957691216057308f * fmaf(0.044715f * y * y, y, y);
  return __fdividef(1.f, 1.f + __expf(-z));        // exp overflowing to infinity gives 0
}
__device__ __forceinline__ float act_slope(int act, float y, float p) {
  const float q = 1.f - p;
  if (p == 0.f || q == 0.f) return p;              // the tails: the second term is 0, its factors may be infinite
  const float dz = act == LORA_ACT_SILU ? 1.f : 1.5957691216057308f * fmaf(0.134145f * y, y, 1.f);
  return fmaf(y * p, q * dz, p);
}

// 32 rows by 32 columns of the warp, as bf16: lane l holds row row0 + l's columns from `col` on. Rows at or
// past m and columns at or past n (a multiple of 8) are left alone. Lanes of a quad first trade 8-column
// pieces, so that a store writes 64 bytes of each of 8 rows: 16 bytes of each of 32 rows took four times
// the accesses (dW of one token 5120 x 17408, which went this way then: 208 -> 109 us).
__device__ __forceinline__ void store_rows32(__nv_bfloat16* out, int64_t row0, int64_t m, int64_t ld, int col, int n,
                                             const float (&v)[32], uint32_t lane) {
  uint32_t p[4][4];                                // [piece][word]
#pragma unroll
  for (int j = 0; j < 16; ++j) p[j >> 2][j & 3] = bf16x2_bits(v[2 * j], v[2 * j + 1]);
  // a 4 x 4 transposition: piece j of lane t of the quad becomes piece t of lane j
#pragma unroll
  for (int b = 1; b <= 2; b <<= 1) {
    const bool up = lane & b;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j & b) continue;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? p[j][w] : p[j | b][w], b);
        if (up) p[j][w] = got;
        else p[j | b][w] = got;
      }
    }
  }
  const int c = col + 8 * int(lane & 3);
  const int64_t r = row0 + (lane & ~3u);
  __nv_bfloat16* at = out + r * ld + c;
  if (c < n) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (r + j < m) *reinterpret_cast<uint4*>(at + j * ld) = make_uint4(p[j][0], p[j][1], p[j][2], p[j][3]);
  }
}

// One of the forward's kept values, the warp's 32 rows by 32 columns from `col`, those before `end`. Packed:
// `col` is a multiple of 32, and `end` the row's unless a whole chunk away.
__device__ __forceinline__ void keep_rows32(const FfnArgs& P, int which, int64_t row0, int col, int end, float (&v)[32],
                                            uint32_t lane) {
  if (P.keep_kind == LORA_KEEP_BF16) {
    store_rows32(static_cast<__nv_bfloat16*>(P.keep[which]), row0, P.m, P.n, col, end, v, lane);
    return;
  }
  const int64_t row = row0 + lane;
  if (row >= P.m) return;
  const int G = (P.n + 31) >> 5;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    if (col + i >= P.n) v[i] = 0.f;                // the padding of the last group (never read from here on)
    m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  }
  const uint32_t s = scale_byte(m);
  const float inv = inv_step(s);
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = codes4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3], inv, s);
  uint4* q = reinterpret_cast<uint4*>(static_cast<int8_t*>(P.keep[which]) + (row * G + (col >> 5)) * 32);
  q[0] = make_uint4(w[0], w[1], w[2], w[3]);
  q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  P.keep_scales[which][row * G + (col >> 5)] = uint8_t(s);
}

// A unit of work: a tile, or (pairs only, the last round's) the left or right half of one's columns.
// Tiles lie in groups of up to 16 row tiles, row tiles fastest: the CTAs at work together then share
// a few column tiles and the operand rows of at most 16 row tiles, which stay in L2.
struct Unit {
  int prod, tm, col, bn;           // product (kDw), row tile, first column and columns (of each projection in kFwd)
};
template <int MODE, int CG>
__device__ __forceinline__ Unit unit_at(const FfnArgs& P, int u) {
  int tile = u, half = -1;
  if (CG == 2 && u >= P.whole) {
    tile = P.whole + (u - P.whole) / 2;
    half = (u - P.whole) & 1;
  }
  Unit w;
  const int per = P.tiles_m * P.tiles_n;
  w.prod = MODE == kDw ? tile / per : 0;
  tile -= w.prod * per;
  const int group = tile / (16 * P.tiles_n), m0 = 16 * group;
  const int gm = min(16, P.tiles_m - m0);
  const int r = tile - 16 * group * P.tiles_n;
  w.tm = m0 + r % gm;
  w.bn = half < 0 ? P.bn : P.bn / 2;
  w.col = (r / gm) * P.bn + (half == 1 ? w.bn : 0);
  return w;
}

template <int MODE, int CG, int SPLIT = 0, int DEEP = 1>
__global__ void __launch_bounds__(kGemmThreads, 1) ffn_gemm_kernel(const __grid_constant__ FfnArgs P, uint32_t* status) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem_raw + (base - raw) + kRingBytes + kRingSlack);
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  auto tfull = [&](int b) { return bar0 + 8u * (2 * kMaxStages + b); };
  auto tempty = [&](int b) { return bar0 + 8u * (2 * kMaxStages + kMaxAccs + b); };
  const uint32_t drain = bar0 + 8u * (2 * kMaxStages + 2 * kMaxAccs);
  const uint32_t never = drain + 8u;
  const uint32_t sent = drain + 16u;                 // SPLIT: what the other CTAs send has arrived
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kMaxStages + 2 * kMaxAccs + 3);
  volatile uint32_t* abort_flag = tmem_slot + 1;

  const uint32_t warp = warp_id(), lane = lane_id();
  static_assert(!SPLIT || (MODE == kDx && CG == 1), "a split is dx's");
  static_assert(SPLIT == 0 || SPLIT == 2 || SPLIT == 8, "by product or by piece");
  constexpr int kCluster = SPLIT ? SPLIT : CG;
  constexpr int kAccs = SPLIT == 2 ? 4 : 2, kAccCols = 512 / kAccs;   // accumulators of up to 256 (or 128) columns
  const int peer = kCluster > 1 ? int(cluster_rank()) : 0;
  const int rank = CG == 2 ? peer : 0;                      // of a pair: 0 issues the MMAs
  const int stages = P.stages, stage_bytes = DEEP * P.block_bytes;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < kAccs; ++b) {
      mbar_init(tfull(b), 1);
      mbar_init(tempty(b), CG * kEpiWarps);
    }
    mbar_init(drain, 1);
    mbar_init(never, 1);
    mbar_init(sent, SPLIT == 8 ? 2 * SPLIT : kEpiWarps);
    *abort_flag = 0u;
    mbar_fence_init();
    for (int i = 0; i < 2; ++i) {
      prefetch_map(&P.a[i]);
      prefetch_map(&P.b[i]);
    }
  }
  // A pair's TMEM is allocated, and at the end freed, by both CTAs together: each only once the other is
  // known to run (the hardware starts a cluster's CTAs together, but not in the same instant, and an
  // allocation met by no peer does not return). The same meeting shows that the peer's barriers are set up.
  __syncwarp();
  if constexpr (kCluster > 1) cluster_sync_all();
  if (warp == 1) acc_alloc<CG>(smem_u32(tmem_slot));
  __syncwarp();
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  grid_dependents_launch();
  const Abort ab = make_abort(abort_flag, status);

  // A tile's pieces of this CTA (pair), each into the next accumulator, and their k-blocks. Of a split by
  // piece it is piece peer & 3 of product peer >> 2 (of fewer than four, the rest have no blocks).
  const int pieces = MODE != kDx || SPLIT == 8 ? 1 : (SPLIT ? 1 : 2) * P.pieces;
  const int piece0 = SPLIT == 8 ? (peer & 3) * P.piece : 0;
  auto blocks_of = [&](int i) {
    if constexpr (MODE != kDx) return P.nk;
    const int k0 = SPLIT == 8 ? piece0 : (i >= P.pieces ? i - P.pieces : i) * P.piece;
    return min(max(P.nk - k0, 0), P.piece);
  };
  const bool empty_piece = SPLIT == 8 && blocks_of(0) == 0;
  const int first = blockIdx.x / kCluster, step = gridDim.x / kCluster;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // The whole warp runs this loop and the next (their addresses stay in uniform registers), one lane
    // issues, and a stage's barrier is tested before the stage in front of it is issued. Its bookkeeping
    // (and the issuer's: tests, commit) takes some 400 cycles, more than the copies and MMAs of a narrow
    // tile's k-block: so a stage holds DEEP of them, up to four where the ring has room for four such stages.
    const bool one = elect_one();
    if (stall_requested(status, kKindFfn + MODE) && one) stall_wait(never, ab, kSiteFfn + 1);   // test hook
    __syncwarp();
    // x is read again by every column of tiles (kFwd) or every group of row tiles (kDw): it stays
    // in L2. The rest is shared by the CTAs at work at one time only.
    const uint64_t keep = policy_evict_last(), once = policy_normal();
    const uint64_t pa = MODE == kFwd ? keep : once, pb = MODE == kDw ? keep : once;
    const uint32_t full0 = CG == 2 ? peer_addr(full(0), 0) : full(0);
    int idx = 0;
    uint32_t phase = 0, issued = 0;
    bool ready = true;                               // stage idx is free (at first all are)
    for (int u = first; u < P.total; u += step) {
      const Unit w = unit_at<MODE, CG>(P, u);
      const int row0 = (w.tm * CG + rank) * kBM;           // this CTA's rows of A
      const int col0 = w.col + rank * (w.bn / 2);          // kDx, kDw: its columns of B
      // the boxes are a whole tile's: half a tile uses half of what it loads
      for (int i = 0; i < pieces; ++i) {
        const bool second = MODE == kDx && !SPLIT && i >= P.pieces;
        const int h = SPLIT == 8 ? peer >> 2 : (SPLIT ? peer : int(second));       // dx: the product
        const CUtensorMap* ma = &P.a[MODE == kDw ? w.prod : h];
        const CUtensorMap* mb = &P.b[MODE == kFwd && CG == 2 ? rank : h];
        const int begin = piece0 + (MODE == kDx ? (i - (second ? P.pieces : 0)) * P.piece : 0), end = begin + blocks_of(i);
        for (int kb = begin; kb < end; kb += DEEP) {
          if (!__all_sync(0xffffffffu, ready || wait_longer(empty(idx), phase ^ 1u, ab, kSiteFfn + 2))) goto given_up;
          const uint32_t st0 = base + uint32_t(idx) * stage_bytes, bar = full0 + 8u * idx, here = full(idx);
          if (++idx == stages) idx = 0, phase ^= 1u;
          ready = completed(empty(idx), phase ^ 1u);
          ++issued;
          if (one) {
            if (rank == 0) mbar_expect_tx(here, uint32_t(CG * (DEEP == 1 ? 1 : min(DEEP, end - kb)) * P.block_bytes));
#pragma unroll
            for (int k = 0; k < DEEP; ++k) {
              if (k > 0 && kb + k >= end) break;
              const uint32_t st = st0 + k * P.block_bytes, sb = st + P.a_bytes;
              const int k0 = (kb + k) * kBK;
              if constexpr (MODE == kFwd) {
                load2d<CG>(st, ma, bar, k0, row0, pa);
                load2d<CG>(sb, mb, bar, k0, w.col, pb);    // (of a pair, the columns: 128 of the gate, 128 of up)
                if constexpr (CG == 1) load2d<CG>(sb + P.bn * 128, &P.b[1], bar, k0, w.col, pb);
              } else {
                if constexpr (MODE == kDx) {
                  load2d<CG>(st, ma, bar, k0, row0, pa);
                } else if (P.blocked) {
                  load3d<CG>(st, ma, bar, k0, row0 / 64, pa);
                } else {
                  load2d<CG>(st, ma, bar, row0, k0, pa);
                  load2d<CG>(st + 8192, ma, bar, row0 + 64, k0, pa);
                }
                if (P.blocked)
                  load3d<CG>(sb, mb, bar, k0, col0 / 64, pb);
                else
                  for (int j = 0; j < P.bn / CG / 64; ++j) load2d<CG>(sb + j * 8192, mb, bar, col0 + 64 * j, k0, pb);
              }
            }
          }
          __syncwarp();
        }
      }
    }
  given_up:
    // Nothing may reach this CTA's shared memory once it has gone: neither copies (those of both CTAs
    // report to the first one) nor the MMAs' last arrivals at `empty`, which come from the other CTA's
    // tensor core and which no later copy waits for. (A CTA of the next launch may take the place at once.)
    for (uint32_t s = 0; s < uint32_t(stages) && s < issued; ++s) {
      const uint32_t parity = ((issued - 1u - s) / stages) & 1u;       // of the stage's last use
      if (rank == 0) wait_drain(full(s), parity, ab, kSiteFfn + 3);
      if (!*ab.flag) wait_for(empty(s), parity, ab, kSiteFfn + 8);
    }
    if (*ab.flag)                                  // giving up: what is on its way lands long before this
      for (const uint64_t t0 = global_ns(); global_ns() - t0 < kDrainLimitNs;) {
      }
    __syncwarp();
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer
    if (rank == 0) {
      // K-major operands step 32 bytes inside the swizzle span per 16 of the reduction; MN-major
      // ones (64-column blocks 8 KB apart) step 16 rows of 128 bytes.
      constexpr uint32_t a_step = MODE == kDw ? 2048u : 32u, b_step = MODE == kFwd ? 32u : 2048u;
      const uint64_t a0 = smem_desc(base, MODE == kDw ? 8192u : 16u, 1024u, kLayoutSW128);
      const uint64_t b0 = smem_desc(base + P.a_bytes, MODE == kFwd ? 16u : 8192u, 1024u, kLayoutSW128);
      const bool one = elect_one();
      int idx = 0, buf = 0;
      uint32_t phase = 0, tphase = 0;
      bool ready = false, ok = true;                 // stage idx has landed; no wait has run out
      for (int u = first; u < P.total && ok; u += step) {
        const int bn = unit_at<MODE, CG>(P, u).bn;
        const uint32_t idesc = idesc_bf16(CG * kBM, MODE == kFwd ? 2 * bn : bn, MODE == kDw, MODE != kFwd);
        for (int i = 0; i < pieces; ++i) {
          const int blocks = blocks_of(i);
          if (empty_piece) break;
          ok = __all_sync(0xffffffffu, wait_for(tempty(buf), tphase ^ 1u, ab, kSiteFfn + 4));
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + buf * kAccCols;
          for (int kb = 0; kb < blocks; kb += DEEP) {
            ok = __all_sync(0xffffffffu, ready || wait_for(full(idx), phase, ab, kSiteFfn + 5));
            if (!ok) break;
            tc_fence_after();
            const uint32_t off0 = uint32_t(idx) * stage_bytes, used = empty(idx);
            if (++idx == stages) idx = 0, phase ^= 1u;
            ready = completed(full(idx), phase);
            if (one) {
#pragma unroll
              for (int k = 0; k < DEEP; ++k) {
                if (k > 0 && kb + k >= blocks) break;
                const uint32_t off = off0 + k * P.block_bytes;
#pragma unroll
                for (int j = 0; j < kBK / 16; ++j)
                  mma<CG>(d, desc_advance(a0, off + j * a_step), desc_advance(b0, off + j * b_step), idesc,
                          (kb | k | j) ? 1u : 0u);
              }
              commit<CG>(used);
              if (kb + DEEP >= blocks) commit<CG>(tfull(buf));
            }
            __syncwarp();
          }
          if (!ok) break;
          if (++buf == kAccs) buf = 0, tphase ^= 1u;
        }
      }
      if (one) commit_here<CG>(drain);
      __syncwarp();
      wait_drain(drain, 0u, ab, kSiteFfn + 6);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lanes = uint32_t(q * 32) << 16;
    int buf = 0;
    uint32_t tphase = 0, turn = 0;
    // accumulator `buf` is finished / has been read by this warp
    auto finished = [&]() {
      const bool ok = __all_sync(0xffffffffu, wait_for(tfull(buf), tphase, ab, kSiteFfn + 7));
      tc_fence_after();
      return ok;
    };
    auto leave = [&](bool ok) {
      tc_fence_before();
      __syncwarp();
      if (ok && lane == 0) {
        if constexpr (CG == 2) mbar_arrive_peer(peer_addr(tempty(buf), 0));
        else mbar_arrive(tempty(buf));
      }
      if (++buf == kAccs) buf = 0, tphase ^= 1u;
    };
    for (int u = first; u < P.total; u += step) {
      const Unit w = unit_at<MODE, CG>(P, u);
      const int64_t row0 = int64_t(w.tm * CG + rank) * kBM + q * 32, row = row0 + lane;
      const int end = min(P.n, w.col + w.bn);      // (bn need not be whole chunks)
      if constexpr (SPLIT == 8) {
        // Row r of a piece goes to CTA r / 16: [piece][row][column], rows 16 bytes apart from whole banks.
        const uint32_t pitch = P.bn * 4 + 16, parts = base + kRingBytes + kRingSlack - SPLIT * 16 * pitch;
        const bool ok = empty_piece || finished();
        for (int c = 32 * half; c < w.bn; c += 64) {
          uint32_t r[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) r[e] = 0u;          // a piece of no k-blocks
          if (ok && !empty_piece) {
            tmem_ld32(tmem + lanes + c, r);
            tmem_ld_wait();
            reg_fence(r);
          }
          if (ok && row < P.m) {
            const uint32_t at = peer_addr(parts + (peer * 16 + (lane & 15)) * pitch + c * 4, 2 * q + (lane >> 4));
#pragma unroll
            for (int j = 0; j < 8; ++j)
              asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + 16 * j), "r"(r[4 * j]),
                           "r"(r[4 * j + 1]), "r"(r[4 * j + 2]), "r"(r[4 * j + 3])
                           : "memory");
          }
        }
        tc_fence_before();
        __syncwarp();
        if (ok && (lane & 15) == 0) mbar_arrive_peer(peer_addr(sent, 2 * q + (lane >> 4)));
        if (!__all_sync(0xffffffffu, ok && wait_for(sent, 0u, ab, kSiteFfn + 9))) continue;
        const int col = w.col + 4 * lane;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int i = 2 * (warp - 2) + k;
          const int64_t r = int64_t(w.tm) * kBM + peer * 16 + i;
          if (r >= P.m || 4 * int(lane) >= w.bn || col >= end) continue;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int p = 0; p < SPLIT; ++p) {
            float v[4];
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                         : "r"(parts + (p * 16 + i) * pitch + 16 * lane)
                         : "memory");
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] = __fadd_rn(sum[e], v[e]);
          }
          *reinterpret_cast<uint2*>(P.out[0] + r * P.n + col) =
              make_uint2(bf16x2_bits(sum[0], sum[1]), bf16x2_bits(sum[2], sum[3]));
        }
        continue;
      } else if constexpr (MODE == kDx) {
        constexpr int kChunks = SPLIT ? 2 : 4;     // of 32 columns, of this warp: up to 128 (256) by two
        float sum[kChunks][32];
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
#pragma unroll
          for (int e = 0; e < 32; ++e) sum[i][e] = 0.f;
        bool ok = true;
        // the first product's sums in the second CTA: [4 columns][row]
        const uint32_t sums = base + kRingBytes + kRingSlack - P.bn * kBM * 4 + (q * 32 + lane) * 16;
        if (SPLIT && peer == 1) {
          ok = __all_sync(0xffffffffu, wait_for(sent, 0u, ab, kSiteFfn + 9));
#pragma unroll
          for (int i = 0; i < kChunks; ++i) {
            const int c = 32 * half + 64 * i;
            if (!ok || c >= w.bn) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                           : "=f"(sum[i][4 * j]), "=f"(sum[i][4 * j + 1]), "=f"(sum[i][4 * j + 2]), "=f"(sum[i][4 * j + 3])
                           : "r"(sums + (c / 4 + j) * kBM * 16)
                           : "memory");
          }
        }
        for (int p = 0; p < pieces; ++p) {
          ok = finished() && ok;
#pragma unroll
          for (int i = 0; i < kChunks; ++i) {
            const int c = 32 * half + 64 * i;
            if (!ok || c >= w.bn) continue;
            uint32_t r[32];
            tmem_ld32(tmem + buf * kAccCols + lanes + c, r);
            tmem_ld_wait();
            reg_fence(r);
#pragma unroll
            for (int e = 0; e < 32; ++e) sum[i][e] = __fadd_rn(sum[i][e], __uint_as_float(r[e]));
          }
          leave(ok);
        }
        if (SPLIT && peer == 0) {
#pragma unroll
          for (int i = 0; i < kChunks; ++i) {
            const int c = 32 * half + 64 * i;
            if (!ok || c >= w.bn) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                               peer_addr(sums + (c / 4 + j) * kBM * 16, 1)),
                           "f"(sum[i][4 * j]), "f"(sum[i][4 * j + 1]), "f"(sum[i][4 * j + 2]), "f"(sum[i][4 * j + 3])
                           : "memory");
          }
          __syncwarp();
          if (ok && lane == 0) mbar_arrive_peer(peer_addr(sent, 1));
          continue;
        }
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const int c = 32 * half + 64 * i, col = w.col + c;
          if (ok && c < w.bn && col < end) store_rows32(P.out[0], row0, P.m, P.n, col, end, sum[i], lane);
        }
        continue;
      }
      const bool ok = finished();
      const uint32_t acc = tmem + buf * kAccCols + lanes;
      if (ok) {
        if constexpr (MODE == kFwd) {
          for (int c = 32 * half; c < w.bn; c += 64) {
            const int col = w.col + c;
            if (col >= end) break;
            uint32_t r0[32];
            tmem_ld32(acc + c, r0);
            uint32_t r1[32];
            tmem_ld32(acc + w.bn + c, r1);
            tmem_ld_wait();
            reg_fence(r0);
            reg_fence(r1);
            float g[32], v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              g[i] = __uint_as_float(r0[i]);
              v[i] = __uint_as_float(r1[i]);
            }
            // (A lane reads its own row, 16 bytes at a time: four times the accesses of 64-byte pieces. Their
            // time does not hide under the MMAs: 4096 x 5120 x 17408 1110 us with deltas, 740 to 795 without.)
            if (P.delta[0] && row < P.m) {
              const float* dg = P.delta[0] + row * P.n + col;
              const float* du = P.delta[1] + row * P.n + col;
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (col + 4 * j < end) {
                  const float4 a = __ldcs(reinterpret_cast<const float4*>(dg) + j);
                  const float4 b = __ldcs(reinterpret_cast<const float4*>(du) + j);
                  g[4 * j] += a.x; g[4 * j + 1] += a.y; g[4 * j + 2] += a.z; g[4 * j + 3] += a.w;
                  v[4 * j] += b.x; v[4 * j + 1] += b.y; v[4 * j + 2] += b.z; v[4 * j + 3] += b.w;
                }
            }
            float h[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) h[i] = g[i] * act_p(P.act, g[i]) * v[i];
            store_rows32(P.out[0], row0, P.m, P.n, col, end, h, lane);
            if (P.keep_kind != LORA_KEEP_NONE) {
              keep_rows32(P, 0, row0, col, end, g, lane);
              keep_rows32(P, 1, row0, col, end, v, lane);
            }
          }
        } else {
          // By boxes of 32 rows x 32 columns through shared memory (rows of 64 bytes, 16-byte pieces permuted
          // by the row's bits 1 and 2), two of a warp on their way: where the reduction is short, the stores
          // are the tile's time (64 tokens 5120 x 17408: 100 us in 64-byte stores from registers, 94 so; boxes
          // of 64 columns 90, but the stage of the ring that they cost slows the longer reductions by 3 to 8 %).
          for (int c = 32 * half; c < w.bn; c += 64) {
            const int col = w.col + c;
            if (col >= end) break;
            uint32_t r[32];
            tmem_ld32(acc + c, r);
            tmem_ld_wait();
            reg_fence(r);
            const uint32_t box = base + kRingBytes + ((warp - 2) * 2 + turn) * kBoxBytes;
            turn ^= 1u;
            if (lane == 0) tma_store_wait_read<1>();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                v[e] = bf16x2_bits(__uint_as_float(r[8 * j + 2 * e]), __uint_as_float(r[8 * j + 2 * e + 1]));
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(box + lane * 64 + ((j ^ (lane >> 1 & 3)) << 4)),
                           "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                           : "memory");
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              if (row0 < P.m) tma_store(&P.o[w.prod], box, col, int(row0), policy_normal());
              tma_store_commit();
            }
          }
        }
      }
      leave(ok);
    }
    if (MODE == kDw && lane == 0) tma_store_wait_all<0>();
  }

  __syncwarp();
  tc_fence_before();
  if constexpr (kCluster > 1) cluster_sync_all();   // no CTA leaves while its peer may still signal it
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    acc_free<CG>(tmem);
  }
  __syncwarp();
  if constexpr (CG == 2) cluster_sync_all();       // nor before the peer has freed its half
}

}  // namespace mlp
