// pack8_da.cu -- the adapter gradients of a packed x: dA = du^T x, and the whole backward pass of the
// LoRA delta.
//
// dA[r][k] = sum_m du[m][r] x[m][k] from x's codes and scale bytes, with the sum's tree of the delta's own
// weight gradients: 16-row tensor-core leaves with a fresh accumulator each, added by the canonical
// pairwise tree in 256-row chunks, and the chunks' partials by the canonical tree (combine). The values
// the codes stand for are bf16 values, so the leaves are those of the unpacked x, bit for bit.
//
// Bound by HBM in principle (33 / 32 bytes an element of x and little else: 5.2 us at 8192 x 4096, rank 16);
// in practice by a unit's steps in turn. Of 19.8 us there, 12 are spent with the copies and launches alone
// (3.5 of it the combine launch, which reads the partials of every unit); the expansion of the codes, 2.5
// instructions each, adds 3, the MMAs 2. Work unit = (128 columns, 256 rows); a stage brings 64
// rows of codes (one box, 128-byte swizzle) and of du. Two warps expand a stage, a thread a row of 128
// codes, into two 64-column bf16 blocks in the layout a TMA copy of x would have left; four such teams
// work on the four stages of a unit at once (all eight warps on one stage at a time waited out every
// stage's latencies in turn: 25 us). The tensor core takes both operands transposed (M = 128 columns,
// N = padded rank, K = 16 rows). At 8192 x 4096, rank 16: 38 us for unpacking x and running the delta's
// own kernels on it, 19.8 us here with the combine launch (rank 32: 23, rank 64: 35).
//
// Warps: 0 copies, 1 issues the MMAs, 2..9 add the leaves, 10..17 expand.
#include "../csrc/common.cuh"
#include "../csrc/kernels.h"
#include "elems.cuh"
#include "mlp.h"
#include "waits.cuh"

namespace mlp {
namespace {

using namespace lora;

constexpr uint32_t kKindDa = 13, kSiteDa = 56;      // status block

struct DaArgs {
  CUtensorMap codes, du;            // boxes 64 rows x 128 codes; 64 rows x RP
  const uint8_t* scales;
  float* part;                      // [n_ch][rows][K]
  int M, K, G, rows;                // rows: of a partial that are written (the rank for a single chunk, else RP)
  int n_ct, total;
};

template <int RP>
struct DaCfg {
  static constexpr int kRows = 64, kCols = 128;                 // of a stage
  static constexpr int kCodeBytes = kRows * kCols, kDuBytes = kRows * RP * 2;
  static constexpr int kRawBytes = kCodeBytes + kDuBytes, kRaw = 8;
  static constexpr int kWideBytes = kRows * kCols * 2, kWide = 4;   // expanded: two [64 rows][64 columns] bf16 blocks
  static constexpr int kLeaves = kRows / 16, kGroupCols = kLeaves * RP, kAcc = 512 / kGroupCols;
  static constexpr int kEpi = 8, kTeam = 2, kXf = kTeam * kWide, kThreads = 32 * (2 + kEpi + kXf);
  static constexpr int kSteps = kWgradChunk / kRows;            // stages of a chunk; a team and a place for each
  static constexpr int kCPT = RP / 2;                           // accumulator columns of an epilogue thread
  static constexpr int kBars = 2 * kRaw + kWide + kAcc + 2;
  static constexpr size_t kSmem = size_t(kWide) * kWideBytes + size_t(kRaw) * kRawBytes + 1024 + kBars * 8 + 16;
  static_assert(kSteps == 4 && kWide == kSteps && kTeam * 32 == kRows && kRawBytes % 1024 == 0 && kSmem < 227 * 1024, "layout");
  static_assert(kAcc <= kRaw && kWide <= kRaw, "a stage's barrier is met by all before its next use");
};

// 4 codes of a group with step 2^(s - 127), 1 <= s <= 246, as 4 bf16 values. With b the code's byte,
// 128 + (b & 127) is a bf16 value (0x4300 plus the low bits), and code = that - 128, or - 256 for b >= 128:
// one fused multiply-add by the step, exact. -256 steps is -128 steps with the exponent one higher: bit 7
// of the byte added where the exponent's lowest bit is.
__device__ __forceinline__ uint2 expand4(uint32_t w, uint32_t step2, uint32_t minus128) {
  uint32_t h[2] = {__byte_perm(w, 0u, 0x4140), __byte_perm(w, 0u, 0x4342)};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t a = (h[i] & 0x007F007Fu) | 0x43004300u, c = minus128 + (h[i] & 0x00800080u);
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(h[i]) : "r"(a), "r"(step2), "r"(c));
  }
  return make_uint2(h[0], h[1]);
}
// The same for any s (255: NaN).
__device__ __forceinline__ uint2 expand4_any(uint32_t w, uint32_t s) {
  const float step = scale_step(s);
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = float(int8_t(w >> (8 * i))) * step;
  return make_uint2(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]));
}

template <int RP>
__global__ void __launch_bounds__(DaCfg<RP>::kThreads, 1) pack8_da_kernel(const __grid_constant__ DaArgs P, uint32_t* status) {
  using C = DaCfg<RP>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  constexpr uint32_t raw_off = C::kWide * C::kWideBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(gbase + raw_off + C::kRaw * C::kRawBytes);
  const uint32_t bar0 = smem_u32(bars);
  auto rfull = [&](int s) { return bar0 + 8u * s; };                                   // codes and du landed
  // A stage's MMAs are done: its places may be filled again and its leaves read. One barrier tells all
  // three (a commit each took the issuing warp longer than the MMAs).
  auto done = [&](int s) { return bar0 + 8u * (C::kRaw + s); };
  auto wfull = [&](int s) { return bar0 + 8u * (2 * C::kRaw + s); };                   // expanded
  auto tempty = [&](int g) { return bar0 + 8u * (2 * C::kRaw + C::kWide + g); };       // leaves read
  const uint32_t drain = bar0 + 8u * (C::kBars - 2), never = drain + 8u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kBars);
  volatile uint32_t* abort_flag = tmem_slot + 1;

  const uint32_t warp = warp_id(), lane = lane_id();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kRaw; ++s) mbar_init(rfull(s), 1), mbar_init(done(s), 1);
    for (int s = 0; s < C::kWide; ++s) mbar_init(wfull(s), C::kTeam);
    for (int g = 0; g < C::kAcc; ++g) mbar_init(tempty(g), C::kEpi);
    mbar_init(drain, 1);
    mbar_init(never, 1);
    *abort_flag = 0u;
    mbar_fence_init();
    prefetch_map(&P.codes);
    prefetch_map(&P.du);
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  grid_dependents_launch();
  const Abort ab = make_abort(abort_flag, status);
  // stages of the chunk ch
  auto steps_of = [&](int ch) { return (min(P.M - ch * kWgradChunk, kWgradChunk) + C::kRows - 1) / C::kRows; };

  if (warp == 0) {
    // -------------------------------------------------------------- copies
    // (the whole warp, one lane issuing: the addresses stay in uniform registers)
    const bool one = elect_one();
    if (stall_requested(status, kKindDa) && one) stall_wait(never, ab, kSiteDa);   // test hook: a wait that runs out
    __syncwarp();
    const uint64_t once = policy_evict_first(), keep = policy_evict_last();
    Ring r;
    uint32_t issued = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < P.total && ok; u += gridDim.x) {
      const int ct = u % P.n_ct, ch = u / P.n_ct, n = steps_of(ch);
      for (int i = 0; i < n; ++i) {
        ok = __all_sync(0xffffffffu, wait_for(done(r.idx), r.phase ^ 1u, ab, kSiteDa + 1));
        if (!ok) break;
        const uint32_t st = base + raw_off + r.idx * C::kRawBytes, bar = rfull(r.idx);
        const int m = ch * kWgradChunk + i * C::kRows;
        if (one) {
          mbar_expect_tx(bar, C::kRawBytes);
          tma_load(st, &P.codes, bar, ct * C::kCols, m, once);
          tma_load(st + C::kCodeBytes, &P.du, bar, 0, m, keep);
        }
        __syncwarp();
        ++issued;
        r.next<C::kRaw>();
      }
    }
    for (uint32_t s = 0; s < C::kRaw && s < issued; ++s)
      wait_drain(rfull(s), ((issued - 1u - s) / C::kRaw) & 1u, ab, kSiteDa + 2);
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    constexpr uint32_t idesc = idesc_bf16(128, RP, 1, 1);
    uint64_t xdesc[C::kLeaves], gdesc[C::kLeaves];
#pragma unroll
    for (int j = 0; j < C::kLeaves; ++j) {
      // x transposed: columns contiguous, 64-column blocks 8 KB apart, 8-row groups 1 KB apart
      xdesc[j] = smem_desc(base + j * 2048u, 8192u, 1024u, kLayoutSW128);
      // du rows [64][RP]: one swizzle span a row
      gdesc[j] = smem_desc(base + raw_off + C::kCodeBytes + j * 32u * RP, 16u * RP, 16u * RP, layout_for_span(RP * 2));
    }
    Ring r, g;
    uint32_t wphase = 0;                                // a bit a place
    for (int u = blockIdx.x; u < P.total; u += gridDim.x) {
      const int n = steps_of(u / P.n_ct);
      for (int i = 0; i < n; ++i) {
        // the stage's copies have landed when it has been expanded
        bool ok = wait_for(wfull(i), (wphase >> i) & 1u, ab, kSiteDa + 3);
        ok = __all_sync(0xffffffffu, ok && wait_for(tempty(g.idx), g.phase ^ 1u, ab, kSiteDa + 4));
        if (ok) {
          tc_fence_after();
          const uint32_t d = tmem + g.idx * C::kGroupCols;
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < C::kLeaves; ++j)
              mma_bf16(d + j * RP, desc_advance(xdesc[j], i * C::kWideBytes), desc_advance(gdesc[j], r.idx * C::kRawBytes),
                       idesc, 0u);
            mma_commit(done(r.idx));
          }
          __syncwarp();
        }
        wphase ^= 1u << i;
        r.next<C::kRaw>();
        g.next<C::kAcc>();
      }
    }
    if (elect_one()) mma_commit(drain);
    __syncwarp();
    wait_drain(drain, 0u, ab, kSiteDa + 5);
  } else if (warp < 2 + C::kEpi) {
    // ---------------------------------------------------- leaves to partials
    const int q = warp & 3, h = (warp - 2) >> 2;        // a quarter of the columns of x, a half of the rank
    const uint32_t tbase = tmem + (uint32_t(q * 32) << 16) + h * C::kCPT;
    Ring r, g;
    for (int u = blockIdx.x; u < P.total; u += gridDim.x) {
      const int ct = u % P.n_ct, ch = u / P.n_ct, n = steps_of(ch);
      float sum[C::kCPT], left[2][C::kCPT];
      bool all = true;
#pragma unroll
      for (int i = 0; i < C::kSteps; ++i) {
        if (i < n) {
          const bool ok = __all_sync(0xffffffffu, wait_for(done(r.idx), r.phase, ab, kSiteDa + 6));
          all = all && ok;
          tc_fence_after();
#pragma unroll
          for (int c0 = 0; c0 < C::kCPT; c0 += 8) {
            uint32_t v[C::kLeaves][8];
#pragma unroll
            for (int j = 0; j < C::kLeaves; ++j)
#pragma unroll
              for (int e = 0; e < 8; ++e) v[j][e] = 0u;
            if (ok) {
#pragma unroll
              for (int j = 0; j < C::kLeaves; ++j) tmem_ld8(tbase + g.idx * C::kGroupCols + j * RP + c0, v[j]);
              tmem_ld_wait();
            }
#pragma unroll
            for (int j = 0; j < C::kLeaves; ++j) reg_fence(v[j]);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              sum[c0 + e] = tree4(__uint_as_float(v[0][e]), __uint_as_float(v[1][e]), __uint_as_float(v[2][e]),
                                  __uint_as_float(v[3][e]));
          }
          tc_fence_before();
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(tempty(g.idx));
          r.next<C::kRaw>();
          g.next<C::kAcc>();
        } else {
#pragma unroll
          for (int c = 0; c < C::kCPT; ++c) sum[c] = 0.f;
        }
        // stages 0 + 1, 2 + 3, then the two (a stage past the chunk's end adds 0 to its left neighbour)
        if (i == 0 || i == 2) {
#pragma unroll
          for (int c = 0; c < C::kCPT; ++c) left[i / 2][c] = sum[c];
        } else {
#pragma unroll
          for (int c = 0; c < C::kCPT; ++c) sum[c] = __fadd_rn(left[i / 2][c], sum[c]);
          if (i == 1) {
#pragma unroll
            for (int c = 0; c < C::kCPT; ++c) left[0][c] = sum[c];
          } else {
#pragma unroll
            for (int c = 0; c < C::kCPT; ++c) sum[c] = __fadd_rn(left[0][c], sum[c]);
          }
        }
      }
      const int col = ct * C::kCols + q * 32 + lane;
      if (all && col < P.K) {
        float* dst = P.part + (size_t(ch) * P.rows + h * C::kCPT) * P.K + col;
#pragma unroll
        for (int c = 0; c < C::kCPT; ++c)
          if (h * C::kCPT + c < P.rows) dst[size_t(c) * P.K] = sum[c];
      }
    }
  } else {
    // -------------------------------------------------------------- expand
    // Team i expands stage i of every unit into place i; a thread a row of it. The 16-byte pieces of a
    // row are permuted by the row's lowest three bits, so eight neighbouring lanes meet all the banks.
    const int team = (warp - 2 - C::kEpi) / C::kTeam, row = (warp - 2 - C::kEpi) % C::kTeam * 32 + lane;
    const uint32_t sw = row & 7;
    uint8_t* out = gbase + team * C::kWideBytes + row * 128;
    auto scales_of = [&](int u, uint32_t (&s)[4]) {     // 127 (a step of 1, for codes that are 0) outside the tensor
      const int grp = u % P.n_ct * 4, m = u / P.n_ct * kWgradChunk + team * C::kRows + row;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        s[k] = u < P.total && m < P.M && grp + k < P.G ? uint32_t(__ldg(P.scales + size_t(m) * P.G + grp + k)) : 127u;
    };
    uint32_t stage = 0, before = ~0u;                   // stages of this CTA so far; the last one in this place
    uint32_t next[4];
    scales_of(blockIdx.x, next);
    for (int u = blockIdx.x; u < P.total; u += gridDim.x) {
      const int n = steps_of(u / P.n_ct);
      const uint32_t mine = stage + team;
      stage += n;
      uint32_t s[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] = next[k];
      scales_of(u + gridDim.x, next);                   // the next unit's, loaded under this one's work
      if (team >= n) continue;
      bool ok = wait_for(rfull(mine % C::kRaw), (mine / C::kRaw) & 1u, ab, kSiteDa + 7);
      ok = ok && (before == ~0u || wait_for(done(before % C::kRaw), (before / C::kRaw) & 1u, ab, kSiteDa + 8));
      ok = __all_sync(0xffffffffu, ok);
      before = mine;
      if (ok) {
        const uint8_t* in = gbase + raw_off + mine % C::kRaw * C::kRawBytes + row * 128;
#pragma unroll
        for (int k = 0; k < 4; ++k) {                   // a group of 32 codes: two pieces in, four out
          const uint4 c0 = *reinterpret_cast<const uint4*>(in + (((2 * k) ^ sw) << 4));
          const uint4 c1 = *reinterpret_cast<const uint4*>(in + (((2 * k + 1) ^ sw) << 4));
          const uint32_t word[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
          uint2 v[8];
          if (s[k] - 1u < 246u) {
            const uint32_t step2 = (s[k] << 7) * 0x00010001u, minus128 = (0x8000u | ((s[k] + 7u) << 7)) * 0x00010001u;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = expand4(word[j], step2, minus128);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = expand4_any(word[j], s[k]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(out + (k >> 1) * 8192 + ((((k & 1) * 4 + j) ^ sw) << 4)) =
                make_uint4(v[2 * j].x, v[2 * j].y, v[2 * j + 1].x, v[2 * j + 1].y);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(wfull(team));
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

bool shape_ok(int64_t M, int64_t K) { return size_ok(M) && size_ok(K) && K > 0 && K % 8 == 0; }
bool rank_ok(int64_t R) { return R >= 8 && R <= 64 && R % 8 == 0; }
int64_t chunks(int64_t M) { return cdiv(M, kWgradChunk); }

// The chunk partials of dA (none for a single chunk, which goes straight to da).
size_t part_bytes(int64_t M, int64_t K, int64_t R) {
  return chunks(M) > 1 ? round256(size_t(chunks(M)) * padded_rank(int(R)) * size_t(K) * 4) : 0;
}

template <int RP>
cudaError_t launch_da_as(const DaArgs& P, uint32_t* status, int nsm, cudaStream_t st) {
  return launch_pdl(pack8_da_kernel<RP>, dim3(unsigned(P.total < nsm ? P.total : nsm)), dim3(DaCfg<RP>::kThreads),
                    DaCfg<RP>::kSmem, st, P, status);
}

// dA into da by way of the partials (as part_bytes says).
lora_status run_da(const void* du, const void* codes, const void* scales, int64_t M, int64_t K, int64_t R, float* da,
                   float* part, uint32_t* status, int nsm, cudaStream_t st) {
  const int RP = padded_rank(int(R));
  const int64_t C = chunks(M), ld = kGroup * groups(K);
  DaArgs P{};
  if (!tensor_map(&P.codes, codes, Elem::u8, M, ld, ld, 128, 64, 128) ||
      !tensor_map(&P.du, du, Elem::bf16, M, R, R, RP, 64, RP * 2))
    return LORA_ERR_CUDA;
  P.scales = static_cast<const uint8_t*>(scales);
  P.part = C > 1 ? part : da;
  P.rows = C > 1 ? RP : int(R);
  P.M = int(M);
  P.K = int(K);
  P.G = int(groups(K));
  P.n_ct = int(cdiv(K, 128));
  if (P.n_ct * C >= int64_t(1) << 30) return LORA_ERR_SHAPE;
  P.total = int(P.n_ct * C);
  const cudaError_t e = RP == 16   ? launch_da_as<16>(P, status, nsm, st)
                        : RP == 32 ? launch_da_as<32>(P, status, nsm, st)
                                   : launch_da_as<64>(P, status, nsm, st);
  if (e != cudaSuccess) return LORA_ERR_CUDA;
  if (C == 1) return LORA_OK;
  CombineJobs jobs{};
  jobs.n = 1;
  jobs.j[0] = CombineJob{part, da, int(C), int(K), int(R), RP, 0};
  return launch_combine(jobs, st) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

// Workspace of the whole backward pass: lora_delta_bwd's control block, then the partials of dU, dB, dA.
struct BwdLayout {
  size_t du, db, da, bytes;
};
BwdLayout bwd_layout(int64_t M, int64_t K, int64_t N, int64_t R) {
  const int RP = padded_rank(int(R));
  BwdLayout l;
  l.du = LORA_DELTA_CONTROL_BYTES;
  l.db = l.du + round256(size_t(cdiv(N, du_slice(RP))) * size_t(M) * RP * 4);
  l.da = l.db + round256(size_t(chunks(M)) * RP * size_t(N) * 4);
  l.bytes = l.da + part_bytes(M, K, R);
  return l;
}

template <int RP>
cudaError_t prepare() {
  return cudaFuncSetAttribute(pack8_da_kernel<RP>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(DaCfg<RP>::kSmem));
}

}  // namespace

cudaError_t prepare_pack8_da() {
  cudaError_t e;
  if ((e = prepare_down()) != cudaSuccess || (e = prepare_up()) != cudaSuccess || (e = prepare_wgrad()) != cudaSuccess ||
      (e = prepare_dy()) != cudaSuccess || (e = prepare<16>()) != cudaSuccess || (e = prepare<32>()) != cudaSuccess)
    return e;
  return prepare<64>();
}

}  // namespace mlp

using namespace mlp;

extern "C" {

size_t lora_pack8_da_workspace_size(int64_t M, int64_t K, int64_t R) {
  return shape_ok(M, K) && rank_ok(R) ? part_bytes(M, K, R) + 256 : 0;
}

lora_status lora_pack8_da(const void* du, const void* codes, const void* scales, int64_t M, int64_t K, int64_t R,
                          float* da, void* workspace, size_t workspace_bytes, void* stream) {
  if (!shape_ok(M, K)) return LORA_ERR_SHAPE;
  if (!rank_ok(R)) return LORA_ERR_RANK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  lora_status s;
  int nsm = 0;
  if (M == 0) {                                     // a sum over no rows
    if ((s = check_ptrs(da)) != LORA_OK || (s = device_ready(&nsm)) != LORA_OK) return s;
    return cudaMemsetAsync(da, 0, size_t(R) * size_t(K) * 4, st) == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
  }
  if ((s = check_ptrs(du, codes, scales, da, workspace)) != LORA_OK) return s;
  if (workspace_bytes < lora_pack8_da_workspace_size(M, K, R)) return LORA_ERR_WORKSPACE;
  if ((s = device_ready(&nsm)) != LORA_OK) return s;
  return run_da(du, codes, scales, M, K, R, da, static_cast<float*>(workspace), status_block(), nsm, st);
}

size_t lora_delta_bwd_packed8_workspace_size(int64_t M, int64_t K, int64_t N, int64_t R) {
  return lora_delta_bwd_workspace_size(M, K, N, R) ? bwd_layout(M, K, N, R).bytes : 0;
}

lora_status lora_delta_bwd_packed8(const void* dy, const void* codes, const void* scales, const void* a, const void* b,
                                   const void* u, float alpha, int64_t M, int64_t K, int64_t N, int64_t R, float* dx,
                                   float* da, float* db, void* du, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  if (!rank_ok(R)) return shape_ok(M, K) && shape_ok(M, N) ? LORA_ERR_RANK : LORA_ERR_SHAPE;
  if (!shape_ok(M, K) || !shape_ok(M, N)) return LORA_ERR_SHAPE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  lora_status s;
  int nsm = 0;
  if (M == 0) {                                     // sums over no rows
    // (where there is no device there is no tensor to write either: the no-op of lora_delta_bwd)
    if ((s = check_ptrs(da, db)) != LORA_OK || !any_device()) return s;
    if ((s = device_ready(&nsm)) != LORA_OK) return s;
    // lora_delta_bwd does not look at the pointers of a call on no rows: what a caller of it got away with
    // becomes an error here and not a stray write
    if (!in_device_memory(da) || !in_device_memory(db)) return LORA_ERR_CUDA;
    return cudaMemsetAsync(da, 0, size_t(R) * size_t(K) * 4, st) == cudaSuccess &&
                   cudaMemsetAsync(db, 0, size_t(N) * size_t(R) * 4, st) == cudaSuccess
               ? LORA_OK
               : LORA_ERR_CUDA;
  }
  s = check_ptrs(dy, codes, scales, a, b, u, dx, da, db, du, workspace);
  if (s != LORA_OK) return s;
  const BwdLayout L = bwd_layout(M, K, N, R);
  if (workspace_bytes < L.bytes) return LORA_ERR_WORKSPACE;
  if ((s = device_ready(&nsm)) != LORA_OK) return s;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint32_t* status = reinterpret_cast<uint32_t*>(ws);
  float *du_part = reinterpret_cast<float*>(ws + L.du), *db_part = reinterpret_cast<float*>(ws + L.db);
  const int RP = padded_rank(int(R)), span = 2 * RP, m = int(M), n = int(N), k = int(K), C = int(chunks(M));
  auto grid = [&](int64_t units) { return int(units < nsm ? units : nsm); };
  // dU and dB partials: one pass over dy for ranks of up to 16, else a pass each
  if (RP == 16) {
    DyArgs y{};
    y.n = 1;
    DySite& d = y.s[0];
    if (!tensor_map(&d.dy, dy, Elem::bf16, M, N, N, 32, 128, 64) ||
        !tensor_map(&d.b, b, Elem::bf16, N, R, R, RP, 128, span) ||
        !tensor_map(&d.u, u, Elem::bf16, M, R, R, RP, 128, span))
      return LORA_ERR_CUDA;
    d.du_part = du_part;
    d.db_part = db_part;
    d.M = m;
    d.N = n;
    d.alpha = alpha;
    if (launch_dy(y, status, grid(cdiv(M, kDyChunk) * cdiv(N, kDySlice)), st) != cudaSuccess) return LORA_ERR_CUDA;
  } else {
    DownArgs down{};
    WgArgs wg{};
    down.n = wg.n = 1;
    DownSite& d = down.s[0];
    WgSite& w = wg.s[0];
    if (!tensor_map(&d.in, dy, Elem::bf16, M, N, N, 32, 128, 64) ||
        !tensor_map(&d.w, b, Elem::bf16, N, R, R, RP, 64, span) ||
        !tensor_map(&w.in, dy, Elem::bf16, M, N, N, 64, 64, 128) ||
        !tensor_map(&w.g, u, Elem::bf16, M, R, R, RP, 64, span))
      return LORA_ERR_CUDA;
    d.part = du_part;
    d.M = w.M = m;
    d.Kred = w.Cw = n;
    d.alpha = w.alpha = alpha;
    w.part = db_part;
    if (launch_down(RP, true, down, status, grid(down_units(M, N, RP)), st) != cudaSuccess ||
        launch_wgrad(RP, true, wg, status, grid(wgrad_units(M, N, RP)), st) != cudaSuccess)
      return LORA_ERR_CUDA;
  }
  // the rows of dU, and dB, from their partials
  RowsArgs rows{};
  rows.n = 1;
  rows.R = int(R);
  rows.RP = RP;
  rows.s[0] = RowsSite{du_part, static_cast<__nv_bfloat16*>(du), m, int(cdiv(N, du_slice(RP))), 0};
  CombineJobs jobs{};
  jobs.n = 1;
  jobs.j[0] = CombineJob{db_part, db, C, n, int(R), RP, 1};
  if (launch_rows(rows, &jobs, nsm, st) != cudaSuccess) return LORA_ERR_CUDA;
  // dX, then dA from the codes
  UpArgs up{};
  up.n = 1;
  up.R = int(R);
  UpSite& q = up.s[0];
  if (!tensor_map(&q.a, du, Elem::bf16, M, R, R, RP, 128, span) || !tensor_map(&q.b, a, Elem::bf16, R, K, K, 64, RP, 128) ||
      !tensor_map(&q.out, dx, Elem::f32, M, K, K, 32, 32, 128))
    return LORA_ERR_CUDA;
  q.M = m;
  q.Nout = k;
  q.alpha = 1.0f;
  if (launch_up(RP, true, false, up, status, grid(up_units(M, K, RP)), st) != cudaSuccess) return LORA_ERR_CUDA;
  return run_da(du, codes, scales, M, K, R, da, reinterpret_cast<float*>(ws + L.da), status, nsm, st);
}

}  // extern "C"
