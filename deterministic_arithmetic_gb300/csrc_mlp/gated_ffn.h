// gated_ffn.h -- arguments of the gated feed-forward block's tensor-core kernel.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "ffn_plan.h"

namespace mlp {

constexpr uint32_t kKindFfn = 16, kSiteFfn = 64;   // status block: kind kKindFfn + product, sites from kSiteFfn

struct FfnArgs {
  CUtensorMap a[2], b[2];          // kFwd: x | Wg, Wu.  kDx: dG, dU | Wg, Wu.  kDw: dG, dU | x
  CUtensorMap o[2];                // kDw: of the outputs, boxes 32 rows x 32 columns
  __nv_bfloat16* out[2];           // [m][n]: h | dx | dWg, dWu
  const float* delta[2];           // kFwd: Dg, Du [m][n], or null
  void* keep[2];                   // kFwd: G and U, kept as keep_kind says
  uint8_t* keep_scales[2];
  int keep_kind, act;
  int m, n;                        // rows and columns of the outputs
  int nk;                          // 64-deep blocks of one product's reduction
  int piece, pieces;               // kDx: a product is taken in `pieces` of `piece` blocks (the last may be shorter)
  int bn;                          // tile columns (in kFwd of each projection)
  int blocked;                     // kDx, kDw: the maps whose rows lie along the reduction are block_map's
  int stages;                      // of the ring
  int block_bytes, a_bytes;        // of a k-block (all of it copied); of it A's rows
  int tiles_m, tiles_n;            // tiles of one product
  int whole, total;                // units of work: `whole` tiles, then halves of the remaining ones
};

}  // namespace mlp
