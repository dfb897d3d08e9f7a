// ffn_plan.h -- which way the gated feed-forward block's products are taken. Host code without CUDA.
#pragma once

#include <algorithm>
#include <cstdint>

namespace mlp {

constexpr int kFwd = 0, kDx = 1, kDw = 2;          // the kernel's products (gemm.cuh)
constexpr int kBM = 128, kBK = 64;                 // rows of A of a CTA's tile, and depth of a k-block

// SMs of a device, and how many pairs of CTAs, clusters of two and of eight it holds at once. Where it holds
// none of a kind (a part of a device may have no eight SMs that can form a cluster), that way is not taken.
struct FfnFit {
  int nsm = 0, pairs = 0, two = 0, eight = 0;
};
struct FfnPlan {
  int cg, split, bn;               // CTAs of a tile's pair (2) or alone (1); CTAs a tile's sums are split over (0: none); columns
};

// What a 64-deep block of a lone CTA's tile of w columns takes, and in a split of dx what a cluster takes
// besides its blocks (starting, filling its ring, joining the sums), in units of 0.5 to 0.8 ns, by the rows.
// Fitted to the times of 27 shapes of dx from 1 x 96 to 2048 x 8192, taken in each way: the way and width
// of least cost are the fastest there, or within 2 % of it.
inline int64_t block_cost(int mode, int w) { return mode == kFwd ? 2 * w + 64 : w + (mode == kDx ? 256 : 64); }
constexpr int kJoinTwo = 4000, kJoinEight = 10000, kJoinRow = 50;    // (a row of a tile, sent by all eight)

// Of a product's output [m][n] from nk k-blocks (dx: of each product, in pieces of `piece`).
//
// Pairs of CTAs where the output has more rows than one CTA's and the 256 x 256 tiles give every
// pair one. CTAs alone otherwise, in tiles narrow enough to occupy the SMs: the width whose rounds
// over all SMs cost least. For dx a cluster a tile where that costs less, a CTA a product or eight with
// a piece each (us a call, alone / two / eight: 1 x 11392 -> 96 78 / 31 / 12; 64 x 17408 -> 5120
// 116 / 83 / 91; 512 x 8192 -> 2048 67 / 60 / 93; 300 x 11008 -> 4096 98 / 133 / 148).
inline FfnPlan ffn_plan(int mode, int m, int n, int nk, int piece, bool whole_groups, const FfnFit& fit) {
  const auto cdiv = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  const int most = mode == kFwd ? 128 : 256;
  // narrower tiles go in steps of whole groups of 32 (packed values kept), 8 columns, or 64-column blocks
  const int step = mode != kFwd ? 64 : (whole_groups ? 32 : 8), least = mode == kFwd ? 32 : 64;
  const int64_t products = mode == kDw ? 2 : 1, rows = cdiv(m, kBM);
  if (fit.pairs > 0 && m > kBM && products * cdiv(m, 2 * kBM) * cdiv(n, most) >= fit.pairs) return {2, 0, most};
  const int64_t blocks = int64_t(mode == kDx ? 2 : 1) * nk;
  FfnPlan plan{1, 0, most};
  int64_t best = INT64_MAX;
  for (int w = most; w >= least; w -= step) {
    const int64_t cost = cdiv(products * rows * cdiv(n, w), fit.nsm) * blocks * block_cost(mode, w);
    if (cost < best) best = cost, plan = {1, 0, w};
  }
  for (int w = 128; mode == kDx && w >= 64; w -= 64) {
    const int64_t tiles = rows * cdiv(n, w), block = block_cost(mode, w);
    const int64_t two = fit.two < 1 ? INT64_MAX : cdiv(tiles, fit.two) * (nk * block + kJoinTwo);
    const int64_t eight =
        fit.eight < 1 ? INT64_MAX : cdiv(tiles, fit.eight) * (piece * block + kJoinEight + kJoinRow * std::min(m, kBM));
    if (two < best) best = two, plan = {1, 2, w};
    if (eight < best) best = eight, plan = {1, 8, w};
  }
  return plan;
}

}  // namespace mlp
