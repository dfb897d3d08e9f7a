// linear_plan.h -- which way a product with 8-bit weights is taken. Host code without CUDA.
#pragma once

#include <algorithm>
#include <cstdint>

namespace mlp {

// CTAs of a tile's pair (2) or alone (1); columns of a tile, and of an accumulator; k-blocks of a stage.
struct LinPlan {
  int cg, bn, w, deep;
};

// Pairs of CTAs, 256 x 256 tiles, where the output has more rows than one CTA's and they give every pair one. CTAs
// alone otherwise, in tiles narrow enough to occupy the SMs: the width whose rounds over all SMs cost least.
inline LinPlan lin_plan(bool bwd, int m, int n, int nsm, int pairs) {
  const auto cdiv = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  if (pairs > 0 && m > 128 && cdiv(m, 256) * cdiv(n, 256) >= pairs) return {2, 256, 256, 1};
  static constexpr int widths[] = {256, 128, 96, 64, 48, 32};
  LinPlan plan{1, 256, 256, 1};
  int64_t best = INT64_MAX;
  for (int w : widths) {
    if (bwd && (w == 96 || w == 48)) continue;         // a copied piece is a whole swizzle span
    const int64_t cost = cdiv(cdiv(m, 128) * cdiv(n, w), nsm) * (w + 64);
    if (cost < best) best = cost, plan = {1, w, w > 128 ? 256 : (w > 64 ? 128 : (w > 32 ? 64 : 32)), w > 128 ? 1 : (w > 64 ? 2 : 4)};
  }
  return plan;
}

}  // namespace mlp
