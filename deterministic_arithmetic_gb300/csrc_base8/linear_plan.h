// linear_plan.h -- which way a product with 8-bit weights is taken. Host code without CUDA.
#pragma once

#include <algorithm>
#include <cstdint>

namespace mlp {

// CTAs of a tile's pair (2) or alone (1); columns of a tile, and of an accumulator; k-blocks of a stage.
struct LinPlan {
  int cg, bn, w, deep;
};

// The way whose rounds over all SMs (pairs) cost least. A lone CTA's k-block of w columns costs w + 64, a pair's of 256 columns
// 0.84 of a lone one's (its operands are read from shared memory half as often): fitted to 38 shapes of both passes from
// 1 x 4096 x 4096 to 4096 x 5120 x 1024 taken in each way. The way chosen is the fastest there or within 5 %, but for short
// reductions of many rows (4096 x 512 -> 512: 7.1 us, 6.0 in tiles of 256).
// wide: the kernels of 256 columns can run (linear.cu).
inline LinPlan lin_plan(bool bwd, int m, int n, int nsm, int pairs, bool wide) {
  const auto cdiv = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  static constexpr int widths[] = {256, 128, 96, 64, 48, 32};
  LinPlan plan{1, 256, 256, 1};
  int64_t best = INT64_MAX;
  if (wide && pairs > 0 && m > 128) best = cdiv(cdiv(m, 256) * cdiv(n, 256), pairs) * 26900, plan.cg = 2;
  for (int w : widths) {
    if (bwd && (w == 96 || w == 48)) continue;         // a copied piece is a whole swizzle span
    if (w == 256 && !wide) continue;
    const int64_t cost = cdiv(cdiv(m, 128) * cdiv(n, w), nsm) * (w + 64) * 100;
    if (cost < best) best = cost, plan = {1, w, w > 128 ? 256 : (w > 64 ? 128 : (w > 32 ? 64 : 32)), w > 128 ? 1 : (w > 64 ? 2 : 4)};
  }
  return plan;
}

}  // namespace mlp
