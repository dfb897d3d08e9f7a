// linear.h -- arguments of the tensor-core kernel of the products with 8-bit weights.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "base8.h"

namespace mlp {

constexpr int kLinFwd = 0, kLinBwd = 1;

struct LinArgs {
  CUtensorMap a, b;                // codes of x (dy); of w
  CUtensorMap o, d;                // out, boxes of 32 rows x 64 bytes; delta's
  const float *sa, *sb;            // scales of x (dy) [m][nk]; of w
  int64_t sb_out, sb_red;          // strides of the weight's scales: an output's block, a block of the reduction
  const float* delta;              // [m][n], or null
  void* out;                       // [m][n]
  int boxes;                       // 256-column tiles: out (and delta) go by TMA, rows are whole 16 bytes
  int out_f32, vec;                // out's type; columns come in whole vectors of 4
  int m, n, nk;                    // rows, columns; 128-deep blocks of the reduction
  int bn;                          // tile columns
  int stages, block_bytes, a_bytes;   // of the ring; of a k-block (all of it copied); of it A's rows
  int tiles_m, tiles_n;
  int total;                       // tiles
};

}  // namespace mlp
