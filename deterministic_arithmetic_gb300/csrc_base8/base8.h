// base8.h -- internal interface of the operators of include/lora_base8.h.
#pragma once

#include "../../include/lora_base8.h"
#include "../csrc_mlp/mlp.h"

namespace mlp {

constexpr uint32_t kKindLinear = 24, kSiteLinear = 96;   // status block: kind kKindLinear + pass, sites from kSiteLinear

// Raise the shared-memory limits of the kernels (on device dev, the current one), and find how many pairs of the products'
// CTAs it holds: with the other operators' prepare calls.
cudaError_t prepare_linear(int dev);
cudaError_t prepare_distill();

inline int64_t blocks128(int64_t n) { return cdiv(n, 128); }

}  // namespace mlp
