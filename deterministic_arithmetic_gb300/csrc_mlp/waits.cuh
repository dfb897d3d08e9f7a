// waits.cuh -- the bounded waits of the tensor-core kernels of the MLP-block operators.
#pragma once

#include "../csrc/common.cuh"

namespace mlp {

// Whether the phase of `bar` with that parity has completed, at once (mbarrier.try_wait, which the
// delta's waits begin with, may hold the thread for a while).
__device__ __forceinline__ bool completed(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0u;
}

// Wait for that phase (completed by this CTA, its copies and tensor core, or a peer of its cluster), for
// at most the abort state's limit. False: the CTA is giving up, because this wait ran out (its site is
// recorded) or another one did. A CTA that gives up passes its remaining waits at once: a long
// reduction has thousands of them.
static __device__ __noinline__ bool wait_longer(uint32_t bar, uint32_t parity, lora::Abort ab, uint32_t site) {
  const uint64_t t0 = lora::global_ns();
  while (true) {
    if (*ab.flag) return false;
    if (lora::mbar_test_cluster(bar, parity)) return true;
    if (lora::global_ns() - t0 > ab.limit_ns) {
      *ab.flag = 1u;
      if (ab.status) atomicCAS(ab.status, 0u, (site << 8) | lora::kDevTimeout);   // the first code stays
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, lora::Abort ab, uint32_t site) {
  return completed(bar, parity) || wait_longer(bar, parity, ab, site);
}

}  // namespace mlp
