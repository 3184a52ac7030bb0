// Bounded waits of kernels whose warps have roles: the slow path is out of line
// and takes few arguments, since the roles' loops together have to stay small enough
// for the instruction cache.
#pragma once

#include "tc_common.cuh"

namespace dsi {
namespace {

__shared__ volatile int s_abort;               // a role has given up: the others follow
__shared__ int* s_err;                         // device status word

__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = tc::global_ns();
  for (uint32_t i = 1;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    if (ok) return true;
    if ((i & 255u) == 0) {
      if (s_abort) return false;
      if (tc::global_ns() - t0 > tc::kWaitLimitNs) {
        s_abort = 1;
        report(s_err, kErrTimeout);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait1(uint64_t* bar, uint32_t parity) {
  return tc::mbar_try_wait(bar, parity) || wait_on(tc::smem_u32(bar), parity);
}
// Whole warps: all lanes proceed or none.
__device__ __forceinline__ bool wait32(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait1(bar, parity));
}

}  // namespace
}  // namespace dsi
