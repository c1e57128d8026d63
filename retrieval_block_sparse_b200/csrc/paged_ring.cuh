// A warp's own ring of bulk copies: each place has an mbarrier that one lane arms with the bytes on
// their way, and lanes copy straight from global memory.  No other warp takes part.
#pragma once

#include "decode_persist.cuh"

namespace rba {
namespace {

// Whether the barrier's phase is over, for the whole warp (shared-memory address).
__device__ __forceinline__ bool phase_over(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
      " vote.sync.all.pred p, p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}
// Arms the barrier with `bytes` where `arm`, and copies `bytes1` to dst where they are not 0
// (predicated: no branch).
__device__ __forceinline__ void arm_and_copy(uint32_t bar, int arm, uint32_t bytes, uint32_t dst,
                                             const void* src, uint32_t bytes1) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.s32 p, %0, 0;\n setp.ne.u32 q, %4, 0;\n"
      " @p mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%1], %2;\n"
      " @q cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%3], [%5], %4, [%1];\n}\n"
      :
      : "r"(arm), "r"(bar), "r"(bytes), "r"(dst), "r"(bytes1), "l"(src)
      : "memory");
}
// Waits, within a bound, for a phase: false when it ran out.
__device__ __forceinline__ bool await_phase(uint32_t bar, uint32_t parity) {
  if (phase_over(bar, parity)) return true;
  const unsigned long long t0 = now_ns();
  while (true) {
    if (phase_over(bar, parity)) return true;
    if (__shfl_sync(0xffffffffu, now_ns() - t0 > kTimeoutNs, 0)) return phase_over(bar, parity);
  }
}

}  // namespace
}  // namespace rba
