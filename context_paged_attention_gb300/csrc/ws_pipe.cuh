// Producer / consumer pieces of the warp-specialised kernels: mbarrier arrivals,
// 16-byte copies counted on an mbarrier, and bounded waits that an abort flag
// ends early.
#pragma once

#include "common.cuh"

namespace cpattn {

__device__ __forceinline__ void ws_arrive(uint32_t mbar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(mbar) : "memory");
}
// each lane arrives once when all of its earlier cp.async copies have landed
__device__ __forceinline__ void ws_cp_arrive(uint32_t mbar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(mbar) : "memory");
}
__device__ __forceinline__ void ws_cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
// 16 zero bytes through the same copy path (nothing is read)
__device__ __forceinline__ void ws_cp16_zero(uint32_t dst, const void* any_gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, 0;\n" ::"r"(dst), "l"(any_gmem) : "memory");
}
// bounded wait on a phase; gives up when the abort flag is raised
__device__ __forceinline__ bool ws_wait(uint32_t mbar, uint32_t parity, const volatile int* abort_flag) {
  for (uint32_t it = 0; it < (1u << 22); ++it) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(mbar), "r"(parity)
        : "memory");
    if (done) return true;
    if ((it & 63u) == 63u && *abort_flag) return false;
  }
  return false;
}

}  // namespace cpattn
