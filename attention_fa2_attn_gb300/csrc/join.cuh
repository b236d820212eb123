// join.cuh -- waits, votes and stores of the kernels that cut a row's keys over several CTAs. (How
// they join the partial results differs: tree.cu takes a lane's columns as one vector, prefix.cu as
// several. One text for both gave prefix attention other last bits and no time.)
#pragma once

#include "common.cuh"

namespace fa {

// Whether the phase is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// mbar_wait in a quarter of its code, for kernels with many kinds of work: what a CTA runs for
// the first time comes from L2, a microsecond or more for a few KB while that is busy.
__device__ __forceinline__ bool mbar_wait_lean(uint64_t* bar, uint32_t parity, uint64_t timeout_ns,
                                               const volatile int* abort = nullptr) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait(a, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  int i = 0;
#pragma unroll 1
  while (!mbar_try_wait(a, parity)) {
    if ((++i & 31) == 0 && ((abort && *abort) || globaltimer_ns() - t0 > timeout_ns)) return false;
  }
  return true;
}

// 32 bytes in one store: a warp whose threads each write a row of their own spends a
// wavefront per row and store, so half as many as with 16 bytes.
__device__ __forceinline__ void st32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Whether all `nthreads` threads at the barrier say yes; it is their barrier as well.
__device__ __forceinline__ bool vote_all(int id, int nthreads, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(nthreads), "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}

}  // namespace fa
