// What the warp-specialised kernels over the paged KV cache share: bounded waits and the exponential.
#pragma once
#include "kv_cache.cuh"
#include "ptx.cuh"

namespace hstu {

// Waits for a phase of a barrier. After timeout_ns the CTA's abort flag is set and HSTU_DEVERR_TIMEOUT
// reported; false then, and wherever the flag is found set: the role leaves its loop. (Bars: a block of
// barriers with that flag, `volatile int abort`.)
template <class Bars>
__device__ __forceinline__ bool wait_bar(const SoftmaxParams& p, Bars* bars, uint64_t* bar,
                                         uint32_t parity) {
  const uint32_t a = ptx::smem_u32(bar);
  if (ptx::mbar_try_wait(a, parity)) return true;
  const uint64_t start = ptx::globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (ptx::mbar_try_wait(a, parity)) return true;
    if ((i & 15u) == 0) {
      if (bars->abort) return false;
      if ((long long)(ptx::globaltimer_ns() - start) > p.timeout_ns) {
        bars->abort = 1;
        report(p.c, HSTU_DEVERR_TIMEOUT);
        return false;
      }
    }
  }
}

// The same by every lane of a warp, with a warp-uniform result (the tcgen05 loads and stores
// that follow are executed by whole warps).
template <class Bars>
__device__ __forceinline__ bool warp_wait(const SoftmaxParams& p, Bars* bars, uint64_t* bar,
                                          uint32_t parity) {
  return __all_sync(0xffffffffu, wait_bar(p, bars, bar, parity));
}

// 2^x; a subnormal result is 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace hstu
