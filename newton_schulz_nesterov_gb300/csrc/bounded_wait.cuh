// Bounded mbarrier waits of the MXFP4 product kernels: a wait without
// progress for `limit_ns` sets the CTA's abort flag, records bit 0 of *err and
// gives up; the other roles of the CTA see the flag in their own waits.
#pragma once

#include "ptx.cuh"

namespace dmuon {

constexpr uint64_t kWaitNs = 4000000000ull;  // default limit: 4 s

__device__ __noinline__ static bool bounded_wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err,
                                                      bool honour_abort, uint64_t limit_ns) {
  const uint64_t t0 = ptx::globaltimer();
  while (true) {
    if (ptx::mbar_try(bar, parity)) return true;
    if (honour_abort && *abort_flag) return false;
    if (ptx::globaltimer() - t0 > limit_ns) {
      *abort_flag = 1;
      atomicOr(err, 1);
      return false;
    }
  }
}

__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err,
                                             uint64_t limit_ns) {
  if (ptx::mbar_try(bar, parity)) return true;
  return bounded_wait_slow(bar, parity, abort_flag, err, true, limit_ns);
}

// The same for a converged warp, every lane of which gets the same answer:
// what follows may need the whole warp (elect, tensor-memory loads and stores).
__device__ __noinline__ static bool bounded_wait_warp_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                                           int* err, uint64_t limit_ns) {
  const uint64_t t0 = ptx::globaltimer();
  while (true) {
    if (__all_sync(0xffffffffu, ptx::mbar_try(bar, parity))) return true;
    const bool late = ptx::globaltimer() - t0 > limit_ns;
    if (__any_sync(0xffffffffu, late)) {
      if ((threadIdx.x & 31) == 0) {
        *abort_flag = 1;
        atomicOr(err, 1);
      }
      return false;
    }
    if (__any_sync(0xffffffffu, *abort_flag)) return false;
  }
}

__device__ __forceinline__ bool bounded_wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err,
                                                  uint64_t limit_ns) {
  if (__all_sync(0xffffffffu, ptx::mbar_try(bar, parity))) return true;
  return bounded_wait_warp_slow(bar, parity, abort_flag, err, limit_ns);
}

}  // namespace dmuon
