// Bounded mbarrier waits of the MXFP4 product kernels (the Newton-Schulz
// kernels have their own, and take the drains): a wait without
// progress for `limit_ns` sets the CTA's abort flag, records bit 0 of *err and
// gives up; the other roles of the CTA see the flag in their own waits.
//
// A role may have ended, all of its copies or products issued, before another
// gives up.  So what is in flight is waited for (drain_*) after the barrier
// that ends the roles, when the flag is final, and not by each role for itself.
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

// The copies of the last stages that this CTA issued land.  One thread calls it.
__device__ __forceinline__ void drain_stages(uint32_t full0, uint32_t n, uint32_t issued, volatile int* abort_flag, int* err) {
  for (uint32_t i = issued > n ? issued - n : 0; i < issued; ++i)
    bounded_wait_slow(full0 + i % n * 8, (i / n) & 1u, abort_flag, err, false, kWaitNs);
}

// The same on rank 0 of a pair, whose barriers count both ranks' copies,
// rank_bytes of each a stage; rank 0 expects both.  A stage that one rank
// issued and the other did not gets the missing bytes, or the missing
// expectation, so that its phase ends when what was issued has landed.  The
// ranks are at most n stages apart: both wait for the products of stage i - n
// before they issue stage i.
__device__ __forceinline__ void drain_pair_stages(uint32_t full0, uint32_t n, uint32_t mine, uint32_t peers, uint32_t rank_bytes,
                                                  volatile int* abort_flag, int* err) {
  const uint32_t most = mine > peers ? mine : peers;
  for (uint32_t i = most > n ? most - n : 0; i < most; ++i) {
    const uint32_t bar = full0 + i % n * 8;
    if (i >= peers) ptx::mbar_complete_tx(bar, rank_bytes);
    else if (i >= mine) ptx::mbar_expect_tx(bar, rank_bytes);
    bounded_wait_slow(bar, (i / n) & 1u, abort_flag, err, false, kWaitNs);
  }
}

}  // namespace dmuon
