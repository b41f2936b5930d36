// What the workgroups of one launch tell each other (device functions).
#pragma once

#include "loss_kernels.h"

namespace muon {

// Exchange between the workgroups of one launch.  What is exchanged goes
// through agent-scope atomics, which do not stay in the L2 of one of the eight
// XCDs; a workgroup waits for its stores to have arrived and then counts
// itself.  (A release at that point would write back the whole L2 for stores
// that nobody in the launch reads: with it, scoring 2044 x 151936 scores took 1109 us
// instead of 90.)
__device__ __forceinline__ void publish(uint64_t* to, uint64_t v) {
  __hip_atomic_store(to, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t published(const uint64_t* from) {
  return __hip_atomic_load(from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ unsigned count_one(uint64_t* at) {
  return __hip_atomic_fetch_add(reinterpret_cast<unsigned*>(at), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Whether all other workgroups of the launch have counted themselves; called by
// the thread that published.  kCountedTogether workgroups share a counter, and
// the last of them counts for all in the first: at one address 480 workgroups
// wait 5 us for each other, in this way 1.
__device__ __forceinline__ bool arrive_last(uint64_t* counters) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  const unsigned g = blockIdx.x / kCountedTogether, groups = (gridDim.x - 1) / kCountedTogether + 1;
  const unsigned in_group = min(gridDim.x - g * kCountedTogether, static_cast<unsigned>(kCountedTogether));
  uint64_t* mine = counters + (1 + g) * kCounterWords;
  bool last = count_one(mine) == in_group - 1;
  if (last) {
    *mine = 0;
    last = count_one(counters) == groups - 1;
    if (last) *counters = 0;
  }
  asm volatile("" ::: "memory");
  return last;
}

// Whether this workgroup is the last one of the launch to get here.
__device__ __forceinline__ bool last_to_arrive(uint64_t* counters) {
  __shared__ int last;
  if (threadIdx.x == 0) last = arrive_last(counters);
  __syncthreads();
  return last;
}

}  // namespace muon
