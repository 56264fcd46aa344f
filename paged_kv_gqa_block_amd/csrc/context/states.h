// Partial states of splits that one launch writes and joins.
//
// They cross from one XCD's L2 to another's inside a launch: stores and loads
// at agent scope pass through both.
#pragma once

#include "device_common.h"

namespace pkv {

__device__ __forceinline__ void put_state(float* p, float x, float y) {
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p),
                     __builtin_bit_cast(uint64_t, make_float2(x, y)), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
// Four channels of chunk c of a head's D: two halves apart, so that the lanes of
// either store write without gaps.
template <int D>
__device__ __forceinline__ void put_state4(float* head, int c, const float4& o) {
  put_state(head + 2 * c, o.x, o.y);
  put_state(head + D / 2 + 2 * c, o.z, o.w);
}
__device__ __forceinline__ float2 get_state2(const float* p) {
  return __builtin_bit_cast(
      float2, __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED,
                                __HIP_MEMORY_SCOPE_AGENT));
}
template <int D>
__device__ __forceinline__ float4 get_state4(const float* head, int c) {
  const float2 a = get_state2(head + 2 * c), b = get_state2(head + D / 2 + 2 * c);
  return make_float4(a.x, a.y, b.x, b.y);
}

// Arrival counter of pair k < 65536: the first 2048 lie on cache lines of their
// own, so that atomics of different pairs never share one (256 compute units are
// worth ranges for no more pairs than that).  (With 8 pairs of 32
// arrivals it makes no difference: the last arrival takes 2.1-2.4 us either way.)
__device__ __forceinline__ int32_t* arrival_counter(int32_t* arrivals, int64_t k) {
  return arrivals + ((k & 2047) << 5) + (k >> 11);
}

// Called by the whole workgroup after its stores of one split's state: true in
// the workgroup that is the last of `ns` to get here, in every thread.  The
// counter is zero again for the next call.
__device__ __forceinline__ bool last_to_arrive(int32_t* counter, int ns, bool* s_last) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this thread's state has reached memory
  __syncthreads();
  if (threadIdx.x == 0) {
    const bool last = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT) == ns - 1;
    if (last) __hip_atomic_store(counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *s_last = last;
  }
  __syncthreads();
  return *s_last;
}

}  // namespace pkv
