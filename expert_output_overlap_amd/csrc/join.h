// Sums that the workgroups of one launch hand to the last of them.
#pragma once

#include "common.h"
#include "tile_util.h"

namespace {

// What a workgroup hands to another one inside the launch goes out with device-scope stores, which write through to the level that the
// XCDs share, and is read with device-scope loads, past the caches that may hold an older call's: no cache has to be written back
// or emptied (with such fences in every workgroup, the router's losses of 16384 x 256 logits by 256 of them took 65 us instead of 24)
template <class V>
__device__ __forceinline__ void hand_out(V* p, V v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class V>
__device__ __forceinline__ V take(const V* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Whether this workgroup, number id of n, is the last of them to come here; its own stores are complete then, and so are the
// others'.  The counters, 256 bytes apart, are 0 before and after.  Beyond JOIN_GROUP workgroups each group of them has a counter of its
// own and its last one goes on to the first: 2048 workgroups at one counter took 20 us.
constexpr uint32_t JOIN_GROUP = 32, JOIN_STRIDE = 64;
__host__ __device__ inline int64_t join_words(int64_t n) {
  return n <= 1 ? 0 : JOIN_STRIDE * (1 + (n <= JOIN_GROUP ? 0 : (n + JOIN_GROUP - 1) / JOIN_GROUP));
}
__device__ __forceinline__ bool last_of(uint32_t* counters, uint32_t id, uint32_t n, int* shared) {
  wait_stores();
  __syncthreads();
  if (n == 1) return true;
  if (threadIdx.x == 0) {
    bool last;
    if (n <= JOIN_GROUP) last = atomicInc(counters, n - 1) == n - 1;  // wraps to 0
    else {
      const uint32_t g = id / JOIN_GROUP, groups = (n + JOIN_GROUP - 1) / JOIN_GROUP, size = min(JOIN_GROUP, n - g * JOIN_GROUP);
      last = size == 1 || atomicInc(counters + (1 + g) * JOIN_STRIDE, size - 1) == size - 1;
      if (last) last = atomicInc(counters, groups - 1) == groups - 1;
    }
    *shared = last;
  }
  __syncthreads();
  return *shared != 0;
}

}  // namespace
