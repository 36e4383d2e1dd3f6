// The check of a device batch by every CTA that works on it (internal to libmamba2). Included inside an anonymous
// namespace of each translation unit that uses it.
#pragma once

constexpr int kSeenWords = 1024;  // slots that a bitmap in shared memory holds: 32 times as many

// The status of a device batch, as launch_check_device_batch finds it: the count, then the slots' range, then
// whether two sequences share one. mine: the slot of sequence threadIdx.x. All threads of the CTA call it and get
// the same answer. A pool of more slots than the bitmap holds is compared pair by pair.
template <int kThreads>
__device__ __forceinline__ int check_batch(int num, int capacity, int num_slots, int mine) {
  __shared__ uint32_t seen[kSeenWords];
  if (num < 0 || num > capacity) return MAMBA2_ERR_INVALID_ARGUMENT;
  const int me = (int)threadIdx.x;
  const bool in = me < num, small = num_slots <= 32 * kSeenWords;
  int bad = in && (mine < 0 || mine >= num_slots) ? 1 : 0;
  if (small) {
    for (int w = me; w < (num_slots + 31) / 32; w += kThreads) seen[w] = 0u;
    __syncthreads();
    if (in && !bad) {
      const uint32_t bit = 1u << (mine & 31);
      if (atomicOr(&seen[mine >> 5], bit) & bit) bad = 2;
    }
  } else {
    seen[me] = (uint32_t)mine;
    __syncthreads();
    if (in)
      for (int j = 0; j < me; ++j)
        if (seen[j] == (uint32_t)mine) bad |= 2;
  }
  if (__syncthreads_or(bad & 1)) return MAMBA2_ERR_SLOT_OUT_OF_RANGE;
  return __syncthreads_or(bad) ? MAMBA2_ERR_SLOT_SHARED : MAMBA2_OK;
}
