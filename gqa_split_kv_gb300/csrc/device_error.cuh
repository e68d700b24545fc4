// The device error word and the bounded wait that sets it.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"

namespace da {

// Device error word (bit 0: a bounded wait ran out; bit 1: a segment counter
// update gave up; bit 2: a page-table entry outside [0, num_pages); bit 3: a token
// at or past the cache's capacity was not written).  Each translation unit has its
// own; decode_device_error() reads and clears them all, through take_error_word of
// each unit.
static __device__ unsigned int g_error_word = 0;

// Bounded mbarrier wait.  Gives up after timeout_ns: sets the device error word
// and the CTA's abort flag, after which every later wait returns at once, so
// all warps still reach the same named barriers and the CTA exits.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                             unsigned long long timeout_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  if (*abort_flag) return false;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > timeout_ns) {
      atomicOr(&g_error_word, 1u);
      *abort_flag = 1;
      return false;
    }
  }
}

// Reads and clears this unit's word of the current device (or-ed into *flags); the
// stream's work must be done.
static int take_unit_error_word(unsigned int* flags) {
  unsigned int w = 0;
  if (cudaMemcpyFromSymbol(&w, g_error_word, sizeof(w)) != cudaSuccess) {
    cudaGetLastError();
    return 1;
  }
  if (w) {
    const unsigned int zero = 0;
    if (cudaMemcpyToSymbol(g_error_word, &zero, sizeof(zero)) != cudaSuccess) {
      cudaGetLastError();
      return 1;
    }
  }
  *flags |= w;
  return 0;
}

// The words of the other units (each defined in its unit).
int take_cache_error_word(unsigned int* flags);
int take_latent_error_word(unsigned int* flags);

}  // namespace da
