// asv_ring.h -- places in a ring of barriers (without CUDA, so that a host compiler takes it too).
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define ASV_HOST_DEVICE __host__ __device__
#else
#define ASV_HOST_DEVICE
#endif

namespace asv {

// Slot and phase of the next use of a ring of `n` barriers: `next` goes on by a use (or `by`), `back` undoes that.  Back
// from a ring's start are phases that a new barrier counts as complete.
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  ASV_HOST_DEVICE void next(int n, int by = 1) {
    slot += by;
    if (slot >= n) {
      slot -= n;
      phase ^= 1;
    }
  }
  ASV_HOST_DEVICE void back(int n, int by = 1) {
    slot -= by;
    if (slot < 0) {
      slot += n;
      phase ^= 1;
    }
  }
};

}  // namespace asv
