// The copies of a ring of stages whose arrival a barrier for each stage tells.  Plain
// arithmetic on what a warp knows, in its registers; no CUDA in it, so that a test on the
// host can run out a wait.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define DA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define DA_HOST_DEVICE inline
#endif

namespace da {

// Bits of stages.  A copy is out from when it is sent until a wait has seen it arrive: one
// whose wait ran out is still on its way, and drain() waits for it again, so that none writes
// to shared memory that the block no longer has.
struct Copies {
  uint32_t out = 0;    // on their way
  uint32_t phase = 0;  // parity of each stage's barrier that the copy completes
  bool lost = false;   // a wait ran out: no copy is sent or waited for any more, but by drain()

  DA_HOST_DEVICE void sent(int stage) { out |= 1u << stage; }

  // arrived(stage, parity): waits; false if that ran out.
  template <typename F>
  DA_HOST_DEVICE void wait(int stage, F arrived) {
    if (!(out >> stage & 1) || lost) return;
    if (!arrived(stage, phase >> stage & 1)) {
      lost = true;
      return;
    }
    out ^= 1u << stage;
    phase ^= 1u << stage;
  }

  template <typename F>
  DA_HOST_DEVICE void drain(int stages, F arrived) {
    for (int stage = 0; stage < stages; ++stage)
      if (out >> stage & 1) arrived(stage, phase >> stage & 1);
  }
};

}  // namespace da
