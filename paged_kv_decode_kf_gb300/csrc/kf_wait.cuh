// kf_wait.cuh -- how long a warp waits for another part of its CTA that may be busy with
// a whole unit of work, and how it learns earlier that another one gave up. Host code too
// (the tests count its polls).
#pragma once

#include <stdint.h>

namespace kf {

// A wait polls in slices and looks between them whether another role has given up: 4 ms
// a slice at the 3.75 us that a failed mbarrier.try_wait takes.
constexpr uint32_t kPollsASlice = 1u << 10;
// Slices until it gives up: 2^23 polls, 31 s. A unit takes 30-40 ns a key: 21 s for 2^29 keys,
// beyond which q, k, v and the output of one head of 64 exceed the GPU's memory. (A limit
// from the call's lengths, read at run time, cost 3-10 % of the kernels' time.)
constexpr int kWaitSlices = 1 << 13;

}  // namespace kf

// The body of a wait: true once `slice` is (what is waited for has come within a slice's
// polls), false once `stop` is (another role has given up) or after the last slice. A macro,
// because as a function of two lambdas the same loop cost the tree kernel up to 9 % (64
// requests of 16384 tokens, 16/8 heads of 64, from L2: 361 us -> 396).
#define KF_WAIT_IN_SLICES(slice, stop)             \
    for (int i = 0; i < kf::kWaitSlices; ++i) {    \
        if (slice) return true;                    \
        if (stop) return false;                    \
    }                                              \
    return false
