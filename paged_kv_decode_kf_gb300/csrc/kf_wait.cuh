// kf_wait.cuh -- how long a warp waits for another part of its CTA that may be busy with
// a whole unit of work, and how it learns earlier that another one gave up. Host code too
// (the tests count its polls).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define KF_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define KF_HOST_DEVICE inline
#endif

namespace kf {

// A wait polls in slices and looks between them whether another role has given up: 4 ms
// a slice at the 3.75 us that a failed mbarrier.try_wait takes.
constexpr uint32_t kPollsASlice = 1u << 10;
// Slices until it gives up: 2^23 polls, 31 s. A unit takes 30-40 ns a key: 21 s for 2^29 keys,
// beyond which q, k, v and the output of one head of 64 exceed the GPU's memory. (A limit
// from the call's lengths, read at run time, cost 3-10 % of the kernels' time.)
constexpr int kWaitSlices = 1 << 13;

// slice(): true if what is waited for has come within a slice's polls; stop(): true if
// another role has given up.
template <typename Slice, typename Stop>
KF_HOST_DEVICE bool wait_in_slices(const Slice &slice, const Stop &stop) {
    for (int i = 0; i < kWaitSlices; ++i) {
        if (slice()) return true;
        if (stop()) return false;
    }
    return false;
}

}  // namespace kf
