// kf_runs.cuh -- equal runs over a ragged batch.
//
// Requests cost different amounts of work. Laid end to end in request order their
// work is one list of T tiles, which is cut into equal runs, one a CTA (or warp).
// Lengths live on the device, so every CTA finds its place by itself: a prefix
// sum of the requests' costs over its threads.
#pragma once

#include "kf_internal.cuh"

namespace kf {

// The first tile of CTA i's run when T tiles are cut into min(ctas, T) equal runs
// (CTAs past the last run have none).
__device__ __forceinline__ int64_t cut_at(int i, int ctas, int64_t T) {
    const int64_t P = ctas < T ? ctas : T;
    return i < P ? i * T / P : T;
}

struct Place {
    int b;
    int64_t off;  // tiles into the request
};

// Where the batch's tile `slot = slot_of(T)` lies, and T; cost(b) is request b's
// tiles. All threads of the block (whole warps) call it; `sm` holds 36 int64. The
// place is unspecified where slot >= T.
template <typename C, typename F>
__device__ __forceinline__ int64_t locate(int batch, C cost, int64_t *sm, F slot_of, Place &place, int64_t &slot) {
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
    const int per = (batch + nt - 1) / nt;
    const int b0 = min(tid * per, batch), b1 = min(b0 + per, batch);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += cost(b);
    int64_t v = mine;
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    if (lane == 31) sm[warp] = v;
    __syncthreads();
    int64_t before = v - mine, total = 0;
    for (int w = 0; w < nt / 32; ++w) {
        if (w < warp) before += sm[w];
        total += sm[w];
    }
    slot = slot_of(total);
    if (slot >= before && slot < before + mine) {
        int64_t at = before;
        for (int b = b0; b < b1; ++b) {
            const int64_t n = cost(b);
            if (slot < at + n) {
                sm[34] = b;
                sm[35] = slot - at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    place.b = (int)sm[34];
    place.off = sm[35];
    return total;
}

}  // namespace kf
