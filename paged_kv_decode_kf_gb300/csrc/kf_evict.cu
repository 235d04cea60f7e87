// kf_evict.cu -- eviction of the tokens with the least accumulated weight.
//
// Which tokens stay: of a request's L tokens the `keep` first in the order
// (protected, larger score, lower index). Protected are the first `sink` and
// the last `recent` positions of the sequence. Where they go: a kept token at an
// index below `keep` stays where it is; the i-th kept token at or above `keep`
// moves into the i-th evicted slot below it. No source is a destination, so the
// rows move in place in any order, and no row moves that need not.
//
// Selection: the rank order as an unsigned 32-bit key (protected = all ones; a
// float's bits with the sign folded; NaN = 0, below -inf; -0 = +0). The keep-th
// largest key comes from a radix search, 8 bits a pass, over a histogram in
// shared memory; keys equal to it stay in index order until `keep` are found.
// Then one pass in index order lists holes and movers with block-wide scans.
#include "kf_evict.cuh"

namespace kf {
namespace {

constexpr int kSelThreads = 1024;

struct Keys {
    const float *scores;
    const int32_t *positions;
    int64_t sink, recent_from;  // protected: position < sink or >= recent_from

    __device__ __forceinline__ uint32_t operator()(int64_t t) const {
        const int64_t pos = positions ? positions[t] : t;
        if (pos < sink || pos >= recent_from) return 0xffffffffu;
        const float s = scores[t];
        if (s != s) return 0u;
        const uint32_t u = __float_as_uint(s == 0.f ? 0.f : s);
        return (u >> 31) ? ~u : (u | 0x80000000u);
    }
};

// Exclusive prefix sum of `x` over the block, and the block's total.
__device__ __forceinline__ int block_scan(int x, int *warp_sums, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int v = x;
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    __syncthreads();  // warp_sums is free again
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int w = warp_sums[lane];
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    total = warp_sums[31];
    return v - x + (warp ? warp_sums[warp - 1] : 0);
}

__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(const EvictParams p) {
    __shared__ int hist[256];
    __shared__ int warp_sums[32];
    __shared__ uint32_t s_key;
    __shared__ int s_left;
    const int b = blockIdx.x, tid = threadIdx.x;
    int64_t L = p.ctx_lens[b];
    __syncthreads();  // every thread has read the length: ctx_out may be the same array
    const int64_t cap = (int64_t)p.bt_stride * p.block_size;
    if (L < 0 || L > cap) {
        if (tid == 0) raise_error(p.err, KF_DEVERR_CONTEXT_LEN);
        L = L < 0 ? 0 : cap;
    }
    if (L > p.max_context_len) {
        if (tid == 0) raise_error(p.err, KF_DEVERR_MAX_CONTEXT);
        L = p.max_context_len;
    }
    const float *scores = p.scores + b * p.score_stride;
    float *scores_out = p.scores_out + b * p.score_stride;
    const int32_t *positions = p.positions ? p.positions + b * p.score_stride : nullptr;
    int32_t *positions_out = p.positions_out ? p.positions_out + b * p.score_stride : nullptr;
    const int keep = p.keep;
    if (L <= keep) {
        for (int64_t t = tid; t < L; t += kSelThreads) {
            scores_out[t] = scores[t];
            if (positions) positions_out[t] = positions[t];
        }
        if (tid == 0) {
            p.counts[b] = 0;
            p.ctx_out[b] = (int32_t)L;
        }
        return;
    }
    Keys key{scores, positions, p.sink, (positions ? (int64_t)p.seq_lens[b] : L) - p.recent};

    // the keep-th largest key, from its highest byte down
    uint32_t prefix = 0;
    int left = keep;  // how many of the keys that share the prefix stay
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int64_t t = tid; t < L; t += kSelThreads) {
            const uint32_t k = key(t);
            if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
                atomicAdd(&hist[(k >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int n = left, d = 255;
            while (d > 0 && hist[d] < n) n -= hist[d--];
            s_key = prefix | ((uint32_t)d << shift);
            s_left = n;
        }
        __syncthreads();
        prefix = s_key;
        left = s_left;
        __syncthreads();
    }

    // in index order: which tokens stay, the holes below `keep` and the movers above it
    int *dst = p.dst + (int64_t)b * p.max_moves, *src = p.src + (int64_t)b * p.max_moves;
    int seen_eq = 0, holes = 0, movers = 0;
    for (int64_t t0 = 0; t0 < L; t0 += kSelThreads) {
        const int64_t t = t0 + tid;
        const uint32_t k = t < L ? key(t) : 0u;
        const bool eq = t < L && k == prefix;
        int total;
        const int rank = seen_eq + block_scan(eq, warp_sums, total);
        seen_eq += total;
        const bool kept = t < L && (k > prefix || (eq && rank < left));
        const bool hole = t < keep && !kept, mover = t >= keep && kept;
        // t < keep and t >= keep never mix in one thread: one scan of both counts, 16 bits each
        int both;
        const int at = block_scan((hole ? 1 : 0) + (mover ? 1 << 16 : 0), warp_sums, both);
        if (hole) dst[holes + (at & 0xffff)] = (int)t;
        if (mover) src[movers + (at >> 16)] = (int)t;
        holes += both & 0xffff;
        movers += both >> 16;
        if (t < keep && kept) {
            scores_out[t] = scores[t];
            if (positions) positions_out[t] = positions[t];
        }
    }
    __syncthreads();
    for (int i = tid; i < movers; i += kSelThreads) {
        scores_out[dst[i]] = scores[src[i]];
        if (positions) positions_out[dst[i]] = positions[src[i]];
    }
    if (tid == 0) {
        p.counts[b] = movers;
        p.ctx_out[b] = keep;
    }
}

// One warp a moved row.
__global__ void __launch_bounds__(256)
evict_move_kernel(const EvictParams p) {
    const int b = blockIdx.y, lane = threadIdx.x & 31;
    const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i >= p.counts[b]) return;
    int64_t row[2];
    const int tok[2] = {p.src[(int64_t)b * p.max_moves + i], p.dst[(int64_t)b * p.max_moves + i]};
    for (int k = 0; k < 2; ++k) {
        const int64_t phys = p.block_tables[(int64_t)b * p.bt_stride + tok[k] / p.block_size];
        if (phys < 0 || phys >= p.num_blocks) {
            if (lane == 0) raise_error(p.err, KF_DEVERR_BLOCK_ID);
            return;
        }
        row[k] = (phys * p.block_size + tok[k] % p.block_size) * p.row_vecs;
    }
    for (int v = lane; v < p.row_vecs; v += 32) {
        p.cache_a[row[1] + v] = p.cache_a[row[0] + v];
        if (p.cache_b) p.cache_b[row[1] + v] = p.cache_b[row[0] + v];
    }
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, int sm_count, cudaStream_t stream) {
    evict_select_kernel<<<p.batch, kSelThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.max_moves == 0) return e;
    evict_move_kernel<<<dim3((p.max_moves + 7) / 8, p.batch), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace kf
