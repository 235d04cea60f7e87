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
// largest key comes from a radix search, 8 bits a pass, over histograms in shared
// memory (eight copies a bin, by lane: scores share their exponents, and one
// copy would serialise the atomics); keys equal to it stay in index order until
// `keep` are found. Two scans then place holes and movers in their lists.
//
// One cluster of CL CTAs a request, each with a contiguous part of its tokens,
// whose keys stay in shared memory from one global read on (up to 49152 a CTA;
// beyond, every pass computes them again). Histograms and counts meet through
// distributed shared memory, one cluster barrier a pass.
//
// What bounds it: 4 bytes a token to select (8 with positions), 2 row_bytes a moved
// row and cache (8 requests of 64K-128K tokens cut to 12289, 12 K rows of 2 x 2 KB
// moved at 6.9 TB/s: 102 us of 137). The selection is latency: a chain of four passes
// and two scans, 12 us for 2K tokens, 30 for 128K.
#include <algorithm>
#include <atomic>

#include "kf_evict.cuh"

namespace kf {
namespace {

constexpr int kSelThreads = 1024;

struct Keys {
    const float *scores;
    const int32_t *positions;
    int64_t sink, recent_from;  // protected: position < sink or >= recent_from

    __device__ __forceinline__ uint32_t operator()(int64_t t) const {
        return of(scores[t], positions ? positions[t] : t);
    }

    __device__ __forceinline__ static uint32_t rank_of(float s) {
        if (s != s) return 0u;
        const uint32_t u = __float_as_uint(s == 0.f ? 0.f : s);
        return (u >> 31) ? ~u : (u | 0x80000000u);
    }

    __device__ __forceinline__ uint32_t of(float s, int64_t pos) const {
        return pos < sink || pos >= recent_from ? 0xffffffffu : rank_of(s);
    }
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

template <int CL>
__device__ __forceinline__ void cluster_sync() {
    if (CL == 1) __syncthreads();
    else asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The int at `p` (shared memory) in CTA `rank` of the cluster.
template <int CL>
__device__ __forceinline__ int remote(const int *p, int rank) {
    if (CL == 1) return *p;
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), r;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(r) : "memory");
    return v;
}

// Exclusive prefix sum over the block's 32 warps of `x` (one value a warp).
__device__ __forceinline__ int warp_scan(int x, int *sums, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();  // `sums` is free again
    if (lane == 0) sums[warp] = x;
    __syncthreads();
    int all = sums[lane], before = lane < warp ? all : 0;
    for (int o = 16; o; o >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, o);
        before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    total = all;
    return before;
}

__device__ __forceinline__ void move_row(const EvictParams &p, int b, int src, int dst, int lane) {
    const int32_t *table = p.block_tables + (int64_t)b * p.bt_stride;
    const int64_t ps = table[src / p.block_size], pd = table[dst / p.block_size];
    if (ps < 0 || ps >= p.num_blocks || pd < 0 || pd >= p.num_blocks) {
        if (lane == 0) raise_error(p.err, KF_DEVERR_BLOCK_ID);
        return;
    }
    const int64_t from = (ps * p.block_size + src % p.block_size) * p.row_vecs;
    const int64_t to = (pd * p.block_size + dst % p.block_size) * p.row_vecs;
    // both caches' vectors in flight before the first store: 4 KB a warp
    for (int v0 = 0; v0 < p.row_vecs; v0 += 128) {
        uint4 x[2][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int v = v0 + 32 * i + lane;
            if (v < p.row_vecs) {
                x[0][i] = p.cache_a[from + v];
                if (p.cache_b) x[1][i] = p.cache_b[from + v];
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int v = v0 + 32 * i + lane;
            if (v < p.row_vecs) {
                p.cache_a[to + v] = x[0][i];
                if (p.cache_b) p.cache_b[to + v] = x[1][i];
            }
        }
    }
}

constexpr int kKeyCap = 49152;  // keys a CTA keeps in shared memory
constexpr int kCopies = 8;

// MOVE: the kernel moves the rows too (few of them; no second launch).
template <int CL, bool MOVE>
__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(const EvictParams p, int key_slots) {
    __shared__ int hist[256 * kCopies];
    __shared__ int sums[2][256];  // this CTA's histogram, double-buffered over passes
    __shared__ int warp_sums[64];
    __shared__ int s_digit, s_left;
    __shared__ int s_counts[2];   // this CTA's holes and movers
    __shared__ int s_before[3], all_bins[CL > 1 ? 256 : 1];
    extern __shared__ uint32_t keys[];
    const int b = blockIdx.x / CL, tid = threadIdx.x;
    const int rank = CL == 1 ? 0 : (int)cluster_rank();
    int64_t L64 = p.ctx_lens[b];
    cluster_sync<CL>();  // every thread has read the length: ctx_out may be the same array
    const int64_t cap = (int64_t)p.bt_stride * p.block_size;
    const bool report = rank == 0 && tid == 0;
    if (L64 < 0 || L64 > cap) {
        if (report) raise_error(p.err, KF_DEVERR_CONTEXT_LEN);
        L64 = L64 < 0 ? 0 : cap;
    }
    if (L64 > p.max_context_len) {
        if (report) raise_error(p.err, KF_DEVERR_MAX_CONTEXT);
        L64 = p.max_context_len;
    }
    const int L = (int)L64;
    const float *scores = p.scores + b * p.score_stride;
    float *scores_out = p.scores_out + b * p.score_stride;
    const int32_t *positions = p.positions ? p.positions + b * p.score_stride : nullptr;
    int32_t *positions_out = p.positions_out ? p.positions_out + b * p.score_stride : nullptr;
    const int keep = p.keep;
    const int per = (L + CL - 1) / CL;                 // this CTA's tokens: [lo, hi)
    const int lo = min(rank * per, L), hi = min(lo + per, L);
    const bool cached = per <= key_slots && L > keep;
    const Keys key{scores, positions, p.sink, (positions ? (int64_t)p.seq_lens[b] : (int64_t)L) - p.recent};
    // one read of scores and positions: below `keep` they keep their place (movers come
    // after), and the keys go to shared memory
    const int end = cached ? hi : min(hi, keep);
    for (int t0 = lo + tid; t0 < end; t0 += 4 * kSelThreads) {
        float sc[4];
        int32_t pos[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = t0 + i * kSelThreads;
            sc[i] = t < end ? scores[t] : 0.f;
            pos[i] = positions && t < end ? positions[t] : t;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = t0 + i * kSelThreads;
            if (t < min(end, keep)) {
                scores_out[t] = sc[i];
                if (positions) positions_out[t] = pos[i];
            }
            if (cached && t < end) keys[t - lo] = key.of(sc[i], pos[i]);
        }
    }
    if (L <= keep) {
        if (report) {
            p.counts[b] = 0;
            p.ctx_out[b] = L;
        }
        return;
    }
    auto key_at = [&](int t) { return cached ? keys[t - lo] : key(t); };

    // the keep-th largest key, from its highest byte down
    uint32_t prefix = 0;
    int left = keep;  // how many of the keys that share the prefix stay
    int eq_before = 0;
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        for (int i = tid; i < 256 * kCopies; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        for (int t = lo + tid; t < hi; t += kSelThreads) {
            const uint32_t k = key_at(t);
            if (pass == 0 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
                atomicAdd(&hist[((k >> shift) & 255) * kCopies + (tid & (kCopies - 1))], 1);
        }
        __syncthreads();
        int *mine = sums[pass & 1];
        if (tid < 256) {
            int n = 0;
#pragma unroll
            for (int i = 0; i < kCopies; ++i) n += hist[tid * kCopies + i];
            mine[tid] = n;
        }
        cluster_sync<CL>();
        const int *bins = mine;
        if (CL > 1) {  // a bin a thread, all ranks' loads in flight at once
            if (tid < 256) {
                int v[CL], n = 0;
#pragma unroll
                for (int r = 0; r < CL; ++r) v[r] = remote<CL>(&mine[tid], r);
#pragma unroll
                for (int r = 0; r < CL; ++r) n += v[r];
                all_bins[tid] = n;
            }
            __syncthreads();
            bins = all_bins;
        }
        // warp 0 finds the digit: lane l holds bins 255 - 8 l down to 248 - 8 l
        if (tid < 32) {
            int bin[8], n = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                bin[i] = bins[255 - 8 * tid - i];
                n += bin[i];
            }
            int above = n;  // inclusive sum from the largest digit down
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, above, o);
                if (tid >= o) above += y;
            }
            int at = above - n;
            if (at < left && left <= above) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (at < left && left <= at + bin[i]) {
                        s_digit = 255 - 8 * tid - i;
                        s_left = left - at;
                    }
                    at += bin[i];
                }
            }
        }
        __syncthreads();
        prefix |= (uint32_t)s_digit << shift;
        left = s_left;
    }
    // keys equal to the last kept one in the CTAs before this: lane r asks CTA r
    if (CL > 1) {
        if (tid < 32) {
            int n = tid < rank ? remote<CL>(&sums[1][prefix & 255], tid) : 0;
            for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
            if (tid == 0) s_before[2] = n;
        }
        __syncthreads();
        eq_before = s_before[2];
    }

    // which tokens stay: each warp takes a run of this CTA's tokens, 32 at a time in order
    const int lane = tid & 31, warp = tid >> 5;
    const int len = (((per + 31) / 32) + 31) & ~31;
    const int t0 = min(lo + warp * len, hi), t1 = min(t0 + len, hi);
    const uint32_t below = (1u << lane) - 1;
    int eq = 0;
    for (int t = t0 + lane; t - lane < t1; t += 32) eq += __popc(__ballot_sync(0xffffffffu, t < t1 && key_at(t) == prefix));
    int total;
    const int eq_rank = eq_before + warp_scan(eq, warp_sums, total);
    // fn(token, hole, mover) for each of the warp's tokens, whole warps at a time
    auto each = [&](auto &&fn) {
        int e = eq_rank;
        for (int t = t0 + lane; t - lane < t1; t += 32) {
            const uint32_t k = t < t1 ? key_at(t) : 0u;
            const bool same = t < t1 && k == prefix;
            const uint32_t m = __ballot_sync(0xffffffffu, same);
            const bool kept = t < t1 && (k > prefix || (same && e + __popc(m & below) < left));
            e += __popc(m);
            fn(t, t < t1 && t < keep && !kept, kept && t >= keep);
        }
    };
    int holes = 0, movers = 0;
    each([&](int t, bool hole, bool mover) {
        holes += __popc(__ballot_sync(0xffffffffu, hole));
        movers += __popc(__ballot_sync(0xffffffffu, mover));
    });
    int all_holes, all_movers;
    int hole_at = warp_scan(holes, warp_sums, all_holes), mover_at = warp_scan(movers, warp_sums + 32, all_movers);
    if (CL > 1) {
        if (tid == 0) {
            s_counts[0] = all_holes;
            s_counts[1] = all_movers;
        }
        cluster_sync<CL>();
        if (tid < 32) {
            const int h = tid < rank ? remote<CL>(&s_counts[0], tid) : 0;
            const int m = tid < CL ? remote<CL>(&s_counts[1], tid) : 0;
            int before[3] = {h, tid < rank ? m : 0, m};
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                for (int o = 16; o; o >>= 1) before[i] += __shfl_xor_sync(0xffffffffu, before[i], o);
                if (tid == 0) s_before[i] = before[i];
            }
        }
        __syncthreads();
        hole_at += s_before[0];
        mover_at += s_before[1];
        all_movers = s_before[2];
    }
    int *dst = p.dst + (int64_t)b * p.max_moves, *src = p.src + (int64_t)b * p.max_moves;
    each([&](int t, bool hole, bool mover) {
        const uint32_t h = __ballot_sync(0xffffffffu, hole), m = __ballot_sync(0xffffffffu, mover);
        if (hole) dst[hole_at + __popc(h & below)] = t;
        if (mover) src[mover_at + __popc(m & below)] = t;
        hole_at += __popc(h);
        mover_at += __popc(m);
    });
    if (report) {
        p.counts[b] = all_movers;
        p.ctx_out[b] = keep;
    }
    cluster_sync<CL>();  // lists complete; no CTA leaves while another reads its shared memory
    for (int i = rank * kSelThreads + tid; i < all_movers; i += CL * kSelThreads) {
        scores_out[dst[i]] = scores[src[i]];
        if (positions) positions_out[dst[i]] = positions[src[i]];
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (MOVE)
        for (int i = rank * (kSelThreads / 32) + (tid >> 5); i < all_movers; i += CL * (kSelThreads / 32))
            move_row(p, b, src[i], dst[i], tid & 31);
}

// One warp a moved row at a time. The grid is set up while the selection ends.
__global__ void __launch_bounds__(256)
evict_move_kernel(const EvictParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the lists are there
    const int b = blockIdx.y, n = p.counts[b];
    const int *src = p.src + (int64_t)b * p.max_moves, *dst = p.dst + (int64_t)b * p.max_moves;
    for (int i = blockIdx.x * 8 + (threadIdx.x >> 5); i < n; i += gridDim.x * 8)
        move_row(p, b, src[i], dst[i], threadIdx.x & 31);
}

template <int CL, bool MOVE>
cudaError_t launch_select(const EvictParams &p, cudaStream_t stream) {
    const int per = (p.max_context_len + CL - 1) / CL;
    const int slots = std::min(per, kKeyCap);
    const size_t smem = (size_t)slots * 4;
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done.load() & bit)) {
        e = cudaFuncSetAttribute(evict_select_kernel<CL, MOVE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kKeyCap * 4);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.batch * CL);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {CL, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = CL > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, evict_select_kernel<CL, MOVE>, p, slots);
}

template <bool MOVE>
cudaError_t launch_select(const EvictParams &p, int cl, cudaStream_t stream) {
    switch (cl) {
        case 1: return launch_select<1, MOVE>(p, stream);
        case 2: return launch_select<2, MOVE>(p, stream);
        case 4: return launch_select<4, MOVE>(p, stream);
        default: return launch_select<8, MOVE>(p, stream);
    }
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, int sm_count, cudaStream_t stream) {
    // A warp a row in the selecting CTA while it has one for each, else a launch of their
    // own (8 requests of 4K tokens, rows of 2 x 2 KB: 1 / 16 / 64 / 256 moves take 14.5 /
    // 16.5 / 19.9 / 34.9 us in the CTA, 16.5 / 18.3 / 18.2 / 18.6 in a launch).
    const bool in_place = p.max_moves <= 32;
    // CTAs a request: doubled while each has more than 6144 tokens, and the batch stays one
    // wave (4 requests of 4K / 8K / 32K tokens: 14.5 / 18.6 / 43.1 us with one CTA, 16.6 /
    // 16.5 / 20.6 with eight; 64 requests of 32K: 43.1 with one, 30.8 with two, 76 with eight).
    int cl = 1;
    while (cl < 8 && p.batch * cl * 2 <= sm_count && p.max_context_len > 6144 * cl) cl *= 2;
    const cudaError_t e = in_place ? launch_select<true>(p, cl, stream) : launch_select<false>(p, cl, stream);
    if (e != cudaSuccess || in_place) return e;
    // at most some 4800 CTAs over the batch (a CTA for every eight possible moves was
    // 10000 CTAs, most of them empty, where 33 requests moved 300 rows each)
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(std::min((p.max_moves + 7) / 8, std::max(1, 32 * sm_count / p.batch)), p.batch);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_move_kernel, p);
}

}  // namespace kf
