// kf_tables.cu -- blocks from a pool on the GPU into block tables, slots and positions
// of new rows, blocks back to the pool, and rows written by slot.
//
// extend: request b grows from L_b to L_b + n_b tokens and needs
//   need_b = ceil((L_b + n_b) / bs) - ceil(L_b / bs)
// blocks; with off_b the sum of need over the requests before it, its i-th new block is
// the pool's list[free - 1 - (off_b + i)]. A request grows if off_b + need_b <= free: the
// needs of all requests up to it count, so none behind the first that does not fit does.
// Rows belong to one request: a range that leaves the rows, or starts before the largest end
// of the ranges ahead of it that do not, is refused. That end, which only rises, is also
// what a row's request is searched by, so that a refused range hides no other's rows.
// release: the blocks behind ceil(target / bs), request by request in ascending order,
// go back so that entry j of `total` lands at list[free + total - 1 - j]: the exact
// opposite of an extend between the same lengths.
//
// Rows are the unit of work: a row finds its request and from off_b its block, and the
// row at a new block's first position (every new block has one) writes the table entry.
// So no CTA waits for another: each finds the ends and the needs of the whole batch by itself
// (three words a request, from L2), which replaces a launch between the sums and the rows:
// extend and release together 6.0 us for 64 requests of one row, 8.3 for 33 prompts of 33500
// rows. The last CTA to finish (a ticket in the pool's header) moves the pool's count and
// writes the lengths, which may overwrite those that the others read.
#include "kf_tables.cuh"

#include <algorithm>

#include "kf_mq_tc05.cuh"

namespace kf {
namespace {

constexpr int kThreads = 512;

struct Need {
    int64_t first, rows;  // the request's rows (0: a bad request, or none)
    int64_t len, held, blocks;
};

// Request b's rows [s, e); false where they leave the array's.
__device__ __forceinline__ bool rows_of(const PoolArgs &a, int b, int64_t &s, int64_t &e) {
    s = b;
    e = b + 1;
    if (a.row_start) {
        s = a.row_start[b];
        e = a.row_start[b + 1];
    }
    return s >= 0 && e >= s && e <= a.num_rows;
}

// `end`: the largest end of the rows of the requests before b; b's counts from here on.
__device__ __forceinline__ Need need_of(const PoolArgs &a, int b, bool report, int64_t &end) {
    Need n;
    int64_t s, e;
    const bool inside = rows_of(a, b, s, e), apart = inside && s >= end;
    if (inside && e > end) end = e;
    n.len = a.before[b];
    unsigned int bad = 0;
    if (!apart || n.len < 0) bad = KF_DEVERR_CONTEXT_LEN;
    else if (n.len + (e - s) > (int64_t)a.bt_stride * a.block_size) bad = KF_DEVERR_APPEND_POS;
    if (bad) {
        if (report) raise_error(a.err, bad);
        n.first = s;
        n.rows = n.held = n.blocks = 0;
        return n;
    }
    const int shift = block_shift(a.block_size);
    n.first = s;
    n.rows = e - s;
    n.held = (n.len + a.block_size - 1) >> shift;
    n.blocks = ((n.len + n.rows + a.block_size - 1) >> shift) - n.held;
    return n;
}

// Blocks a release takes from request b, from logical block `keep` on.
__device__ __forceinline__ int64_t freed_of(const PoolArgs &a, int b, bool report, int64_t &keep) {
    const int64_t len = a.before[b], target = a.target ? a.target[b] : 0;
    if (len < 0 || target < 0 || target > len || len > (int64_t)a.bt_stride * a.block_size) {
        if (report) raise_error(a.err, KF_DEVERR_CONTEXT_LEN);
        keep = 0;
        return 0;
    }
    const int shift = block_shift(a.block_size);
    keep = (target + a.block_size - 1) >> shift;
    return ((len + a.block_size - 1) >> shift) - keep;
}

// The sum of every thread's `mine` over the threads before it; `total` of all. `any`: whether
// it is true in some thread.
__device__ __forceinline__ int64_t scan_before(int64_t mine, int64_t *sm_warp, int64_t &total, bool &any) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t v = mine;
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    if (lane == 31) sm_warp[warp] = v;
    any = __syncthreads_or(any);
    int64_t before = v - mine;
    total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += sm_warp[w];
        total += sm_warp[w];
    }
    return before;
}

// The largest of `mine` (none below 0) over the threads before this one.
__device__ __forceinline__ int64_t max_before(int64_t mine, int64_t *sm_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t v = mine;
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v = max(v, y);
    }
    if (lane == 31) sm_warp[warp] = v;
    v = __shfl_up_sync(0xffffffffu, v, 1);
    if (lane == 0) v = 0;
    __syncthreads();
    for (int w = 0; w < warp; ++w) v = max(v, sm_warp[w]);
    return v;
}

// The free count, inside the list whatever the word holds.
__device__ __forceinline__ int64_t free_of(const PoolArgs &a, bool report) {
    const int64_t f = *(volatile int32_t *)a.pool;
    if (f < 0 || f > a.num_blocks) {
        if (report) raise_error(a.err, KF_DEVERR_POOL);
        return f < 0 ? 0 : a.num_blocks;
    }
    return f;
}

// True in the CTA that finishes last: all others have read what they need of the pool's
// count and of the lengths.
__device__ __forceinline__ bool last_cta(int32_t *pool, int *sm_last) {
    __syncthreads();  // (a single CTA's slower warps still read lengths that the others would write)
    if (gridDim.x == 1) return true;
    if (threadIdx.x == 0) {
        __threadfence();
        *sm_last = atomicAdd(reinterpret_cast<unsigned int *>(pool + 1), 1u) == gridDim.x - 1;
    }
    __syncthreads();
    return *sm_last;
}

__global__ void __launch_bounds__(kThreads)
extend_kernel(const PoolArgs a) {
    __shared__ int64_t sm_warp[kThreads / 32], sm_warp_end[kThreads / 32];
    // Of a thread's first request: the blocks before it, and the largest end of the rows before it.
    __shared__ int64_t sm_off[kThreads], sm_end[kThreads];
    __shared__ unsigned long long sm_taken;
    __shared__ int sm_last;
    const int tid = threadIdx.x;
    const int per = (a.batch + kThreads - 1) / kThreads;  // requests a thread
    const int chunks = (a.batch + per - 1) / per;
    const int b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
    const int64_t free = free_of(a, blockIdx.x == 0 && tid == 0);
    // Where no range leaves the rows they ascend, and a request's start is the largest end ahead of it.
    int64_t ahead = 0, mine = 0, total, s, e;
    bool bad = false;
    if (b0 < b1) rows_of(a, b0, ahead, e);
    int64_t end = ahead;
    for (int b = b0; b < b1; ++b) {
        bad = bad || !rows_of(a, b, s, e);
        mine += need_of(a, b, false, end).blocks;
    }
    sm_off[tid] = scan_before(mine, sm_warp, total, bad);
    if (bad) {  // (in all threads) else it has to be found
        int64_t last = 0;
        for (int b = b0; b < b1; ++b)
            if (rows_of(a, b, s, e)) last = max(last, e);
        ahead = end = max_before(last, sm_warp_end);
        mine = 0;
        for (int b = b0; b < b1; ++b) mine += need_of(a, b, false, end).blocks;
        sm_off[tid] = scan_before(mine, sm_warp, total, bad);
    }
    sm_end[tid] = ahead;
    if (tid == 0) sm_taken = 0;
    __syncthreads();

    const int32_t *list = a.pool + KF_POOL_HEADER;
    const int shift = block_shift(a.block_size);
    for (int64_t r = (int64_t)blockIdx.x * kThreads + tid; r < a.num_rows; r += (int64_t)gridDim.x * kThreads) {
        int lo = 0, hi = chunks;  // the last chunk that no rows behind r come ahead of
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sm_end[mid] <= r) lo = mid;
            else hi = mid;
        }
        int64_t off = sm_off[lo];
        end = sm_end[lo];
        int64_t slot = -1, pos = -1;
        for (int b = lo * per; b < min(lo * per + per, a.batch); ++b) {
            const Need n = need_of(a, b, false, end);
            if (r >= n.first && r < n.first + n.rows) {
                if (off + n.blocks <= free) {
                    pos = n.len + (r - n.first);
                    const int64_t lb = pos >> shift;
                    int32_t *entry = a.block_tables + (int64_t)b * a.bt_stride + lb;
                    const int64_t phys = lb >= n.held ? list[free - 1 - (off + lb - n.held)] : *entry;
                    if (lb >= n.held && (pos & (a.block_size - 1)) == 0) *entry = (int32_t)phys;
                    if (phys < 0 || phys >= a.num_blocks) raise_error(a.err, KF_DEVERR_BLOCK_ID);
                    else slot = (phys << shift) + (pos & (a.block_size - 1));
                }
                break;
            }
            off += n.blocks;
        }
        a.slots[r] = slot;
        if (a.positions) a.positions[r] = (int32_t)pos;
    }

    if (!last_cta(a.pool, &sm_last)) return;
    int64_t off = sm_off[tid], taken = 0;
    bool short_of = false;
    end = ahead;
    for (int b = b0; b < b1; ++b) {
        const Need n = need_of(a, b, true, end);
        const bool fits = off + n.blocks <= free;
        off += n.blocks;
        if (fits) taken = off;
        short_of = short_of || !fits;
        a.after[b] = (int32_t)(fits ? n.len + n.rows : n.len);
    }
    if (short_of) raise_error(a.err, KF_DEVERR_POOL);
    if (taken > 0) atomicMax(&sm_taken, (unsigned long long)taken);
    __syncthreads();
    if (tid == 0) {
        a.pool[0] = (int32_t)(free - (int64_t)sm_taken);
        a.pool[1] = 0;
    }
}

__global__ void __launch_bounds__(kThreads)
release_kernel(const PoolArgs a) {
    __shared__ int64_t sm_warp[kThreads / 32];
    __shared__ int64_t sm_off[kThreads];
    __shared__ int sm_last;
    const int tid = threadIdx.x;
    const bool report = blockIdx.x == 0;
    const int per = (a.batch + kThreads - 1) / kThreads;
    const int chunks = (a.batch + per - 1) / per;
    const int b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
    const int64_t free = free_of(a, report && tid == 0);
    int64_t mine = 0, keep;
    for (int b = b0; b < b1; ++b) mine += freed_of(a, b, report, keep);
    int64_t total;
    bool none = false;
    sm_off[tid] = scan_before(mine, sm_warp, total, none);
    __syncthreads();
    const bool fits = free + total <= a.num_blocks;  // else some block is in the list already
    if (!fits && report && tid == 0) raise_error(a.err, KF_DEVERR_POOL);
    if (fits) {
        int32_t *list = a.pool + KF_POOL_HEADER;
        for (int64_t j = (int64_t)blockIdx.x * kThreads + tid; j < total; j += (int64_t)gridDim.x * kThreads) {
            int lo = 0, hi = chunks;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (sm_off[mid] <= j) lo = mid;
                else hi = mid;
            }
            int64_t off = sm_off[lo];
            for (int b = lo * per; b < min(lo * per + per, a.batch); ++b) {
                const int64_t n = freed_of(a, b, false, keep);
                if (j < off + n) {
                    int32_t *entry = a.block_tables + (int64_t)b * a.bt_stride + keep + (j - off);
                    int32_t phys = *entry;
                    if (phys < 0 || phys >= a.num_blocks) {
                        raise_error(a.err, KF_DEVERR_BLOCK_ID);
                        phys = -1;
                    }
                    list[free + total - 1 - j] = phys;
                    *entry = -1;
                    break;
                }
                off += n;
            }
        }
    }
    if (!last_cta(a.pool, &sm_last)) return;
    if (tid == 0) {
        a.pool[0] = (int32_t)(fits ? free + total : free);
        a.pool[1] = 0;
    }
}

__global__ void __launch_bounds__(256)
pool_init_kernel(int32_t *pool, int64_t num_blocks) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < KF_POOL_HEADER) pool[i] = i == 0 ? (int32_t)num_blocks : 0;
    if (i < num_blocks) pool[KF_POOL_HEADER + i] = (int32_t)(num_blocks - 1 - i);  // block 0 is taken first
}

// ---------------------------------------------------------------------------
// Rows by slot: a warp a row, K and V together, four 16-byte loads of each in flight a lane
// before the first store, and none of them behind the load of the slot. HBM bounds it: 37000 rows
// of 8 x 128 into E4M3 caches 40.1 us, 5.7 TB/s of reads and writes.
//
// E4M3: the code of x / s, eight numbers of a head at a time. The division itself costs more
// issue slots than HBM leaves (16 a number; 48.5 us), so the quotient is Markstein's (IBM
// Journal of Research and Development 34, 1990, 111-119): with y = 1 / s rounded, q = x y,
// r = x - q s, q' = q + r y. Its error ahead of the last rounding is below 2^-22 of a unit in the last place. A code can only differ from the
// exact division's if x / s is that near to half a unit beside a border M of two codes (16 <= M
// <= 31 and a whole number, scaled). With s = S / 2^k, 2^23 <= S < 2^24, x's eight bits make x
// 2^j - M S a whole number n, |n| within 2^-17 of S / 2^20, 8 <= n <= 16: so S = 2^20 n + t, |t| <= 8,
// and modulo 2^20 M t = -n or n, which only M = 16, S = 2^24 - 1 fulfils: a significand of all ones,
// which is divided, as are scales beyond 2^60 and their like.
// q is cut to 512, above the largest code, so that infinite quotients do not become NaN; and it
// is taken from -x, so that a zero keeps its sign.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float cut_to_512(float x) {  // with x's sign; NaN: -512 or 512
    float y;
    asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(512.f));
    return y;
}

__device__ __forceinline__ uint2 codes_of(uint4 x, float s) {
    const uint32_t bits = __float_as_uint(s);
    uint32_t w[4] = {x.x, x.y, x.z, x.w}, c[4];
    if (bits - (67u << 23) <= (120u << 23) && (~bits & 0x7fffff) != 0) {  // 2^-60 <= s <= 2^60
        const float y = -__frcp_rn(s);
        const float2 y2 = make_float2(y, y), s2 = make_float2(s, s), none = make_float2(-0.f, -0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t n = w[i] ^ 0x80008000u;
            const float2 nx = make_float2(bf16_lo(n), bf16_hi(n));
            float2 q = mq5::fma_f32x2(nx, y2, none);
            q.x = cut_to_512(q.x);
            q.y = cut_to_512(q.y);
            q = mq5::fma_f32x2(mq5::fma_f32x2(q, s2, nx), y2, q);
            c[i] = tc::f32x2_to_e4m3x2(q.x, q.y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = tc::f32x2_to_e4m3x2(__fdiv_rn(bf16_lo(w[i]), s), __fdiv_rn(bf16_hi(w[i]), s));
    }
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

template <bool FP8>
__global__ void __launch_bounds__(256)
append_rows_kernel(const RowsArgs a) {
    constexpr int kAtOnce = 4;
    const int lane = threadIdx.x & 31;
    const int vecs = a.num_kv_heads * a.head_dim / 8;  // 8 values a read vector
    const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (r >= a.num_rows) return;
    const int64_t slot = __ldg(a.slots + r);
    const uint4 *k = reinterpret_cast<const uint4 *>(a.k_rows) + r * vecs;
    const uint4 *v = reinterpret_cast<const uint4 *>(a.v_rows) + r * vecs;
    for (int i0 = lane; i0 < vecs; i0 += 32 * kAtOnce) {
        uint4 x[kAtOnce], y[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
            if (i0 + 32 * j < vecs) {
                x[j] = __ldg(k + i0 + 32 * j);
                y[j] = __ldg(v + i0 + 32 * j);
            }
        if (slot < 0 || slot >= a.num_slots) {
            if (slot != -1 && lane == 0) raise_error(a.err, KF_DEVERR_APPEND_POS);
            return;
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int i = i0 + 32 * j;
            if (i >= vecs) continue;
            if (FP8) {
                const int h = i * 8 / a.head_dim;
                static_cast<uint2 *>(a.k_cache)[slot * vecs + i] = codes_of(x[j], a.k_scale[h]);
                static_cast<uint2 *>(a.v_cache)[slot * vecs + i] = codes_of(y[j], a.v_scale[h]);
            } else {
                static_cast<uint4 *>(a.k_cache)[slot * vecs + i] = x[j];
                static_cast<uint4 *>(a.v_cache)[slot * vecs + i] = y[j];
            }
        }
    }
}

int ctas_for(int64_t items, int64_t per, int limit) {
    return (int)std::max<int64_t>(1, std::min<int64_t>((items + per - 1) / per, limit));
}

}  // namespace

cudaError_t launch_pool_init(int32_t *pool, int64_t num_blocks, cudaStream_t stream) {
    const int64_t n = std::max<int64_t>(num_blocks, KF_POOL_HEADER);
    pool_init_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(pool, num_blocks);
    return cudaGetLastError();
}

cudaError_t launch_extend(const PoolArgs &a, int sm_count, cudaStream_t stream) {
    extend_kernel<<<ctas_for(a.num_rows, kThreads, 2 * sm_count), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_release(const PoolArgs &a, int sm_count, cudaStream_t stream) {
    const int64_t most = (int64_t)a.batch * a.bt_stride;  // no more blocks than table entries
    release_kernel<<<ctas_for(most, kThreads, sm_count), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_append_rows(const RowsArgs &a, bool fp8, cudaStream_t stream) {
    const unsigned ctas = (unsigned)(((int64_t)a.num_rows + 7) / 8);
    if (fp8) append_rows_kernel<true><<<ctas, 256, 0, stream>>>(a);
    else append_rows_kernel<false><<<ctas, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kf
