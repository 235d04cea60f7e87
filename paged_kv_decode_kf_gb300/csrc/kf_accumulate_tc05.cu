// kf_accumulate_tc05.cu -- attention weight each cached token receives from a window
// of queries, bf16 keys, on tcgen05 (kf_accumulate.cu has the formula).
//
// Per KV head the queries' rows (j, g) are columns, 128 at a time:
//   S[128 tokens x N columns] = K Q^T,   N = min(128, columns left, rounded up to 16)
// with the tokens on the M side: a thread of the epilogue owns a token, so its sum of
// exp2(S * scale * log2 e - lse * log2 e) over columns and heads never leaves the
// thread, in one fixed order, and no token meets another (a NaN row stays its own).
//
// One CTA a run of 128-token tiles, each tile over all heads: per (head, 128 columns)
// 32 KB of Q, per head 32 KB of K (D = 128), 512 cycles of products and 16384
// exponentials, 1024 cycles of the SM's exponential unit: that unit is the bound of
// long runs. 4 requests of 4K-12K tokens, 32 queries of 32 / 8 heads: 25 us (a third of
// it the start and the two tiles a CTA has at most); with mma.sync and the keys in
// registers 66 us, bound by fragment loads.
//   warps 0-3 / 4-7  epilogue of the even / odd (head, column group) items
//   warp 8           TMA producer (K ring, Q ring);  warp 9  MMA issuer, TMEM owner
// Four score tiles of 128 TMEM columns; the two halves' sums meet in shared memory.
// Every wait is bounded; one that gives up sets KF_DEVERR_TIMEOUT, and every role
// still walks its whole run (without waiting again), so that no barrier is left.
#include <algorithm>

#include "kf_evict.cuh"
#include "kf_runs.cuh"
#include "kf_tc05_ops.cuh"

namespace kf {
namespace {

using namespace tc;
using namespace mq5;

constexpr int kTok = 128, kCols = 128;
constexpr int kProducerWarp = 8, kIssuerWarp = 9, kThreads = 320;

template <int D>
struct AShape {
    static constexpr int kAtomBytes = D / 64 * 1024;           // 8 tokens of K
    static constexpr int kKBytes = kTok / 8 * kAtomBytes;
    static constexpr int kQHalfBytes = kCols * 128;            // 128 columns x 64 numbers
    static constexpr int kQBytes = D / 64 * kQHalfBytes;
    static constexpr int kStages = 3;                          // of each ring
    static constexpr int kSmemBytes = std::max(kStages * (kKBytes + kQBytes) + 1024, 117 * 1024);
    static_assert(kSmemBytes <= 226 * 1024, "rings");
};

// Barrier `id` over 128 threads; whether `x` holds for all of them.
__device__ __forceinline__ bool bar_all(int id, bool x) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"((uint32_t)x), "r"(id)
        : "memory");
    return all != 0;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
accumulate_tc05_kernel(const AccumulateParams p, const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_q) {
    using Sh = AShape<D>;
    constexpr int NS = Sh::kStages;
    // kfull[NS], kempty[NS], qfull[NS], qempty[NS], s_full[4], s_empty[4], fin
    __shared__ __align__(8) uint64_t bar_mem[4 * NS + 9];
    __shared__ int64_t sm_loc[36];
    __shared__ __align__(16) float sm_lse[2][2][kCols];  // [half][item parity][column]
    __shared__ float sm_part[kTok];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t sK = base, sQ = base + NS * Sh::kKBytes;
    const uint32_t bars = smem_u32(bar_mem);
    auto kfull = [&](uint32_t i) { return bars + 8 * i; };
    auto kempty = [&](uint32_t i) { return bars + 8 * (NS + i); };
    auto qfull = [&](uint32_t i) { return bars + 8 * (2 * NS + i); };
    auto qempty = [&](uint32_t i) { return bars + 8 * (3 * NS + i); };
    auto s_full = [&](uint32_t i) { return bars + 8 * (4 * NS + i); };
    auto s_empty = [&](uint32_t i) { return bars + 8 * (4 * NS + 4 + i); };
    const uint32_t fin = bars + 8 * (4 * NS + 8);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 4 * NS; ++i) mbar_init(bars + 8 * i, 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(s_full(i), 1);
            mbar_init(s_empty(i), kTok);
        }
        mbar_init(fin, 1);
        abort_flag = (*(volatile unsigned int *)p.err & KF_DEVERR_TIMEOUT) ? 1 : 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kIssuerWarp) tc05::tmem_alloc(smem_u32(&tmem_slot), 512);
    auto tiles_of = [&](int b, bool report) { return (acc_request(p, b, report).L + kTok - 1) / kTok; };
    Place at;
    int64_t first;
    const int64_t total = locate(
        p.batch, [&](int b) { return tiles_of(b, blockIdx.x == 0); }, sm_loc,
        [&](int64_t T) { return cut_at(blockIdx.x, gridDim.x, T); }, at, first);
    int64_t count = cut_at(blockIdx.x + 1, gridDim.x, total) - first;
    if (abort_flag) count = 0;  // an earlier kernel's wait gave up (no role has started yet)
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    const uint32_t tm = tmem_slot;
    const int log_g = 31 - __clz(p.num_q_heads / p.num_kv_heads);
    const int H = p.num_kv_heads;

    // The run, as every role walks it: tiles, and in each (head, 128 columns) items.
    struct Tile {
        AccRequest r;
        int b, t0, cols, col0;  // columns before col0 (a multiple of 128) see no token of the tile
    };
    auto walk = [&](auto &&tile_fn) {
        int b = at.b;
        int64_t tile = at.off, n = count > 0 ? tiles_of(b, false) : 0;
        for (int64_t i = 0; i < count; ++i, ++tile) {
            while (tile >= n) {  // on to the next request with tokens (it exists)
                tile = 0;
                n = tiles_of(++b, false);
            }
            Tile t;
            t.r = acc_request(p, b, false);
            t.b = b;
            t.t0 = (int)tile * kTok;
            t.cols = (int)(t.r.C << log_g);
            t.col0 = 0;
            if (p.causal && t.t0 > t.r.shift) t.col0 = (int)(((t.t0 - t.r.shift) << log_g) & ~(int64_t)(kCols - 1));
            tile_fn(t);
        }
    };

    if (warp == kProducerWarp) {
        const int bs_shift = block_shift(p.block_size);
        const uint32_t box_bytes = (uint32_t)p.block_size * D * 2;
        uint32_t nk = 0, nq = 0;
        bool ok = true;
        walk([&](const Tile &t) {
            const int ntok = t.r.L - t.t0 < kTok ? (int)t.r.L - t.t0 : kTok;
            const int nblk = (ntok + p.block_size - 1) >> bs_shift;  // at most 8
            int64_t phys = 0;
            if (lane < nblk) {
                phys = p.block_tables[(int64_t)t.b * p.bt_stride + (t.t0 >> bs_shift) + lane];
                if (phys < 0 || phys >= p.num_blocks) {
                    raise_error(p.err, KF_DEVERR_BLOCK_ID);
                    phys = 0;
                }
            }
            for (int h = 0; h < H && ok && t.col0 < t.cols; ++h, ++nk) {
                const uint32_t ks = nk % NS;
                int go = 1;
                if (lane == 0) {
                    go = !abort_flag && mbar_wait(kempty(ks), ((nk / NS) & 1) ^ 1);
                    if (go) mbar_arrive_expect_tx(kfull(ks), nblk * box_bytes);
                }
                ok = __shfl_sync(0xffffffffu, go, 0);
                if (!ok) break;
                if (lane < nblk)
                    tma_load_4d(sK + ks * Sh::kKBytes + lane * box_bytes, &tmap_k, 0, 0, h * (D / 64),
                                (int)(phys * (p.block_size / 8)), kfull(ks));
                __syncwarp();
                for (int c0 = t.col0; c0 < t.cols; c0 += kCols, ++nq) {
                    const uint32_t qs = nq % NS;
                    if (lane == 0) {
                        go = !abort_flag && mbar_wait(qempty(qs), ((nq / NS) & 1) ^ 1);
                        if (go) {
                            mbar_arrive_expect_tx(qfull(qs), Sh::kQBytes);
                            tma_load_4d(sQ + qs * Sh::kQBytes, &tmap_q, 0, h << log_g, (int)t.r.q0 + (c0 >> log_g), 0,
                                        qfull(qs));
                        }
                    }
                    ok = __shfl_sync(0xffffffffu, go, 0);
                    if (!ok) break;
                }
                if (!ok) {  // K was asked for: it counts for the drain below
                    ++nk;
                    break;
                }
            }
        });
        if (lane == 0) {
            if (!ok) {
                raise_error(p.err, KF_DEVERR_TIMEOUT);
                abort_flag = 1;
            }
            // drain: every copy has landed before the CTA can exit
            for (uint32_t j = nk > NS ? nk - NS : 0; j < nk; ++j)
                if (!mbar_wait(kfull(j % NS), (j / NS) & 1)) raise_error(p.err, KF_DEVERR_TIMEOUT);
            for (uint32_t j = nq > NS ? nq - NS : 0; j < nq; ++j)
                if (!mbar_wait(qfull(j % NS), (j / NS) & 1)) raise_error(p.err, KF_DEVERR_TIMEOUT);
        }
        __syncwarp();
    } else if (warp == kIssuerWarp) {
        uint32_t nk = 0, nq = 0;
        bool ok = true;
        walk([&](const Tile &t) {
            const int cols = __shfl_sync(0xffffffffu, t.cols, 0), col0 = __shfl_sync(0xffffffffu, t.col0, 0);
            for (int h = 0; h < H && ok && col0 < cols; ++h, ++nk) {
                const uint32_t ks = nk % NS;
                ok = !__any_sync(0xffffffffu, abort_flag) && warp_wait(kfull(ks), (nk / NS) & 1);
                const uint64_t kd = tc05::sdesc_sw128(sK + ks * Sh::kKBytes, 16, Sh::kAtomBytes);
                for (int c0 = col0; c0 < cols && ok; c0 += kCols, ++nq) {
                    const uint32_t qs = nq % NS, sb = nq & 3;
                    ok = warp_wait(qfull(qs), (nq / NS) & 1) && warp_wait(s_empty(sb), ((nq >> 2) & 1) ^ 1);
                    if (!ok) break;
                    tc05::fence_after_sync();
                    const int N = min(kCols, (cols - c0 + 15) & ~15);
                    const uint32_t id = tc05::idesc_bf16(kTok, N, false, false);
                    const uint64_t qd = tc05::sdesc_sw128(sQ + qs * Sh::kQBytes, 16, 1024);
                    if (tc05::elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            tc05::mma_ss(tm + kCols * sb, kd + (uint64_t)(((kk >> 2) * 1024 + 32 * (kk & 3)) / 16),
                                         qd + (uint64_t)(((kk >> 2) * Sh::kQHalfBytes + 32 * (kk & 3)) / 16), id,
                                         kk > 0 ? 1u : 0u);
                        tc05::commit(s_full(sb));
                        tc05::commit(qempty(qs));
                        if (c0 + kCols >= cols) tc05::commit(kempty(ks));
                    }
                    __syncwarp();
                }
            }
        });
        if (tc05::elect_one()) {
            if (!ok) {
                raise_error(p.err, KF_DEVERR_TIMEOUT);
                abort_flag = 1;
            }
            tc05::commit(fin);  // every MMA has completed before TMEM is freed
            if (!mbar_wait(fin, 0)) raise_error(p.err, KF_DEVERR_TIMEOUT);
        }
        __syncwarp();
    } else {
        const int half = warp >> 2, row = threadIdx.x & (kTok - 1);
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        const float c = p.scale_log2;
        uint32_t nq = 0, mine = 0;  // items of the run; items of this half
        bool fail = false;
        walk([&](const Tile &t) {
            const int tok = t.t0 + row;
            // this token is seen by the columns from cmin on
            const int64_t cmin = p.causal ? (tok - t.r.shift) * (1 << log_g) : 0;
            float sum = 0.f;
            for (int h = 0; h < H; ++h)
                for (int c0 = t.col0; c0 < t.cols; c0 += kCols, ++nq) {
                    if ((int)(nq & 1) != half) continue;
                    const uint32_t sb = nq & 3, par = mine++ & 1;
                    // the columns' lse, one a thread; used by all
                    const int col = c0 + row;
                    float l = -INFINITY;
                    if (col < t.cols)
                        l = __ldg(p.lse + (t.r.q0 + (col >> log_g)) * p.num_q_heads + (h << log_g) +
                                  (col & ((1 << log_g) - 1)));
                    sm_lse[half][par][row] = l * 1.4426950408889634f;
                    const bool all_add = bar_all(1 + half, l != -INFINITY);
                    if (!fail) fail = !warp_wait(s_full(sb), (nq >> 2) & 1);
                    tc05::fence_after_sync();
                    const int ncol = min(kCols, t.cols - c0);
                    // every column of the group is there, adds something (an lse of -inf: nothing,
                    // whatever the scores are) and sees every token of the warp
                    const bool fast = __all_sync(0xffffffffu, all_add && cmin <= c0);
                    const float4 *lse4 = reinterpret_cast<const float4 *>(sm_lse[half][par]);
                    float2 acc = make_float2(0.f, 0.f);
                    const float2 c2 = make_float2(c, c);
                    for (int k = 0; k < ncol; k += 32) {
                        uint32_t x[32];
                        tc05::tmem_ld32(tm + lane_base + kCols * sb + k, x);
                        if (fast) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float4 l4 = lse4[k / 4 + e];
                                float2 a = fma_f32x2(make_float2(__uint_as_float(x[4 * e]), __uint_as_float(x[4 * e + 1])),
                                                     c2, make_float2(-l4.x, -l4.y));
                                float2 b = fma_f32x2(
                                    make_float2(__uint_as_float(x[4 * e + 2]), __uint_as_float(x[4 * e + 3])), c2,
                                    make_float2(-l4.z, -l4.w));
                                a.x = ex2f(a.x);
                                a.y = ex2f(a.y);
                                b.x = ex2f(b.x);
                                b.y = ex2f(b.y);
                                acc = add_f32x2(acc, add_f32x2(a, b));
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const float l2 = sm_lse[half][par][k + e];  // (-inf past the last column)
                                const float w = ex2f(fmaf(__uint_as_float(x[e]), c, -l2));
                                if (l2 != -INFINITY && c0 + k + e >= cmin) acc.x += w;
                            }
                        }
                    }
                    sum += acc.x + acc.y;
                    tc05::fence_before_sync();
                    mbar_arrive(s_empty(sb));
                }
            if (half == 1) sm_part[row] = sum;
            asm volatile("barrier.cta.sync 3, 256;" ::: "memory");
            if (half == 0 && tok < t.r.L) {
                const int64_t where = t.b * p.score_stride + tok;
                p.scores_out[where] = (p.scores_in ? p.scores_in[where] : 0.f) + (sum + sm_part[row]);
            }
            asm volatile("barrier.cta.sync 3, 256;" ::: "memory");  // sm_part is free again
        });
        if (fail) {
            if (lane == 0) raise_error(p.err, KF_DEVERR_TIMEOUT);
            abort_flag = 1;
        }
        __syncwarp();
    }
    tc05::fence_before_sync();
    __syncthreads();
    if (warp == kIssuerWarp) {
        tc05::fence_after_sync();
        tc05::tmem_dealloc(tm, 512);
    }
}

template <int D>
cudaError_t launch(const AccumulateParams &p, int sm_count, cudaStream_t stream, tc::EncodeFn fn) {
    using Sh = AShape<D>;
    const int G = p.num_q_heads / p.num_kv_heads;
    MqParams m{};
    m.num_kv_heads = p.num_kv_heads;
    m.head_dim = D;
    m.num_blocks = p.num_blocks;
    m.block_size = p.block_size;
    CUtensorMap mk, mq;
    if (!encode_block_map(fn, &mk, p.k_cache, m)) return cudaErrorInvalidValue;
    // q [num_q_tokens, Hq, D] as (64 numbers, head, token, D / 64): a box of one KV head's
    // group over 128 / G tokens is 128 columns
    const cuuint64_t head = (cuuint64_t)D * 2;
    const cuuint64_t dims[4] = {64, (cuuint64_t)p.num_q_heads, (cuuint64_t)p.num_q_tokens, D / 64};
    const cuuint64_t strides[3] = {head, head * p.num_q_heads, 128};
    const cuuint32_t box[4] = {64, (cuuint32_t)G, (cuuint32_t)(kCols / G), D / 64};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    if (fn(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t *>(p.q), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done.load() & bit)) {
        e = cudaFuncSetAttribute(accumulate_tc05_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Sh::kSmemBytes);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit);
    }
    const int64_t tiles = (int64_t)p.batch * (((int64_t)p.max_context_len + kTok - 1) / kTok);
    accumulate_tc05_kernel<D><<<(unsigned)std::min<int64_t>(sm_count, tiles), kThreads, Sh::kSmemBytes, stream>>>(p, mk,
                                                                                                               mq);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_accumulate_tc05(const AccumulateParams &p, int sm_count, cudaStream_t stream, void *encode_fn) {
    tc::EncodeFn fn = reinterpret_cast<tc::EncodeFn>(encode_fn);
    return p.head_dim == 128 ? launch<128>(p, sm_count, stream, fn) : launch<64>(p, sm_count, stream, fn);
}

}  // namespace kf
