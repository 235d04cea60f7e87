// kf_latent_expand.cu -- keys and values of every cached token from its latent.
//
//   [K | V]_h [256 tokens x (nope + v)] = C [256 tokens x R] [W_uk_h ; W_uv_h]^T
// on CTA pairs (tcgen05.mma.cta_group::2, M = 256): each CTA holds the latents of its
// own token tile of 128 (A, K-major, one box a cache block; 128 KB at R = 512) and
// one of the two weight matrices (half of B's rows: W_uk in the even CTA, W_uv in the
// odd one), and gets its tokens' K and V in its own TMEM, fp32.
//
// The weights of all heads (8 MB at 32 heads, R = 512; in L2) stream through a ring of
// 64-column slices, 16 KB a CTA, that feed 4 instructions of 128 cycles: 32 B a cycle
// and SM from L2. A pair's run is a run of (two token tiles, head), token tiles slowest,
// so the latents are loaded once or twice and every SM gets equal work. Two
// accumulators: the epilogue of one head runs under the products of the next.
// Without pairs the weights take 64 B a cycle and SM, and with N = 128 the operand
// reads alone take shared memory's 128 B a cycle: 295 us on 4 requests of 4K-12K
// tokens, 32 heads, whatever the ring's depth; clusters that multicast the slices
// (two CTAs 286 us, four 553) stop all partners when one waits.
//
// The epilogue's thread owns a token: K as hi = bf16(k) and lo = bf16(k - hi), V as
// fp16, through 4 KB of shared memory a warp, so that a store covers whole 128-byte
// lines (with heads of 128 it spills 16 bytes of its 168 registers). A value above fp16's range sets KF_DEVERR_RANGE.
//   warps 0-3 / 4-7  epilogue of the even / odd heads of the run (their accumulator)
//   warp 8           TMA producer
//   warp 9           even CTA: MMA issuer; odd CTA: tells the even one what has landed
//                    (an mbarrier can be waited on only in its own CTA). TMEM owners.
// Every wait is bounded; one that gives up sets KF_DEVERR_TIMEOUT, and both CTAs still
// meet (a bounded handshake) before either frees its TMEM or leaves.
#include <algorithm>

#include "kf_latent_expanded.cuh"

namespace kf {
namespace {

using namespace tc;
using namespace mq5;

constexpr int kM = 128, kProducerWarp = 8, kIssuerWarp = 9, kThreads = 320;

template <int R, int DN, int DV>
struct XShape {
    static constexpr int kN = DN + DV;                           // columns of a head
    static constexpr int kAtoms = R / 64;
    static constexpr int kGroupBytes = kAtoms * 1024;            // 8 tokens
    static constexpr int kABytes = kM / 8 * kGroupBytes;
    static constexpr int kSliceBytes = DN * 128;                 // 64 columns of one weight matrix
    static constexpr int kStageOut = 8 * 32 * 128;               // a warp's 32 rows x 128 bytes
    static constexpr int kStages = DN == 64 ? 8 : R == 512 ? 4 : 7;
    static constexpr int kSmemBytes = kABytes + kStages * kSliceBytes + kStageOut + 1024;
    static_assert(DN == DV, "the pair's halves of B");
    static_assert(kSmemBytes > 117 * 1024 && kSmemBytes <= 225 * 1024, "one CTA an SM");
};

__device__ __forceinline__ int64_t tiles_of(const LatentParams &p, int b, bool report, int64_t *L) {
    const LatentRequest r = latent_request(p, b, report);
    *L = r.q0 < 0 || r.C == 0 ? 0 : r.L < p.max_context_len ? r.L : p.max_context_len;
    return (*L + kM - 1) / kM;
}

// A run over (pair of token tiles, head), as the CTA of one tile of the pair sees it. A
// tile past the batch's last is empty (L = 0).
struct PairWalker {
    int b, h;
    int64_t tile, tiles, L, left;

    // `at`: the request and tile of this CTA in the run's first pair, if it has one
    __device__ __forceinline__ void start(const LatentParams &p, const Place &at, bool has, int first_head, int64_t n) {
        left = n;
        h = first_head;
        b = has ? at.b : p.batch;
        tile = has ? at.off : 0;
        tiles = L = 0;
        if (has) tiles = tiles_of(p, b, false, &L);
    }
    // On to the next head; false at the run's end. `fresh`: the token tiles changed.
    __device__ __forceinline__ bool step(const LatentParams &p, bool &fresh) {
        if (--left <= 0) return false;
        fresh = false;
        if (++h < p.num_heads) return true;
        h = 0;
        fresh = true;
        tile += 2;
        while (b < p.batch && tile >= tiles) {
            tile -= tiles;
            if (++b < p.batch) tiles = tiles_of(p, b, false, &L);
        }
        if (b >= p.batch) L = 0;
        return true;
    }
};

// 64 16-bit numbers a lane (w: pairs), one row a lane, to row `lane` of `dst` (pitch in
// bytes), rows below `rows`: through the warp's 4 KB at `stage`, eight lanes a row.
__device__ __forceinline__ void store_lines(uint32_t stage, const uint32_t (&w)[32], uint8_t *dst, int pitch, int rows) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int c = 0; c < 8; ++c)
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * 128 + ((c ^ (lane & 7)) << 4)),
                     "r"(w[4 * c]), "r"(w[4 * c + 1]), "r"(w[4 * c + 2]), "r"(w[4 * c + 3])
                     : "memory");
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = 4 * i + (lane >> 3), c = lane & 7;
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(stage + r * 128 + ((c ^ (r & 7)) << 4))
                     : "memory");
        if (r < rows) *reinterpret_cast<uint4 *>(dst + (int64_t)r * pitch + c * 16) = v;
    }
    __syncwarp();
}

template <int R, int DN, int DV>
__global__ void __launch_bounds__(kThreads, 1)
expand_kernel(const LatentParams p, const ExpandedKV kv, const __grid_constant__ CUtensorMap tmap_c,
              const __grid_constant__ CUtensorMap tmap_uk, const __grid_constant__ CUtensorMap tmap_uv) {
    using Sh = XShape<R, DN, DV>;
    constexpr int NS = Sh::kStages, N = Sh::kN;
    constexpr uint16_t both = 3;
    // In each CTA: full[NS], empty[NS], a_full, a_empty, acc_full[2], fin, bye. Used in the
    // even one: pfull[NS] and pa_full (the odd CTA's slices and latents have landed),
    // acc_empty[2] (arrivals of both CTAs' epilogue warps).
    __shared__ __align__(8) uint64_t bar_mem[3 * NS + 9];
    __shared__ int64_t sm_loc[36];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t sA = base, sW = base + Sh::kABytes, sOut = sW + NS * Sh::kSliceBytes;
    const uint32_t bars = smem_u32(bar_mem);
    auto full = [&](uint32_t i) { return bars + 8u * i; };
    auto empty = [&](uint32_t i) { return bars + 8u * (NS + i); };
    auto pfull = [&](uint32_t i) { return bars + 8u * (2 * NS + i); };
    const uint32_t a_full = bars + 8u * (3 * NS), a_empty = a_full + 8, pa_full = a_full + 16, fin = a_full + 24,
                   bye = a_full + 32;
    auto acc_full = [&](uint32_t i) { return a_full + 40 + 8 * i; };
    auto acc_empty = [&](uint32_t i) { return a_full + 56 + 8 * i; };
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t cr = cluster_rank();  // 0: the issuing (even) CTA of the pair
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 3 * NS; ++i) mbar_init(bars + 8 * i, 1);
        mbar_init(a_full, 1);
        mbar_init(a_empty, 1);
        mbar_init(pa_full, 1);
        mbar_init(fin, 1);
        mbar_init(bye, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full(i), 1);
            mbar_init(acc_empty(i), 8);  // four warps of each CTA
        }
        abort_flag = (*(volatile unsigned int *)p.err & KF_DEVERR_TIMEOUT) ? 1 : 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kIssuerWarp) tc05::tmem_alloc2(smem_u32(&tmem_slot), 512);
    Place at;
    int64_t tile0, first = 0, count = 0;
    const int64_t total = locate(
        p.batch,
        [&](int b) {
            int64_t L;
            return tiles_of(p, b, blockIdx.x == 0, &L);
        },
        sm_loc,
        [&](int64_t T) {
            const int64_t work = (T + 1) / 2 * p.num_heads;
            first = cut_at(pair, pairs, work);
            count = cut_at(pair + 1, pairs, work) - first;
            return first / p.num_heads * 2 + cr;
        },
        at, tile0);
    if (abort_flag) count = 0;  // an earlier kernel's wait gave up (no role has started yet)
    PairWalker w;
    w.start(p, at, tile0 < total, (int)(first % p.num_heads), count);
    tc05::fence_before_sync();
    cluster_sync_all();  // both CTAs' barriers exist before any remote arrival
    tc05::fence_after_sync();
    const uint32_t tm = tmem_slot;

    if (count > 0 && warp == kProducerWarp) {
        const int bs_shift = block_shift(p.block_size);
        const uint32_t box_bytes = (uint32_t)p.block_size * R * 2;
        const CUtensorMap *const tmap_w = cr == 0 ? &tmap_uk : &tmap_uv;
        uint32_t g = 0, loads = 0;
        bool ok = true, fresh = true;
        do {
            if (fresh) {  // the token tile's latents, once the products of the previous one are done
                const int64_t t0 = w.tile * kM;
                const int64_t ntok = w.L <= t0 ? 0 : w.L - t0 < kM ? w.L - t0 : kM;
                const int nblk = (int)((ntok + p.block_size - 1) >> bs_shift);  // at most 8
                int64_t phys = 0;
                if (lane < nblk) {
                    phys = p.block_tables[(int64_t)w.b * p.bt_stride + (t0 >> bs_shift) + lane];
                    if (phys < 0 || phys >= p.num_blocks) {
                        raise_error(p.err, KF_DEVERR_BLOCK_ID);
                        phys = 0;
                    }
                }
                int go = 1;
                if (lane == 0) {
                    go = !abort_flag && mbar_wait(a_empty, (loads & 1) ^ 1);
                    if (go) mbar_arrive_expect_tx(a_full, nblk * box_bytes);
                }
                ok = __shfl_sync(0xffffffffu, go, 0);
                if (!ok) break;
                if (lane < nblk)
                    tma_load_4d(sA + lane * box_bytes, &tmap_c, 0, 0, 0, (int)(phys * (p.block_size / 8)), a_full);
                __syncwarp();
                ++loads;
            }
            if (lane == 0) {
                for (int a = 0; a < Sh::kAtoms; ++a, ++g) {
                    const uint32_t st = g % NS;
                    ok = !abort_flag && mbar_wait(empty(st), ((g / NS) & 1) ^ 1);
                    if (!ok) break;
                    mbar_arrive_expect_tx(full(st), Sh::kSliceBytes);
                    tc05::tma_load_3d(sW + st * Sh::kSliceBytes, tmap_w, 0, w.h * DN, a, full(st));
                }
            }
            ok = __shfl_sync(0xffffffffu, (int)ok, 0);
        } while (ok && w.step(p, fresh));
        if (lane == 0) {
            if (!ok) {
                raise_error(p.err, KF_DEVERR_TIMEOUT);
                abort_flag = 1;
            }
            // drain: every copy has landed before the CTA can exit
            for (uint32_t j = g > NS ? g - NS : 0; j < g; ++j)
                if (!mbar_wait(full(j % NS), (j / NS) & 1)) raise_error(p.err, KF_DEVERR_TIMEOUT);
            if (loads > 0 && !mbar_wait(a_full, (loads - 1) & 1)) raise_error(p.err, KF_DEVERR_TIMEOUT);
        }
        __syncwarp();
    } else if (count > 0 && warp == kIssuerWarp && cr == 1) {
        // ------------- odd CTA: passes on what has landed, in the issuer's order -------------
        if (lane == 0) {
            const uint32_t lead_pfull = map_to(pfull(0), 0), lead_pa = map_to(pa_full, 0);
            uint32_t g = 0, loads = 0;
            bool ok = true, fresh = true;
            do {
                if (fresh) {
                    ok = mbar_wait(a_full, loads & 1);
                    if (ok) arrive_cluster(lead_pa);
                    ++loads;
                }
                for (int a = 0; a < Sh::kAtoms && ok; ++a, ++g) {
                    ok = !abort_flag && mbar_wait(full(g % NS), (g / NS) & 1);
                    if (ok) arrive_cluster(lead_pfull + 8 * (g % NS));
                }
            } while (ok && w.step(p, fresh));
            if (!ok) {
                raise_error(p.err, KF_DEVERR_TIMEOUT);
                abort_flag = 1;
            }
        }
        __syncwarp();
    } else if (count > 0 && warp == kIssuerWarp) {
        // ------------------------------ even CTA: MMA issuer ------------------------------
        const uint32_t id = tc05::idesc_bf16(2 * kM, N, false, false);
        const uint64_t ad = tc05::sdesc_sw128(sA, 16, Sh::kGroupBytes);
        const uint64_t wd = tc05::sdesc_sw128(sW, 16, 1024);
        uint32_t g = 0, u = 0, loads = 0;
        bool ok = true, fresh = true;
        do {
            if (fresh) {
                ok = warp_wait(a_full, loads & 1) && warp_wait(pa_full, loads & 1);
                ++loads;
            }
            ok = ok && !__any_sync(0xffffffffu, abort_flag) && warp_wait(acc_empty(u & 1), ((u >> 1) & 1) ^ 1);
            for (int a = 0; a < Sh::kAtoms && ok; ++a, ++g) {
                const uint32_t st = g % NS;
                ok = warp_wait(full(st), (g / NS) & 1) && warp_wait(pfull(st), (g / NS) & 1);
                if (!ok) break;
                tc05::fence_after_sync();
                if (tc05::elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc05::mma2_ss(tm + (u & 1) * 256, ad + (uint64_t)((a * 1024 + 32 * kk) / 16),
                                      wd + (uint64_t)((st * Sh::kSliceBytes + 32 * kk) / 16), id,
                                      (a > 0 || kk > 0) ? 1u : 0u);
                    tc05::commit2(empty(st), both);
                }
                __syncwarp();
            }
            if (!ok) break;
            const bool more = w.step(p, fresh);
            if (tc05::elect_one()) {
                tc05::commit2(acc_full(u & 1), both);
                if (!more || fresh) tc05::commit2(a_empty, both);
            }
            __syncwarp();
            ++u;
            if (!more) break;
        } while (true);
        if (tc05::elect_one()) {
            if (!ok) {
                raise_error(p.err, KF_DEVERR_TIMEOUT);
                abort_flag = 1;
            }
            tc05::commit2(fin, both);  // every MMA has completed before TMEM is freed
            if (!mbar_wait(fin, 0)) raise_error(p.err, KF_DEVERR_TIMEOUT);
        }
        __syncwarp();
    } else if (count > 0 && warp < 8) {
        const int half = warp >> 2;
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t stage = sOut + warp * (32 * 128);
        const uint32_t my_empty = map_to(acc_empty(half), 0);
        uint32_t u = 0;
        bool fresh, range = false;
        do {
            if ((int)(u & 1) != half) {
                ++u;
                continue;
            }
            if (!warp_wait(acc_full(half), (u >> 1) & 1)) {
                if (lane == 0) raise_error(p.err, KF_DEVERR_TIMEOUT);
                abort_flag = 1;
                break;
            }
            tc05::fence_after_sync();
            const int64_t t0 = w.tile * kM + 32 * (warp & 3);    // the warp's first token
            const int64_t left = w.L - t0;
            const int rows = left < 0 ? 0 : left < 32 ? (int)left : 32;
            const int64_t row = (int64_t)w.h * kv.rows + w.b * kv.cap + t0;
            uint8_t *const kr = reinterpret_cast<uint8_t *>(kv.k + row * (2 * DN));
            uint8_t *const vr = reinterpret_cast<uint8_t *>(kv.v + row * DV);
            const uint32_t acc = tm + lane_base + half * 256;
#pragma unroll 1
            for (int c = 0; c < DN; c += 64) {
                uint32_t x[64], lo[32];
                tc05::tmem_ld64(acc + c, x);
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float a = __uint_as_float(x[2 * e]), b = __uint_as_float(x[2 * e + 1]);
                    x[e] = pack_bf16(a, b);
                    lo[e] = pack_bf16(a - bf16_lo(x[e]), b - bf16_hi(x[e]));
                }
                uint32_t hi[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) hi[e] = x[e];
                store_lines(stage, hi, kr + 2 * c, 4 * DN, rows);
                store_lines(stage, lo, kr + 2 * (DN + c), 4 * DN, rows);
            }
#pragma unroll 1
            for (int c = 0; c < DV; c += 64) {
                uint32_t x[64], v[32];
                tc05::tmem_ld64(acc + DN + c, x);
                if (c + 64 == DV) {  // the accumulator is free for the next head but one
                    tc05::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) arrive_cluster(my_empty);
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float a = __uint_as_float(x[2 * e]), b = __uint_as_float(x[2 * e + 1]);
                    range = range || (lane < rows && !(fmaxf(fabsf(a), fabsf(b)) <= 65504.f));
                    v[e] = pack_f16(a, b);
                }
                store_lines(stage, v, vr + 2 * c, 2 * DV, rows);
            }
            ++u;
        } while (w.step(p, fresh));
        if (range) raise_error(p.err, KF_DEVERR_RANGE);
        __syncwarp();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the attention may be set up
    tc05::fence_before_sync();
    __syncthreads();
    if (warp == kIssuerWarp) {
        // neither CTA frees its TMEM (or exits) while the other may still reach into it
        if (lane == 0) {
            arrive_cluster(map_to(bye, cr ^ 1u));
            if (!wait_cl(bye, 0)) raise_error(p.err, KF_DEVERR_TIMEOUT);
        }
        __syncwarp();
        tc05::fence_after_sync();
        tc05::tmem_dealloc2(tm, 512);
    }
}

template <int R, int DN, int DV>
cudaError_t launch(const LatentParams &p, const LatentWeights &w, const ExpandedKV &kv, int sm_count,
                   cudaStream_t stream, tc::EncodeFn fn) {
    using Sh = XShape<R, DN, DV>;
    CUtensorMap mc, mk, mv;
    if (!encode_latent_cache(fn, &mc, p, R / 64) ||
        !encode_rows(fn, &mk, w.w_uk, (int64_t)p.num_heads * DN, R, DN, 1) ||
        !encode_rows(fn, &mv, w.w_uv, (int64_t)p.num_heads * DV, R, DV, 1))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done.load() & bit)) {
        e = cudaFuncSetAttribute(expand_kernel<R, DN, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmemBytes);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit);
    }
    // no more pairs of CTAs than the batch can have (pair of token tiles, head)
    const int64_t work = ((int64_t)p.batch * (kv.cap / kM) + 1) / 2 * p.num_heads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (unsigned)std::min<int64_t>(std::max(1, sm_count / 2), work));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Sh::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;  // the pair: cluster ranks 0 and 1
    attr[0].val.clusterDim = {2, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, expand_kernel<R, DN, DV>, p, kv, mc, mk, mv);
}

}  // namespace

cudaError_t launch_latent_expand(const LatentParams &p, const LatentWeights &w, const ExpandedKV &kv, int sm_count,
                                 cudaStream_t stream, tc::EncodeFn fn) {
    if (p.latent_dim == 512)
        return w.nope == 128 ? launch<512, 128, 128>(p, w, kv, sm_count, stream, fn)
                             : launch<512, 64, 64>(p, w, kv, sm_count, stream, fn);
    return w.nope == 128 ? launch<256, 128, 128>(p, w, kv, sm_count, stream, fn)
                         : launch<256, 64, 64>(p, w, kv, sm_count, stream, fn);
}

}  // namespace kf
