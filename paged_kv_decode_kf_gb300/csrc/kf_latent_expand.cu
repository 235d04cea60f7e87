// kf_latent_expand.cu -- keys and values of every cached token from its latent.
//
//   C [128 tokens x R] W_h^T   (W_h = W_uk_h, then W_uv_h; both at once where nope = v = 64)
// on tcgen05: A = the latents (K-major, one box a cache block), B = the head's
// weights (K-major), fp32 in TMEM, N = 128.
//
// A tile of 128 tokens' latents (128 KB at R = 512) stays in shared memory while the
// weights of all heads (8 MB at 32 heads, R = 512; in L2) stream through a ring of
// 64-column slices of 16 KB. A CTA's run is a run of (token tile, unit) pairs, token
// tile slowest, so the latents are loaded once or twice a CTA and every SM gets
// equal work. Four accumulators: the epilogue of one unit runs under the products of
// the next ones. A slice feeds 4 instructions of 64 cycles, 64 B a cycle and SM from
// L2 with 64 KB in flight: the latency of L2 under that load is the bound. (Clusters
// that multicast the slices were slower: 286 us with two CTAs, 553 with four, against
// 293 -- a CTA that waits stops its partners.)
//
// The epilogue's thread owns a token: K as hi = bf16(k) and lo = bf16(k - hi), V as
// fp16, through 4 KB of shared memory a warp, so that a store covers whole 128-byte
// lines (32-byte pieces of 32 rows a store cost 120 of 295 us on 4 requests of
// 4K-12K tokens, 32 heads). A value above fp16's range sets KF_DEVERR_RANGE.
//   warps 0-3 epilogue, warp 4 TMA producer, warp 5 MMA issuer and TMEM owner.
#include <algorithm>

#include "kf_latent_expanded.cuh"

namespace kf {
namespace {

using namespace tc;
using namespace mq5;

constexpr int kM = 128, kEpiThreads = 128, kProducerWarp = 4, kIssuerWarp = 5, kThreads = 192;

constexpr int kN = 128;  // columns a unit

template <int R, int DN, int DV>
struct XShape {
    static constexpr int kUnits = (DN + DV) / kN;                // units a head
    static constexpr int kAtoms = R / 64;
    static constexpr int kGroupBytes = kAtoms * 1024;            // 8 tokens
    static constexpr int kABytes = kM / 8 * kGroupBytes;
    static constexpr int kSliceBytes = kN * 128;                 // 64 columns of a unit's weights
    static constexpr int kStages = R == 512 ? 5 : 7;
    static constexpr int kStageOut = 4 * 32 * 128;               // a warp's 32 rows x 128 bytes
    static constexpr int kSmemBytes = kABytes + kStages * kSliceBytes + kStageOut + 1024;
    static_assert((kUnits == 2 && DN == kN && DV == kN) || kUnits == 1, "a unit is K, V, or both");
    static_assert(kSmemBytes > 117 * 1024 && kSmemBytes <= 225 * 1024, "one CTA an SM");
};

__device__ __forceinline__ int64_t tiles_of(const LatentParams &p, int b, bool report, int64_t *L) {
    const LatentRequest r = latent_request(p, b, report);
    *L = r.q0 < 0 || r.C == 0 ? 0 : r.L < p.max_context_len ? r.L : p.max_context_len;
    return (*L + kM - 1) / kM;
}

// A run over (token tile, unit) pairs, `units` of them a tile.
struct PairWalker {
    int b, u, units;
    int64_t tile, tiles, L, left;

    __device__ __forceinline__ void start(const LatentParams &p, const Place &at, int n_units, int64_t n) {
        b = at.b;
        units = n_units;
        left = n;
        if (left <= 0) return;
        tiles = tiles_of(p, b, false, &L);
        tile = at.off / units;
        u = (int)(at.off - tile * units);
    }
    // after the current pair; false at the run's end. `fresh`: the token tile changed.
    __device__ __forceinline__ bool step(const LatentParams &p, bool &fresh) {
        if (--left <= 0) return false;
        fresh = false;
        if (++u < units) return true;
        u = 0;
        fresh = true;
        if (++tile < tiles) return true;
        tile = 0;
        do {
            if (++b >= p.batch) return false;
            tiles = tiles_of(p, b, false, &L);
        } while (tiles == 0);
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
    constexpr int NS = Sh::kStages;
    // full[NS], empty[NS], a_full, a_empty, acc_full[4], acc_empty[4], fin
    __shared__ __align__(8) uint64_t bar_mem[2 * NS + 11];
    __shared__ int64_t sm_loc[36];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t sA = base, sW = base + Sh::kABytes, sOut = sW + NS * Sh::kSliceBytes;
    const uint32_t bars = smem_u32(bar_mem);
    auto full = [&](uint32_t i) { return bars + 8u * i; };
    auto empty = [&](uint32_t i) { return bars + 8u * (NS + i); };
    const uint32_t a_full = bars + 8u * (2 * NS), a_empty = a_full + 8, fin = a_full + 80;
    auto acc_full = [&](uint32_t i) { return a_full + 16 + 8 * i; };
    auto acc_empty = [&](uint32_t i) { return a_full + 48 + 8 * i; };
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        mbar_init(a_full, 1);
        mbar_init(a_empty, 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(acc_full(i), 1);
            mbar_init(acc_empty(i), kEpiThreads);
        }
        mbar_init(fin, 1);
        abort_flag = (*(volatile unsigned int *)p.err & KF_DEVERR_TIMEOUT) ? 1 : 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kIssuerWarp) tc05::tmem_alloc(smem_u32(&tmem_slot), 512);
    Place at;
    int64_t slot0;
    const int64_t total = locate(
        p.batch,
        [&](int b) {
            int64_t L;
            return tiles_of(p, b, blockIdx.x == 0, &L) * p.num_heads * Sh::kUnits;
        },
        sm_loc, [&](int64_t T) { return cut_at(blockIdx.x, gridDim.x, T); }, at, slot0);
    int64_t count = cut_at(blockIdx.x + 1, gridDim.x, total) - slot0;
    if (abort_flag) count = 0;  // an earlier kernel's wait gave up (no role has started yet)
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    const uint32_t tm = tmem_slot;
    PairWalker w;
    w.start(p, at, p.num_heads * Sh::kUnits, count);

    if (count > 0 && warp == kProducerWarp) {
        const int bs_shift = block_shift(p.block_size);
        const uint32_t box_bytes = (uint32_t)p.block_size * R * 2;
        uint32_t g = 0, loads = 0;
        bool ok = true, fresh = true;
        do {
            if (fresh) {  // the token tile's latents, once the products of the previous one are done
                const int64_t t0 = w.tile * kM;
                const int64_t ntok = w.L - t0 < kM ? w.L - t0 : kM;
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
                    const uint32_t dst = sW + st * Sh::kSliceBytes;
                    if (Sh::kUnits == 2) {  // W_uk_h, W_uv_h in turn
                        tc05::tma_load_3d(dst, (w.u & 1) ? &tmap_uv : &tmap_uk, 0, (w.u >> 1) * DN, a, full(st));
                    } else {
                        tc05::tma_load_3d(dst, &tmap_uk, 0, w.u * DN, a, full(st));
                        tc05::tma_load_3d(dst + DN * 128, &tmap_uv, 0, w.u * DV, a, full(st));
                    }
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
    } else if (count > 0 && warp == kIssuerWarp) {
        const uint32_t id = tc05::idesc_bf16(kM, kN, false, false);
        const uint64_t ad = tc05::sdesc_sw128(sA, 16, Sh::kGroupBytes);
        const uint64_t wd = tc05::sdesc_sw128(sW, 16, 1024);
        uint32_t g = 0, u = 0, loads = 0;
        bool ok = true, fresh = true;
        do {
            if (fresh) {
                ok = warp_wait(a_full, loads & 1);
                ++loads;
            }
            ok = ok && !__any_sync(0xffffffffu, abort_flag) && warp_wait(acc_empty(u & 3), ((u >> 2) & 1) ^ 1);
            for (int a = 0; a < Sh::kAtoms && ok; ++a, ++g) {
                const uint32_t st = g % NS;
                ok = warp_wait(full(st), (g / NS) & 1);
                if (!ok) break;
                tc05::fence_after_sync();
                if (tc05::elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc05::mma_ss(tm + (u & 3) * kN, ad + (uint64_t)((a * 1024 + 32 * kk) / 16),
                                     wd + (uint64_t)((st * Sh::kSliceBytes + 32 * kk) / 16), id,
                                     (a > 0 || kk > 0) ? 1u : 0u);
                    tc05::commit(empty(st));
                }
                __syncwarp();
            }
            if (!ok) break;
            const bool more = w.step(p, fresh);
            if (tc05::elect_one()) {
                tc05::commit(acc_full(u & 3));
                if (!more || fresh) tc05::commit(a_empty);
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
            tc05::commit(fin);  // every MMA has completed before TMEM is freed
            if (!mbar_wait(fin, 0)) raise_error(p.err, KF_DEVERR_TIMEOUT);
        }
        __syncwarp();
    } else if (count > 0 && warp < 4) {
        const uint32_t lane_base = (uint32_t)(32 * warp) << 16;
        uint32_t u = 0;
        bool fresh, range = false;
        do {
            if (!warp_wait(acc_full(u & 3), (u >> 2) & 1)) {
                if (lane == 0) raise_error(p.err, KF_DEVERR_TIMEOUT);
                abort_flag = 1;
                break;
            }
            tc05::fence_after_sync();
            const int64_t t0 = w.tile * kM + 32 * warp;          // the warp's first token
            const int64_t left = w.L - t0;
            const int rows = left < 0 ? 0 : left < 32 ? (int)left : 32;
            const int h = w.u / Sh::kUnits;
            const int64_t row = (int64_t)h * kv.rows + w.b * kv.cap + t0;
            uint8_t *const kr = reinterpret_cast<uint8_t *>(kv.k + row * (2 * DN));
            uint8_t *const vr = reinterpret_cast<uint8_t *>(kv.v + row * DV);
            const uint32_t acc = tm + lane_base + (u & 3) * kN, stage = sOut + warp * (32 * 128);
#pragma unroll
            for (int c = 0; c < kN; c += 64) {
                uint32_t x[64];
                tc05::tmem_ld64(acc + c, x);
                if (Sh::kUnits == 2 ? !(w.u & 1) : c < DN) {  // keys
                    uint32_t hi[32], lo[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float a = __uint_as_float(x[2 * e]), b = __uint_as_float(x[2 * e + 1]);
                        hi[e] = pack_bf16(a, b);
                        lo[e] = pack_bf16(a - bf16_lo(hi[e]), b - bf16_hi(hi[e]));
                    }
                    store_lines(stage, hi, kr + 2 * c, 4 * DN, rows);
                    store_lines(stage, lo, kr + 2 * (DN + c), 4 * DN, rows);
                } else {
                    uint32_t v[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float a = __uint_as_float(x[2 * e]), b = __uint_as_float(x[2 * e + 1]);
                        range = range || (lane < rows && !(fmaxf(fabsf(a), fabsf(b)) <= 65504.f));
                        v[e] = pack_f16(a, b);
                    }
                    store_lines(stage, v, vr + 2 * (c % DV), 2 * DV, rows);
                }
            }
            tc05::fence_before_sync();
            mbar_arrive(acc_empty(u & 3));
            ++u;
        } while (w.step(p, fresh));
        if (range) raise_error(p.err, KF_DEVERR_RANGE);
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the attention may be set up
    tc05::fence_before_sync();
    __syncthreads();
    if (warp == kIssuerWarp) {
        tc05::fence_after_sync();
        tc05::tmem_dealloc(tm, 512);
    }
}

template <int R, int DN, int DV>
cudaError_t launch(const LatentParams &p, const ExpandedKV &kv, int ctas, cudaStream_t stream, const CUtensorMap &mc,
                   const CUtensorMap &mk, const CUtensorMap &mv) {
    using Sh = XShape<R, DN, DV>;
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
    expand_kernel<R, DN, DV><<<ctas, kThreads, Sh::kSmemBytes, stream>>>(p, kv, mc, mk, mv);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_latent_expand(const LatentParams &p, const LatentWeights &w, const ExpandedKV &kv, int sm_count,
                                 cudaStream_t stream, tc::EncodeFn fn) {
    CUtensorMap mc, mk, mv;
    const int R = p.latent_dim;
    if (!encode_latent_cache(fn, &mc, p, R / 64) ||
        !encode_rows(fn, &mk, w.w_uk, (int64_t)p.num_heads * w.nope, R, w.nope, 1) ||
        !encode_rows(fn, &mv, w.w_uv, (int64_t)p.num_heads * w.v, R, w.v, 1))
        return cudaErrorInvalidValue;
    const int64_t pairs = (int64_t)p.batch * (kv.cap / kM) * p.num_heads;  // (at least)
    const int ctas = (int)std::min<int64_t>(sm_count, pairs);
    if (ctas == 0) return cudaSuccess;
    if (R == 512)
        return w.nope == 128 ? launch<512, 128, 128>(p, kv, ctas, stream, mc, mk, mv)
                             : launch<512, 64, 64>(p, kv, ctas, stream, mc, mk, mv);
    return w.nope == 128 ? launch<256, 128, 128>(p, kv, ctas, stream, mc, mk, mv)
                         : launch<256, 64, 64>(p, kv, ctas, stream, mc, mk, mv);
}

}  // namespace kf
