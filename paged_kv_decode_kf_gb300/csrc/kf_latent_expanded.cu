// kf_latent_expanded.cu -- latent attention, expanded form, on tcgen05.
//
// Head h's keys [W_uk_h c_t ; r_t] and values W_uv_h c_t come from kf_latent_expand.cu
// (K as bf16 pairs hi + lo, V as fp16, in the workspace); the rotary keys r_t are
// read from the cache. Per (request, head, 256 query tokens) one CTA:
//   S[128 rows x 64 tokens] = q_n K_hi^T + q_n K_lo^T + q_r r^T   (bf16)
//   O[128 rows x v]        += P V                                 (fp16)
// The low halves keep S, and so lse, as exact as bf16 inputs with fp32 sums allow;
// they cost 128 of S's 320 columns. P and V as fp16 round an eighth as much as
// bf16 would; a value below 2^-14 is off by up to 2^-25. P uses fp16's range whole:
// weights are taken relative to the running maximum less 7 (base 2), so that, with the
// lazy maximum's 8, P <= 2^15, and fp16's least step is 2^-31 of the row's largest weight
// or less. (Relative to the maximum itself the step was 2^-24: 2^18 tokens 17.4 nats below
// one other were left out.) What remains is the fp32 sum itself: 2^17 tokens behind one of
// the same value and 2^21 / 2^23 times their weight lose 2 / 10 % of their share to it,
// 2^27 times all (the absorbed form, whose sums are cut over CTAs, 0 / 0 / 0.6 %).
//
// TMEM (512 columns): S_t, P_t over it, at 64 t; q_n of tile t (the A operand of 16
// of S's 20 instructions: half the shared-memory reads) at 128 + 64 t; O_t at 256 +
// 128 t. Shared memory: q_r (32 KB) and a ring of 64-token stages [K_hi | K_lo | r | V].
//   warps 0-3 / 4-7  softmax of query tile 0 / 1: thread r owns row r; online softmax
//                    base 2, the maximum moves only by more than 8 (then the thread
//                    rescales its O row); weights over the first columns of S.
//   warp 8           TMA producer;  warp 9  MMA issuer and TMEM owner.
// Tile 0's products run while tile 1's softmax does, and the other way round.
//
// What bounds it: the tensor pipe, 2 x 20 score and 2 x 4 value instructions a 64-token
// stage: 2064 cycles of the 2450 a stage takes (4 requests, 1024 queries each at 4K-12K
// tokens, 32 heads: 614 us, the pipe 68 % busy, with the last wave's tail). The rest is
// the hand-off from a tile's softmax to its next products. An issuing warp a tile
// instead of one for both let the tiles' instructions interleave: 12 % slower.
//
// Tokens past the last row's limit are masked by selection, and their V rows zeroed
// in shared memory (0 * NaN). Every wait is bounded; one that gives up sets
// KF_DEVERR_TIMEOUT and the CTA drains its copies and MMAs and frees its TMEM.
#include <algorithm>

#include "kf_latent_expanded.cuh"

namespace kf {
namespace {

using namespace tc;
using namespace mq5;

constexpr int kRows = 128, kTok = 64;
constexpr int kProducerWarp = 8, kIssuerWarp = 9, kThreads = 320;
constexpr float kLift = 7.f;  // weights are 2^(score - maximum + kLift)
static_assert(kLift + kRescaleSlack <= 15.f, "weights within fp16's range");

template <int DN, int DV>
struct EShape {
    static constexpr int kQBytes = 2 * kRows * 128;              // q_r of both tiles
    static constexpr int kKAtoms = 2 * DN / 64;                  // hi, then lo
    static constexpr int kAtomBytes = kTok * 128;
    static constexpr int kRopeAt = kKAtoms * kAtomBytes;
    static constexpr int kVAt = kRopeAt + kAtomBytes;
    static constexpr int kStageBytes = kVAt + DV / 64 * kAtomBytes;
    static constexpr int kStages = DN == 128 ? 3 : 5;
    static constexpr int kSmemBytes = kQBytes + kStages * kStageBytes + 1024;
    static_assert(kSmemBytes > 116 * 1024 && kSmemBytes <= 227 * 1024, "one CTA an SM");
    __host__ __device__ static constexpr uint32_t col_s(int t) { return 64u * t; }
    __host__ __device__ static constexpr uint32_t col_q(int t) { return 128u + 64u * t; }
    __host__ __device__ static constexpr uint32_t col_o(int t) { return 256u + 128u * t; }
};

template <int DN, int DV>
__global__ void __launch_bounds__(kThreads, 1)
expanded_kernel(const LatentParams p, const ExpandedKV kv, int q_tiles, const __grid_constant__ CUtensorMap tmap_q,
                const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                const __grid_constant__ CUtensorMap tmap_r) {
    using Sh = EShape<DN, DV>;
    constexpr int NS = Sh::kStages;
    // full[NS], empty[NS], q_ready, fin, s_full[2], p_full[2]
    __shared__ __align__(8) uint64_t bar_mem[2 * NS + 6];
    __shared__ uint32_t tmem_slot;
    __shared__ int sm_len[kThreads], sm_b;
    __shared__ volatile int abort_flag;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t sQ = base, sKV = base + Sh::kQBytes;
    const uint32_t bars = smem_u32(bar_mem);
    auto full = [&](uint32_t i) { return bars + 8u * i; };
    auto empty = [&](uint32_t i) { return bars + 8u * (NS + i); };
    const uint32_t q_ready = bars + 8u * (2 * NS), fin = q_ready + 8;
    auto s_full = [&](int t) { return fin + 8u + 8u * t; };
    auto p_full = [&](int t) { return fin + 24u + 8u * t; };
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    // Blocks start in index order, so the longest work comes first: the requests by
    // descending length (as far as one a thread can sort them), and in a request the later
    // query tiles, which see more tokens. Four requests of 4K-12K tokens, 512 blocks:
    // unsorted, the last blocks ran a third longer than the average SM.
    const int qg = q_tiles - 1 - (int)(blockIdx.x % q_tiles);
    const int h = blockIdx.x / q_tiles;
    int b = blockIdx.y;
    if (p.batch > 1 && p.batch <= kThreads) {
        const int t = threadIdx.x;
        if (t < p.batch) sm_len[t] = p.ctx_lens[t];
        __syncthreads();
        if (t < p.batch) {
            int before = 0;
            for (int i = 0; i < p.batch; ++i) before += sm_len[i] > sm_len[t] || (sm_len[i] == sm_len[t] && i < t);
            if (before == (int)blockIdx.y) sm_b = t;
        }
        __syncthreads();
        b = sm_b;
    }
    const int H = p.num_heads;
    const LatentRequest rq = latent_request(p, b, threadIdx.x == 0 && blockIdx.x == 0);
    // Every path waits for the expansion once, those with nothing to do as well: a grid that
    // no thread waits in could end before it, and what follows in the stream begin.
    auto expansion_done = [] { asm volatile("griddepcontrol.wait;" ::: "memory"); };
    if (rq.q0 < 0) {
        expansion_done();
        return;
    }
    const int64_t C = rq.C < p.max_query_len ? rq.C : p.max_query_len;
    const int64_t L = rq.L < p.max_context_len ? rq.L : p.max_context_len;
    const int64_t shift = rq.L - rq.C;  // query j sees tokens [0, min(shift + j + 1, L))
    const int64_t row0 = (int64_t)qg * 2 * kRows;
    if (row0 >= C) {
        expansion_done();
        return;
    }
    const int64_t nrows = C - row0 < 2 * kRows ? C - row0 : 2 * kRows;
    const int nqt = nrows > kRows ? 2 : 1;
    int64_t t_end = L;
    if (p.causal && shift + row0 + nrows < t_end) t_end = shift + row0 + nrows;

    const int tq = warp >> 2, r = threadIdx.x & (kRows - 1);
    const int64_t row = row0 + (int64_t)tq * kRows + r;
    const bool row_ok = warp < 8 && row < C;
    const int64_t at = (rq.q0 + (row_ok ? row : 0)) * H + h;  // (token, head) index of this thread's row

    if (t_end <= 0) {
        expansion_done();
        if (row_ok) {
            for (int i = 0; i < DV; ++i) {
                if (p.out_dtype == KF_F32) static_cast<float *>(p.out)[at * DV + i] = 0.f;
                else static_cast<uint16_t *>(p.out)[at * DV + i] = 0;
            }
            if (p.lse_out) p.lse_out[at] = -INFINITY;
        }
        return;
    }
    const int ntiles = (int)((t_end + kTok - 1) / kTok);
    // the expansion's keys and values are complete from here on (its inputs, which this
    // kernel read above, were so before it started)
    expansion_done();

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        mbar_init(q_ready, 1 + nqt * kRows);  // the q_r boxes, and q_n's rows in TMEM
        mbar_init(fin, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full(t), 1);
            mbar_init(p_full(t), kRows);
        }
        abort_flag = (*(volatile unsigned int *)p.err & KF_DEVERR_TIMEOUT) ? 1 : 0;  // an earlier kernel's wait
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kIssuerWarp) tc05::tmem_alloc(smem_u32(&tmem_slot), 512);
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    const uint32_t tm = tmem_slot;

    if (warp == kProducerWarp) {
        // ------------------------------ producer ------------------------------
        const int bs_shift = block_shift(p.block_size);
        const uint32_t rope_bytes = (uint32_t)p.block_size * 128;
        const int64_t ws_row = (int64_t)h * kv.rows + b * kv.cap;
        if (lane == 0) {
            mbar_arrive_expect_tx(q_ready, (uint32_t)nqt * kRows * 128);
            for (int t = 0; t < nqt; ++t)
                tma_load_4d(sQ + t * kRows * 128, &tmap_q, 0, h, (int)(rq.q0 + row0 + t * kRows), DN / 64, q_ready);
        }
        __syncwarp();
        int last = -1;
        for (int j = 0; j < ntiles; ++j) {
            const uint32_t st = j % NS;
            const int64_t t0 = (int64_t)j * kTok;
            const int ntok = t_end - t0 < kTok ? (int)(t_end - t0) : kTok;
            const int nblk = (ntok + p.block_size - 1) >> bs_shift;
            int64_t phys = 0;
            if (lane < nblk) {
                phys = p.block_tables[(int64_t)b * p.bt_stride + (t0 >> bs_shift) + lane];
                if (phys < 0 || phys >= p.num_blocks) {  // reported where the keys were built, too
                    raise_error(p.err, KF_DEVERR_BLOCK_ID);
                    phys = 0;
                }
            }
            int go = 1;
            if (lane == 0) {
                go = !abort_flag && mbar_wait(empty(st), ((j / NS) & 1) ^ 1);
                if (go) {
                    mbar_arrive_expect_tx(full(st), (Sh::kKAtoms + DV / 64) * Sh::kAtomBytes + nblk * rope_bytes);
                    tc05::tma_load_3d(sKV + st * Sh::kStageBytes, &tmap_k, 0, (int)(ws_row + t0), 0, full(st));
                    tc05::tma_load_3d(sKV + st * Sh::kStageBytes + Sh::kVAt, &tmap_v, 0, (int)(ws_row + t0), 0, full(st));
                } else {
                    raise_error(p.err, KF_DEVERR_TIMEOUT);
                    abort_flag = 1;
                }
            }
            if (!__shfl_sync(0xffffffffu, go, 0)) break;
            if (lane < nblk)
                tma_load_4d(sKV + st * Sh::kStageBytes + Sh::kRopeAt + lane * rope_bytes, &tmap_r, 0, 0,
                            p.latent_dim / 64, (int)(phys * (p.block_size / 8)), full(st));
            __syncwarp();
            last = j;
        }
        if (lane == 0) {
            // drain: the last use of every stage has landed before the CTA can exit
            for (int j = last - NS + 1 > 0 ? last - NS + 1 : 0; j <= last; ++j)
                if (!mbar_wait(full(j % NS), (j / NS) & 1)) raise_error(p.err, KF_DEVERR_TIMEOUT);
            if (!mbar_wait(q_ready, 0)) raise_error(p.err, KF_DEVERR_TIMEOUT);
        }
        __syncwarp();
    } else if (warp == kIssuerWarp) {
        // ------------------------------ MMA issuer -----------------------------
        // Step j: for each query tile t, once its softmax of stage j - 1 is done,
        // O_t += P_t V_{j-1} and then S_t of stage j (issue order keeps S_t's writes
        // behind PV's reads of P_t).
        const uint32_t id_s = tc05::idesc_bf16(kRows, kTok, false, false);
        const uint32_t id_o = tc05::idesc_f16(kRows, DV, false, true);
        bool ok = warp_wait(q_ready, 0);
        for (int j = 0; ok && j <= ntiles; ++j) {
            const bool has_s = j < ntiles, has_pv = j > 0;
            const uint32_t st = j % NS, pst = (j + NS - 1) % NS;
            const uint64_t kd = tc05::sdesc_sw128(sKV + st * Sh::kStageBytes, 16, 1024);
            const uint64_t vd = tc05::sdesc_sw128(sKV + pst * Sh::kStageBytes + Sh::kVAt, Sh::kAtomBytes, 1024);
            for (int t = 0; t < nqt; ++t) {
                const uint32_t s = tm + Sh::col_s(t), q = tm + Sh::col_q(t);
                if (has_pv) {
                    ok = warp_wait(p_full(t), (j - 1) & 1);
                    if (!ok) break;
                    tc05::fence_after_sync();
                    if (tc05::elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < kTok / 16; ++kk)
                            tc05::mma_ts(tm + Sh::col_o(t), s + 8 * kk, vd + (uint64_t)(kk * 2048 / 16), id_o,
                                         (j > 1 || kk > 0) ? 1u : 0u);
                        if (t == nqt - 1) tc05::commit(empty(pst));
                    }
                    __syncwarp();
                }
                // (the stage has nearly always landed: its wait runs under the value product)
                if (t == 0 && has_s) {
                    ok = !__any_sync(0xffffffffu, abort_flag) && warp_wait(full(st), (j / NS) & 1);
                    if (!ok) break;
                    tc05::fence_after_sync();
                }
                if (has_s) {
                    const uint64_t qd = tc05::sdesc_sw128(sQ + t * kRows * 128, 16, 1024);
                    if (tc05::elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 2 * DN / 16; ++kk)  // q_n against hi, then against lo
                            tc05::mma_ts(s, q + 8 * (kk % (DN / 16)),
                                         kd + (uint64_t)(((kk >> 2) * Sh::kAtomBytes + 32 * (kk & 3)) / 16), id_s,
                                         kk > 0 ? 1u : 0u);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc05::mma_ss(s, qd + (uint64_t)(32 * kk / 16),
                                         kd + (uint64_t)((Sh::kRopeAt + 32 * kk) / 16), id_s, 1u);
                        tc05::commit(s_full(t));
                    }
                    __syncwarp();
                }
            }
        }
        if (tc05::elect_one()) {
            if (!ok) {
                raise_error(p.err, KF_DEVERR_TIMEOUT);
                abort_flag = 1;
            }
            tc05::commit(fin);  // every MMA has completed before TMEM is freed
            if (!mbar_wait(fin, 0)) raise_error(p.err, KF_DEVERR_TIMEOUT);
        }
        __syncwarp();
    } else if (tq < nqt) {
        // ------------------------------- softmax --------------------------------
        const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t col_s = Sh::col_s(tq), col_o = Sh::col_o(tq);
        {  // q_n: two bf16 a column, as the MMA reads A from TMEM
            const uint16_t *q = p.q + at * (DN + kRopeDim);
#pragma unroll
            for (int c = 0; c < DN / 2; c += 32) {
                uint32_t x[32];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint4 v = row_ok ? __ldg(reinterpret_cast<const uint4 *>(q + 2 * c) + i) : make_uint4(0, 0, 0, 0);
                    x[4 * i] = v.x;
                    x[4 * i + 1] = v.y;
                    x[4 * i + 2] = v.z;
                    x[4 * i + 3] = v.w;
                }
                tc05::tmem_st32(tm + lane_base + Sh::col_q(tq) + c, x);
            }
            tc05::fence_before_sync();
            mbar_arrive(q_ready);
        }
        int64_t lim = row_ok ? (p.causal && shift + row + 1 < t_end ? shift + row + 1 : t_end) : 0;
        if (lim < 0) lim = 0;
        const float c = p.scale_log2;
        float m = -INFINITY, l = 0.f;  // the running maximum less kLift; the weights' sum
        bool ok = true;
        for (int j = 0; j < ntiles; ++j) {
            const int64_t t0 = (int64_t)j * kTok;
            // (the flag is read warp-uniformly: tcgen05.ld/st need the whole warp)
            if (__any_sync(0xffffffffu, abort_flag != 0) || !warp_wait(s_full(tq), j & 1)) {
                ok = false;
                break;
            }
            tc05::fence_after_sync();
            uint32_t x[64];
            tc05::tmem_ld64(tm + lane_base + col_s, x);
            const int ntok = t_end - t0 < kTok ? (int)(t_end - t0) : kTok;
            if (ntok < kTok) {  // zero the V rows past the range (each tile's warps zero all of them)
                const uint32_t vb = sKV + (j % NS) * Sh::kStageBytes + Sh::kVAt;
                for (int i = r; i < (kTok - ntok) * (DV / 8); i += kRows) {
                    const int t = ntok + i / (DV / 8), ch = i % (DV / 8);
                    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vb + (ch >> 3) * Sh::kAtomBytes +
                                                                                    t * 128 + (ch & 7) * 16),
                                 "r"(0u)
                                 : "memory");
                }
                fence_proxy_async_smem();
            }
            const int64_t nv64 = lim - t0;
            const int nv = nv64 <= 0 ? 0 : (nv64 >= kTok ? kTok : (int)nv64);
            // Fast path: every row of the warp sees the whole stage and the scale is
            // positive; otherwise scores are scaled and masked to -inf first.
            const bool fast = c > 0.f && __all_sync(0xffffffffu, nv == kTok);
            float mx = -INFINITY;
            if (fast) {
#pragma unroll
                for (int i = 0; i < 64; i += 2) mx = max3f(mx, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
                mx *= c;
            } else {
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    const float v = i < nv ? __uint_as_float(x[i]) * c : -INFINITY;
                    x[i] = __float_as_uint(v);
                    mx = fmaxf(mx, v);
                }
            }
            const bool need = mx > m + (kLift + kRescaleSlack);
            const float lifted = mx - kLift;
            const float alpha = need ? exp2f(m - lifted) : 1.f;  // m = -inf: 0
            if (need) {
                l *= alpha;
                m = lifted;
            }
            const float mu = m == -INFINITY ? 0.f : m;
            float2 ls = make_float2(0.f, 0.f);
            const float2 c2 = make_float2(c, c), nm = make_float2(-mu, -mu);
#pragma unroll
            for (int q2 = 0; q2 < 2; ++q2) {
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int e = 32 * q2 + 2 * i;
                    float2 a;
                    if (fast) a = fma_f32x2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), c2, nm);
                    else a = make_float2(__uint_as_float(x[e]) - mu, __uint_as_float(x[e + 1]) - mu);
                    a.x = ex2f(a.x);
                    a.y = ex2f(a.y);
                    ls = add_f32x2(ls, a);
                    pk[i] = pack_f16(a.x, a.y);
                }
                tc05::tmem_st16(tm + lane_base + col_s + 16 * q2, pk);
            }
            l += ls.x + ls.y;
            if (j > 0 && __any_sync(0xffffffffu, need)) {
                // O holds the products up to stage j - 1 (s_full of stage j came after
                // them); the next one waits for p_full below
#pragma unroll
                for (int cc = 0; cc < DV / 32; ++cc) {
                    uint32_t o[32];
                    tc05::tmem_ld32(tm + lane_base + col_o + 32 * cc, o);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                    tc05::tmem_st32(tm + lane_base + col_o + 32 * cc, o);
                }
            }
            tc05::fence_before_sync();
            mbar_arrive(p_full(tq));
        }
        if (ok && warp_wait(fin, 0)) {
            tc05::fence_after_sync();
            const float inv = l != 0.f ? 1.f / l : 0.f;  // (no token seen: 0; a NaN stays one)
#pragma unroll
            for (int cc = 0; cc < DV / 32; ++cc) {
                uint32_t o[32];
                tc05::tmem_ld32(tm + lane_base + col_o + 32 * cc, o);
                if (!row_ok) continue;
                float v[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = l != 0.f ? __uint_as_float(o[i]) * inv : 0.f;
                if (p.out_dtype == KF_F32) {
                    float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at * DV + 32 * cc);
#pragma unroll
                    for (int i = 0; i < 8; ++i) dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                } else {
                    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + at * DV + 32 * cc);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        dst[i] = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                                            pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
                }
            }
            if (row_ok && p.lse_out) p.lse_out[at] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
        } else {
            if (r == 0) raise_error(p.err, KF_DEVERR_TIMEOUT);
            abort_flag = 1;
        }
    }
    tc05::fence_before_sync();
    __syncthreads();
    if (warp == kIssuerWarp) {
        tc05::fence_after_sync();
        tc05::tmem_dealloc(tm, 512);
    }
}

// q [num_q_tokens, H, nope + 64] as (64 columns, head, token, column chunk): a box of
// 128 tokens of one head's rotary chunk.
bool encode_q_rope(tc::EncodeFn fn, CUtensorMap *map, const LatentParams &p, int nope) {
    const cuuint64_t head = (cuuint64_t)(nope + kRopeDim) * 2;
    const cuuint64_t dims[4] = {64, (cuuint64_t)p.num_heads, (cuuint64_t)p.num_q_tokens, head / 128};
    const cuuint64_t strides[3] = {head, head * p.num_heads, 128};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)kRows, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t *>(p.q), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DN, int DV>
cudaError_t launch(const LatentParams &p, const ExpandedKV &kv, bool behind_expand, cudaStream_t stream,
                   tc::EncodeFn fn) {
    using Sh = EShape<DN, DV>;
    const int64_t rows = (int64_t)p.num_heads * kv.rows;
    CUtensorMap mq, mk, mv, mr;
    if (!encode_q_rope(fn, &mq, p, DN) || !encode_rows(fn, &mk, kv.k, rows, 2 * DN, kTok, 2 * DN / 64) ||
        !encode_rows(fn, &mv, kv.v, rows, DV, kTok, DV / 64) || !encode_latent_cache(fn, &mr, p, 1))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done.load() & bit)) {
        e = cudaFuncSetAttribute(expanded_kernel<DN, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmemBytes);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit);
    }
    const int64_t q_tiles = ((int64_t)p.max_query_len + 2 * kRows - 1) / (2 * kRows);
    if (q_tiles * p.num_heads > 0x7fffffff) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(q_tiles * p.num_heads), p.batch);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Sh::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // set up while the expansion ends
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = behind_expand ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, expanded_kernel<DN, DV>, p, kv, (int)q_tiles, mq, mk, mv, mr);
}

int64_t token_cap(int max_context_len) { return ((int64_t)max_context_len + 127) / 128 * 128; }
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

size_t latent_expanded_workspace_bytes(int batch, int max_context_len, int num_heads, int nope, int v) {
    const size_t rows = (size_t)batch * token_cap(max_context_len) * num_heads;
    return align256(rows * 2 * nope * 2) + align256(rows * v * 2);
}

cudaError_t launch_latent_expanded(const LatentParams &p, const LatentWeights &w, void *workspace, int sm_count,
                                   cudaStream_t stream, void *encode_fn) {
    tc::EncodeFn fn = reinterpret_cast<tc::EncodeFn>(encode_fn);
    ExpandedKV kv;
    // (a bound of no tokens still needs valid tensor maps: one tile that is never read)
    kv.cap = std::max<int64_t>(token_cap(p.max_context_len), 128);
    kv.rows = p.batch * kv.cap;
    kv.k = static_cast<uint16_t *>(workspace);
    kv.v = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(workspace) +
                                        align256((size_t)kv.rows * p.num_heads * 2 * w.nope * 2));
    if (p.max_context_len > 0) {
        const cudaError_t e = launch_latent_expand(p, w, kv, sm_count, stream, fn);
        if (e != cudaSuccess) return e;
    }
    const bool behind = p.max_context_len > 0;
    return w.nope == 128 ? launch<128, 128>(p, kv, behind, stream, fn) : launch<64, 64>(p, kv, behind, stream, fn);
}

}  // namespace kf
