// kf_prompt.cu -- attention over whole prompts, packed end to end, on tcgen05.
//
//   S = scale Q K^T,  P = softmax rows (causal: key <= query),  O = P V
// per head and sequence, by tiles: 128 queries of one head against 128 keys.
//
// A unit is two query tiles that share their keys: the same 128 tokens of two heads of
// one KV head, or, without grouped heads, 256 tokens of one head. Units of all sequences
// are taken in descending order of their block's index in its sequence (those of a (sequence,
// token block) side by side, so that their keys and values meet in L2), CTA c of P taking the
// c-th of every P, forwards and backwards in turn. In a causal call that is the order of
// their keys, and the sums come out even; without the mask every block of a sequence costs the
// whole sequence, and they are less so. One CTA an SM walks its units without a pause: the
// next unit's loads and first scores run while the last one's rows are written out.
// A unit is found by reading the batch's ranges once and once more for each step of a search
// over the block index, which beyond some 500 sequences takes longer than short units do:
// 1024 prompts of 64 tokens, 8/2 heads, 0.21 ms, 4096 2.5 ms, 65535 of 4 tokens 0.55 s.
//
//   warps 0-3 / 4-7  softmax of query tile 0 / 1: thread r owns row r of 128 scores;
//                    online softmax base 2, the maximum moves only by more than
//                    8 (then the thread rescales its O row in TMEM); weights as bf16 pairs
//                    over the scores of each half, each half announced by itself, so that the
//                    value product starts while the second's exponentials run.
//   warp 8           TMA producer: one box a key or value tile (128 tokens x D);
//   warp 10          finds the CTA's units ahead (the lengths are on the device);
//   warp 11          waits for the loaded tiles on the issuer's behalf (feeder);
//   warps 12-15      write finished rows out, while the softmax warps go on;
//   warp 9           MMA issuer and TMEM owner: per key tile j and query tile t
//                      O_t += P_t V_{j-1}  (A = P_t from TMEM, B = V, MN-major)
//                      S_t  = Q_t K_j^T    (both K-major shared memory)
//                    tile 0's products run while tile 1's softmax does, and the other way round.
// TMEM: S_t at 128 t, its halves' weights at 128 t and 128 t + 64, O_t at 256 + D t.
//
// Precision: scores and sums fp32; weights enter the value product as bf16, v's type (half a
// step is 2^-8 of the weight; an output in bf16 rounds as much itself). An fp32 output takes
// them in three pieces (24 bits), three value products, the second and third summed apart: the
// tensor cores cut their fp32 sums off instead of rounding them, every 16 tokens and product
// (9 prompts of 1-1261 tokens, against 64 bits: 1.1e-6 in one sum, 4.2e-7 in two; one bf16 piece
// would be off by 1e-3, two by 1.8e-6). And every four key tiles the softmax warps add the sum to
// one of their own, rounded, and clear it: 16384 tokens are off by 6.5e-7 instead of 5.6e-6
// (plain fp32 5e-7) and take 5300 us instead of 5010; eight tiles: 1.0e-6, 5220.
//
// With 128 columns an fp32 output has no room in TMEM for two tiles and their low sums: one
// query tile a unit.
//
// Bound and measured (32/8 heads of 128, causal). A key tile of both query tiles is 2070 cycles
// of MMAs and takes 2900-3100: each tile's chain of score product, softmax (1700 cycles: 128
// exponentials a row at 4 cycles a warp instruction, maximum, packing) and hand-offs is longer
// than the other tile's products that hide it. One prompt of 16384 tokens 1312-1350 us (1.63-1.68
// PFLOP/s, 0.86 of the library's burst rate for a plain product), four of 4096 363, 16 of 1024 144
// (a unit's start and end are some 5000 cycles), 64 of 64 36, one of 16 8.2; 16384 tokens of 16/8 heads
// of 64 620; 16384 tokens into fp32 5300 (three value products, one tile). Loads by the feeder's
// arrivals 1334 us, by waits of the issuer 1403 (16 prompts of 1024: 144, 137). Uneven lengths, 16 of
// 299-4086 tokens: 413 us causal, 764 not (1300 and 1410 TFLOP/s). Tried without gain: weights announced by
// quarters, first weights on the old maximum, an issuer a query tile (10 % slower), one elected
// lane for waits and MMAs (3-10 % slower on short prompts).
//
// Tokens that a row must not see are masked by selection, and the value rows past the
// sequence zeroed in shared memory (0 * NaN). Every wait is bounded; one that gives up
// sets KF_DEVERR_TIMEOUT and the CTA drains its copies and MMAs and frees its TMEM.
#include <algorithm>

#include "kf_prompt.cuh"
#include "kf_row_tile.cuh"
#include "kf_wait.cuh"

namespace kf {
namespace {

using namespace rows;

constexpr int kRows = 128, kTok = 128;
constexpr int kProducerWarp = 8, kIssuerWarp = 9, kPlanWarp = 10, kFeedWarp = 11, kStoreWarp = 12, kThreads = 512;
constexpr int kPlanned = 4;  // units found ahead
constexpr int kFlush = 4;    // F32: key tiles that the tensor cores sum before their sum is set aside
// Registers a thread, once the four warpgroups (two of softmax, whose rows' 128 scores stay
// in registers) have shared out the 128 each that 512 threads start with.
constexpr int kSoftRegs = 176, kOtherRegs = 80;
static_assert(2 * kSoftRegs + 2 * kOtherRegs <= 4 * 128, "no more than the block starts with");

template <int D, bool F32>
struct PShape {
    static constexpr int kHalves = D / 64;
    static constexpr int kHalfBytes = 128 * 128;               // 128 rows x 64 columns
    static constexpr int kTileBytes = kHalves * kHalfBytes;
    // F32: the sums set aside lie in shared memory, [tile][column][row], or (D = 128) in the
    // second tile's score columns
    static constexpr int kAsideBytes = F32 && D == 64 ? 2 * D * 128 * 4 : 0;
    static constexpr int kNK = D == 128 ? 3 : F32 ? 4 : 6, kNV = D == 128 ? 2 : F32 ? 3 : 5;
    static constexpr int kAsideAt = (2 + kNK + kNV) * kTileBytes;
    static constexpr int kSmemBytes = kAsideAt + kAsideBytes + 1024;
    static_assert(kSmemBytes > 116 * 1024 && kSmemBytes <= 225 * 1024, "one CTA an SM");  // (+ 1.5 KB static)
    __host__ __device__ static constexpr uint32_t col_s(int t) { return 128u * t; }
    __host__ __device__ static constexpr uint32_t col_o(int t) { return 256u + (uint32_t)D * t; }
    // F32: the weights' low parts are summed by themselves (D = 128: in the second tile's place)
    __host__ __device__ static constexpr uint32_t col_lo(int t) { return 384u + 64u * t; }
};

// ---------------------------------------------------------------------------
// Units
// ---------------------------------------------------------------------------
struct Unit {
    int64_t first;   // the sequence's first token
    int n;           // its tokens
    int tok0[2];     // the tiles' first tokens in the sequence
    int head[2];
    int tiles[2];    // key tiles of each (0: no such tile; [0] is -1 behind the last unit)
    int kv_head;
};

// One query tile a unit: where the low parts of an fp32 output's sums take the second
// tile's place in TMEM.
__host__ __device__ constexpr bool single_tile(int head_dim, bool f32) { return f32 && head_dim == 128; }

struct Units {
    int block;       // tokens a unit
    int pairs;       // units a (sequence, token block)
    int total;
};

__device__ __forceinline__ int blocks_of(const PromptParams &p, int block, int b) {
    return (int)((sequence_of(p, b, false).n + block - 1) / block);
}

// Blocks at index i or above in their sequences. All lanes call it.
__device__ __forceinline__ int blocks_from(const PromptParams &p, int block, int i) {
    int n = 0;
    for (int b = threadIdx.x & 31; b < p.batch; b += 32) n += max(0, blocks_of(p, block, b) - i);
    return __reduce_add_sync(0xffffffffu, n);
}

__device__ __forceinline__ Units units_of(const PromptParams &p, bool single) {
    const bool grouped = p.num_q_heads > p.num_kv_heads;
    Units s;
    s.block = grouped || single ? kRows : 2 * kRows;
    s.pairs = grouped && !single ? p.num_q_heads / 2 : p.num_q_heads;
    s.total = blocks_from(p, s.block, 0) * s.pairs;
    return s;
}

// The i-th unit by descending block index. Whole warps call it.
__device__ __forceinline__ Unit unit_at(const PromptParams &p, const Units &s, bool single, int at) {
    const int lane = threadIdx.x & 31;
    const int place = at / s.pairs, pair = at - place * s.pairs;
    // the largest index i with more than `place` blocks at i or above
    int lo = 0, hi = (p.max_seq_len + s.block - 1) / s.block, above = 0;  // blocks_from(hi) = 0
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1, n = blocks_from(p, s.block, mid);
        if (n > place) {
            lo = mid;
        } else {
            hi = mid;
            above = n;
        }
    }
    // of the sequences with a block lo, the (place - above)-th
    int nth = place - above, b = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
        const bool has = b0 + lane < p.batch && blocks_of(p, s.block, b0 + lane) > lo;
        const unsigned int mask = __ballot_sync(0xffffffffu, has);
        const int n = __popc(mask);
        if (nth < n) {
            b = b0 + __fns(mask, 0, nth + 1);
            break;
        }
        nth -= n;
    }
    const Sequence q = sequence_of(p, b, false);
    Unit u;
    u.first = q.first;
    u.n = (int)q.n;
    const bool grouped = s.block == kRows;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        u.tok0[t] = lo * s.block + (grouped ? 0 : t * kRows);
        u.head[t] = grouped && !single ? 2 * pair + t : pair;
        const int end = p.causal ? min(u.n, u.tok0[t] + kRows) : u.n;
        u.tiles[t] = u.tok0[t] < u.n && !(single && t) ? (end + kTok - 1) / kTok : 0;
    }
    u.kv_head = u.head[0] / (p.num_q_heads / p.num_kv_heads);
    return u;
}

// CTA c's k-th unit: forwards and backwards in turn.
__device__ __forceinline__ int unit_index(int k) {
    const int P = gridDim.x, c = blockIdx.x;
    return k * P + ((k & 1) ? P - 1 - c : c);
}

// ---------------------------------------------------------------------------
// Kernel. F32: an fp32 output, weights in three pieces.
// ---------------------------------------------------------------------------
template <int D, bool F32>
__global__ void __launch_bounds__(kThreads, 1)
prompt_kernel(const PromptParams p, const __grid_constant__ CUtensorMap tmap_q,
              const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v) {
    using Sh = PShape<D, F32>;
    constexpr int NK = Sh::kNK, NV = Sh::kNV, NP = F32 ? 3 : 1;
    constexpr bool kSingle = single_tile(D, F32);
    // kfull[NK], kempty[NK], vfull[NV], vempty[NV], then two each of q_full, q_empty, s_full,
    // p_half, p_full, o_full, o_empty, l_full, w_free, then fin and u_full, u_empty[kPlanned]
    __shared__ __align__(8) uint64_t bar_mem[2 * (NK + NV) + 19 + 2 * kPlanned];
    // rows' 1 / sum, for the storing warps; F32: behind them the factors of the sums set aside
    __shared__ float sm_inv[F32 && !kSingle ? 4 : 2][kRows];
    constexpr int kKeep = kSingle ? 1 : 2;
    __shared__ Unit sm_unit[kPlanned];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t sQ = base, sK = sQ + 2 * Sh::kTileBytes, sV = sK + NK * Sh::kTileBytes;
    const uint32_t bars = smem_u32(bar_mem);
    auto kfull = [&](uint32_t i) { return bars + 8u * i; };
    auto kempty = [&](uint32_t i) { return bars + 8u * (NK + i); };
    auto vfull = [&](uint32_t i) { return bars + 8u * (2 * NK + i); };
    auto vempty = [&](uint32_t i) { return bars + 8u * (2 * NK + NV + i); };
    const uint32_t rest = bars + 8u * (2 * (NK + NV));
    auto q_full = [&](int t) { return rest + 8u * t; };
    auto q_empty = [&](int t) { return rest + 16u + 8u * t; };
    auto s_full = [&](int t) { return rest + 32u + 8u * t; };
    auto p_half = [&](int t) { return rest + 48u + 8u * t; };
    auto p_full = [&](int t) { return rest + 64u + 8u * t; };
    auto o_full = [&](int t) { return rest + 80u + 8u * t; };
    auto o_empty = [&](int t) { return rest + 96u + 8u * t; };
    auto l_full = [&](int t) { return rest + 112u + 8u * t; };
    auto w_free = [&](int t) { return rest + 128u + 8u * t; };  // F32: a half tile's weights have been read
    const uint32_t fin = rest + 144u;
    auto u_full = [&](uint32_t i) { return rest + 152u + 8u * i; };
    auto u_empty = [&](uint32_t i) { return rest + 152u + 8u * (kPlanned + i); };
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * (NK + NV); ++i) mbar_init(bars + 8u * i, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(q_full(t), 2);  // (the query tile, and the feeder for the first key tile)
            mbar_init(q_empty(t), 1);
            mbar_init(s_full(t), 1);
            mbar_init(p_half(t), 5);  // (a softmax warp arrives once, and the feeder)
            mbar_init(p_full(t), 4);
            mbar_init(o_full(t), 1);
            mbar_init(o_empty(t), 4);
            mbar_init(l_full(t), 4);
            mbar_init(w_free(t), 1);
        }
        mbar_init(fin, 1);
        for (int i = 0; i < kPlanned; ++i) {
            mbar_init(u_full(i), 1);
            mbar_init(u_empty(i), 15);  // the producer's, the issuer's, the feeder, eight softmax and four storing warps
        }
        abort_flag = (*(volatile unsigned int *)p.err & KF_DEVERR_TIMEOUT) ? 1 : 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (blockIdx.x == 0)  // bad ranges, reported once
        for (int b = threadIdx.x; b < p.batch; b += kThreads) sequence_of(p, b, true);
    if (warp == kIssuerWarp) tc05::tmem_alloc(smem_u32(&tmem_slot), 512);
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    const uint32_t tm = tmem_slot;
    // F32: where the sums set aside are
    auto aside_at = [&](int t, int r, int c) { return base + Sh::kAsideAt + (uint32_t)(((t * D + c) * kRows + r) * 4); };
    auto load_aside = [&](uint32_t tw, int t, int r, int cc, uint32_t (&v)[16]) {
        if (kSingle) {
            tmem_ld16(tw + Sh::col_s(1) + cc, v);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[i]) : "r"(aside_at(t, r, cc + i)) : "memory");
        }
    };
    auto warp_arrive = [&](uint32_t bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    // A wait that may last as long as a unit does; given up early if another role has (kf_wait.cuh).
    auto long_wait = [&](uint32_t bar, uint32_t parity) {
        KF_WAIT_IN_SLICES(__all_sync(0xffffffffu, mbar_wait(bar, parity, kPollsASlice)),
                          __any_sync(0xffffffffu, abort_flag != 0));
    };
    // The k-th unit of this CTA; false behind the last one, or where a wait gave up (`ok`).
    auto next_unit = [&](int k, Unit &u, bool &ok) {
        const uint32_t e = k % kPlanned;
        ok = ok && long_wait(u_full(e), (k / kPlanned) & 1);
        if (!ok) return false;
        u = sm_unit[e];
        __syncwarp();
        if (lane == 0) mbar_arrive(u_empty(e));
        return u.tiles[0] >= 0;
    };

    // (the three parts of the block are one if each: setmaxnreg is for whole warpgroups, and
    // what follows it is compiled for its count)
    if (warp >= 8 && warp < kStoreWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kPlanWarp) {
        // ------------------------------- planner --------------------------------
        const Units units = units_of(p, kSingle);
        for (int k = 0;; ++k) {
            const uint32_t e = k % kPlanned;
            const bool more = unit_index(k) < units.total;
            Unit u;
            if (more) u = unit_at(p, units, kSingle, unit_index(k));
            else u.tiles[0] = -1;
            if (!long_wait(u_empty(e), ((k / kPlanned) & 1) ^ 1)) {
                if (lane == 0) raise_error(p.err, KF_DEVERR_TIMEOUT);
                abort_flag = 1;
                break;
            }
            if (lane == 0) {
                sm_unit[e] = u;
                mbar_arrive(u_full(e));
            }
            __syncwarp();
            if (!more) break;
        }
    } else if (warp == kFeedWarp) {
        // -------------------------------- feeder --------------------------------
        // Waits for the key and value tiles in the issuer's place and adds its arrival to the
        // barrier that the issuer waits on anyway: a wait behind issued MMAs is served once the
        // tensor pipe has taken them, and a second one there leaves it idle. An arrival belongs
        // to one phase: the one before is over first.
        uint32_t kc = 0, vc = 0, qc[2] = {0, 0}, pc[2] = {0, 0};
        bool ok = true;
        Unit u;
        for (int k = 0; next_unit(k, u, ok); ++k) {
            const int n = max(u.tiles[0], u.tiles[1]);
            for (int j = 0; ok && j <= n; ++j) {
                if (j > 0) {
                    ok = long_wait(vfull(vc % NV), (vc / NV) & 1);
                    ++vc;
                }
                if (j < n) {
                    ok = ok && long_wait(kfull(kc % NK), (kc / NK) & 1);
                    ++kc;
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (!ok || j > u.tiles[t] || u.tiles[t] == 0) continue;
                    const uint32_t bar = j == 0 ? q_full(t) : p_half(t);
                    uint32_t &phase = j == 0 ? qc[t] : pc[t];
                    ok = long_wait(bar, (phase & 1) ^ 1);
                    if (ok && lane == 0) mbar_arrive(bar);
                    ++phase;
                }
                __syncwarp();
            }
        }
        if (!ok) {
            if (lane == 0) raise_error(p.err, KF_DEVERR_TIMEOUT);
            abort_flag = 1;
        }
    } else if (warp == kProducerWarp) {
        // ------------------------------ producer ------------------------------
        uint32_t kc = 0, vc = 0, qc[2] = {0, 0};  // loads so far
        bool ok = true;
        Unit u;
        for (int k = 0; next_unit(k, u, ok); ++k) {
            const int n = max(u.tiles[0], u.tiles[1]);
            if (lane == 0) {
                // the next unit's first tiles, into L2: its queries can only be loaded once
                // this one's last scores are there
                auto prefetch_next = [&]() {
                    const uint32_t e = (k + 1) % kPlanned;
                    if (!mbar_try_wait(u_full(e), ((k + 1) / kPlanned) & 1)) return;
                    const Unit &v = sm_unit[e];
                    for (int t = 0; t < 2; ++t)
                        if (v.tiles[0] >= 0 && v.tiles[t] > 0) prefetch_4d(&tmap_q, 0, v.head[t], (int)v.first + v.tok0[t], 0);
                };
                auto load_k = [&](int j) {
                    const uint32_t st = kc % NK;
                    if (abort_flag || !mbar_wait(kempty(st), ((kc / NK) & 1) ^ 1)) return false;
                    mbar_arrive_expect_tx(kfull(st), Sh::kTileBytes);
                    tma_load_4d(sK + st * Sh::kTileBytes, &tmap_k, 0, u.kv_head, (int)u.first + j * kTok, 0, kfull(st));
                    ++kc;
                    return true;
                };
                ok = load_k(0);
                for (int t = 0; t < 2 && ok; ++t) {
                    if (u.tiles[t] == 0) continue;
                    ok = !abort_flag && mbar_wait(q_empty(t), (qc[t] & 1) ^ 1);
                    if (!ok) break;
                    mbar_arrive_expect_tx(q_full(t), Sh::kTileBytes);
                    tma_load_4d(sQ + t * Sh::kTileBytes, &tmap_q, 0, u.head[t], (int)u.first + u.tok0[t], 0, q_full(t));
                    ++qc[t];
                }
                prefetch_next();
                for (int j = 0; j < n && ok; ++j) {
                    if (j > 0) ok = load_k(j);
                    const uint32_t st = vc % NV;
                    ok = ok && !abort_flag && mbar_wait(vempty(st), ((vc / NV) & 1) ^ 1);
                    if (!ok) break;
                    mbar_arrive_expect_tx(vfull(st), Sh::kTileBytes);
                    tma_load_4d(sV + st * Sh::kTileBytes, &tmap_v, 0, u.kv_head, (int)u.first + j * kTok, 0, vfull(st));
                    ++vc;
                }
                if (!ok) {
                    raise_error(p.err, KF_DEVERR_TIMEOUT);
                    abort_flag = 1;
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        if (lane == 0) {
            // drain: the last use of every slot has landed before the CTA can exit
            bool done = true;
            for (uint32_t i = kc > NK ? kc - NK : 0; i < kc; ++i) done = mbar_wait(kfull(i % NK), (i / NK) & 1) && done;
            for (uint32_t i = vc > NV ? vc - NV : 0; i < vc; ++i) done = mbar_wait(vfull(i % NV), (i / NV) & 1) && done;
            for (int t = 0; t < 2; ++t)
                if (qc[t] > 0) done = mbar_wait(q_full(t), (qc[t] - 1) & 1) && done;
            if (!done) raise_error(p.err, KF_DEVERR_TIMEOUT);
        }
        __syncwarp();
    } else if (warp == kIssuerWarp) {
        // ------------------------------ MMA issuer -----------------------------
        // (whole warps wait, one elected lane issues: the descriptors then stay in uniform
        // registers)
        const uint32_t id_s = tc05::idesc_bf16(kRows, kTok, false, false);
        const uint32_t id_o = tc05::idesc_bf16(kRows, D, false, true);
        uint32_t kc = 0, vc = 0, qc[2] = {0, 0}, pc[2] = {0, 0};  // tiles used so far
        bool ok = true;
        Unit u;
        for (int k = 0; next_unit(k, u, ok); ++k) {
            const int n = max(u.tiles[0], u.tiles[1]);
            for (int j = 0; ok && j <= n; ++j) {
                const uint32_t kst = kc % NK, vst = vc % NV;
                const uint64_t kd = tc05::sdesc_sw128(sK + kst * Sh::kTileBytes, 16, 1024);
                const uint64_t vd = tc05::sdesc_sw128(sV + vst * Sh::kTileBytes, Sh::kHalfBytes, 1024);
                bool k_here = false, v_here = false;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const uint32_t s = tm + Sh::col_s(t), o = tm + Sh::col_o(t);
                    if (ok && j > 0 && j <= u.tiles[t]) {
                        v_here = true;
                        // the last unit's rows have been read out of O
                        if (ok && j == 1) ok = warp_wait(o_empty(t), (qc[t] & 1));
#pragma unroll
                        for (int half = 0; half < 2 && ok; ++half) {
                            ok = long_wait(half ? p_full(t) : p_half(t), pc[t] & 1);
                            if (!ok) break;
                            tc05::fence_after_sync();
                            if (tc05::elect_one()) {
#pragma unroll
                                for (int kk = 4 * half; kk < 4 * half + 4; ++kk) {
                                    const uint32_t w = s + (NP == 3 ? 0 : 64 * half) + 8 * (kk & 3);
#pragma unroll
                                    for (int i = 0; i < NP; ++i)
                                        tc05::mma_ts(i == 0 ? o : tm + Sh::col_lo(t), w + 32 * i,
                                                     vd + (uint64_t)(kk * 2048 / 16), id_o,
                                                     (j > 1 || kk > 0 || i > 1) ? 1u : 0u);
                                }
                                if (NP == 3 && !half) tc05::commit(w_free(t));
                                if (half && j == u.tiles[t]) tc05::commit(o_full(t));
                                if (half && (t == 1 || j > u.tiles[1])) tc05::commit(vempty(vst));
                            }
                            __syncwarp();
                        }
                        ++pc[t];
                    }
                    if (ok && j < u.tiles[t]) {
                        k_here = true;
                        if (ok && j == 0) {
                            ok = long_wait(q_full(t), qc[t] & 1);
                            ++qc[t];
                        }
                        if (!ok) break;
                        tc05::fence_after_sync();
                        const uint64_t qd = tc05::sdesc_sw128(sQ + t * Sh::kTileBytes, 16, 1024);
                        if (tc05::elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint64_t off = (uint64_t)(((kk >> 2) * Sh::kHalfBytes + 32 * (kk & 3)) / 16);
                                tc05::mma_ss(s, qd + off, kd + off, id_s, kk > 0 ? 1u : 0u);
                            }
                            tc05::commit(s_full(t));
                            if (j == u.tiles[t] - 1) tc05::commit(q_empty(t));
                            if (t == 1 || j >= u.tiles[1]) tc05::commit(kempty(kst));
                        }
                        __syncwarp();
                    }
                }
                if (v_here) ++vc;
                if (k_here) ++kc;
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
    }
    } else if (warp < 8) {
        // ------------------------------- softmax --------------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        const int t = warp >> 2, r = threadIdx.x & (kRows - 1);
        const uint32_t tw = tm + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t ts = tw + Sh::col_s(t), to = tw + Sh::col_o(t);
        const float c = p.scale_log2, cs = c > 0.f ? c : 1.f;  // (a scale of zero or less is applied first)
        uint32_t sc = 0, oc = 0;  // score tiles and units so far
        uint32_t vbase = 0;       // value tiles before this unit
        bool ok = true;
        Unit u;
        for (int k = 0; next_unit(k, u, ok); ++k) {
            const int tiles = u.tiles[t], row = u.tok0[t] + r;
            const bool row_ok = row < u.n;
            const int lim = !row_ok ? 0 : p.causal ? row + 1 : u.n;  // tokens this row sees
            float m = -INFINITY, l = 0.f;
            float aside = -INFINITY;  // F32: the maximum that the sums set aside are relative to
            for (int j = 0; j < tiles; ++j, ++sc) {
                const int t0 = j * kTok;
                // (the flag is read warp-uniformly: tcgen05.ld/st need the whole warp)
                if (!long_wait(s_full(t), sc & 1)) {
                    ok = false;
                    break;
                }
                tc05::fence_after_sync();
                if (u.n - t0 < kTok) {  // zero the value rows past the sequence (both tiles' warps zero all of them)
                    const uint32_t vi = vbase + j, vst = vi % NV;
                    if (!warp_wait(vfull(vst), (vi / NV) & 1)) {
                        ok = false;
                        break;
                    }
                    constexpr int kChunks = 8 * Sh::kHalves;  // 16-byte chunks a row
                    const uint32_t to_zero =
                        sV + vst * Sh::kTileBytes + (r / 8 % Sh::kHalves) * Sh::kHalfBytes + r % 8 * 16;
                    for (int tok = u.n - t0 + r / kChunks; tok < kTok; tok += kRows / kChunks)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(to_zero + tok * 128), "r"(0u)
                                     : "memory");
                    fence_proxy_async_smem();
                }
                uint32_t x[2][64];
                if (F32 && j > 0 && j % kFlush == 0) {  // O, complete up to the tile before, is set aside
                    const float keep = aside == m ? 1.f : exp2f(aside - m);
                    aside = m;
                    const uint32_t zero[16] = {};
#pragma unroll 1
                    for (int cc = 0; cc < D; cc += 16) {
                        uint32_t o[16], v[16];
                        tmem_ld16(to + cc, o);
                        if (j > kFlush) load_aside(tw, t, r, cc, v);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (j > kFlush) o[i] = __float_as_uint(fmaf(__uint_as_float(v[i]), keep, __uint_as_float(o[i])));
                        if (kSingle) {
                            tmem_st16_async(tw + Sh::col_s(1) + cc, o);
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                asm volatile("st.shared.u32 [%0], %1;" ::"r"(aside_at(t, r, cc + i)), "r"(o[i]) : "memory");
                        }
                        tmem_st16_async(to + cc, zero);
                    }
                    tmem_wait_st();
                }
                tmem_ld64_async(ts, x[0]);
                tmem_ld64_async(ts + 64, x[1]);
                tmem_landed(x[0]);
                tmem_landed(x[1]);
                if (!(c > 0.f)) {  // (the maximum below is one of unscaled scores)
#pragma unroll
                    for (int i = 0; i < 128; ++i)
                        x[i >> 6][i & 63] = __float_as_uint(__uint_as_float(x[i >> 6][i & 63]) * c);
                }
                // Columns by 32: those all rows of the warp see, those some see (on a tile's
                // diagonal, or at the sequence's end), those none sees.
                const int nv = lim - t0;
                int most = kTok;
                if (!__all_sync(0xffffffffu, nv >= kTok)) {
                    most = __reduce_max_sync(0xffffffffu, nv);
                    const int least = __reduce_min_sync(0xffffffffu, nv);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (least >= 32 * q + 32) continue;
#pragma unroll
                        for (int i = 32 * q; i < 32 * q + 32; ++i)
                            if (i >= nv) x[i >> 6][i & 63] = 0xff800000u;  // -inf
                    }
                }
                ok = row_tile<D, NP, false>(
                    ts, to, F32 ? tw + Sh::col_lo(t) : 0, x, most, cs, j > 0, m, l,
                    [&](int half) { warp_arrive(half ? p_full(t) : p_half(t)); },
                    [&] { return long_wait(w_free(t), sc & 1); });
                if (!ok) break;
            }
            vbase += max(u.tiles[0], u.tiles[1]);
            if (!ok || tiles == 0) continue;
            // (the last unit's have been read)
            if (!warp_wait(o_empty(t), (oc & 1) ^ 1)) {
                ok = false;
                continue;
            }
            sm_inv[t][r] = l != 0.f ? 1.f / l : 0.f;
            if (F32) sm_inv[kKeep + t][r] = aside == m ? 1.f : exp2f(aside - m);
            warp_arrive(l_full(t));
            if (row_ok && p.lse_out)
                p.lse_out[(u.first + row) * p.num_q_heads + u.head[t]] = (m + log2f(l)) * 0.6931471805599453f;
            ++oc;
        }
        if (!ok) {
            if (lane == 0) raise_error(p.err, KF_DEVERR_TIMEOUT);
            abort_flag = 1;
        }
    } else {
        // ------------------------------- rows out -------------------------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        const int r = threadIdx.x & (kRows - 1);
        const uint32_t tw = tm + ((uint32_t)(32 * (warp & 3)) << 16);
        const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
        uint32_t oc[2] = {0, 0};
        bool ok = true;
        Unit u;
        for (int k = 0; next_unit(k, u, ok); ++k) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (!ok || u.tiles[t] == 0) continue;
                ok = long_wait(l_full(t), oc[t] & 1) && long_wait(o_full(t), oc[t] & 1);
                if (!ok) continue;
                ++oc[t];
                tc05::fence_after_sync();
                const float inv = sm_inv[t][r];
                const int row = u.tok0[t] + r;
                const bool row_ok = row < u.n;
                const int64_t at = (u.first + row) * p.num_q_heads + u.head[t];
                if (F32) {
                    float *const dst = static_cast<float *>(p.out) + at * D;
                    const bool aside = u.tiles[t] > kFlush;
                    const float keep = sm_inv[kKeep + t][r];
#pragma unroll 1
                    for (int cc = 0; cc < D; cc += 16) {
                        uint32_t o[16], lo[16], v[16] = {};
                        tmem_ld16(tw + Sh::col_o(t) + cc, o);
                        tmem_ld16(tw + Sh::col_lo(t) + cc, lo);
                        if (aside) load_aside(tw, t, r, cc, v);
                        if (cc == D - 16) {
                            tc05::fence_before_sync();
                            warp_arrive(o_empty(t));
                        }
                        if (!row_ok) continue;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t w[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float x = __uint_as_float(o[8 * i + e]) + __uint_as_float(lo[8 * i + e]);
                                w[e] = __float_as_uint(fmaf(__uint_as_float(v[8 * i + e]), keep, x) * inv);
                            }
                            store32(dst + cc + 8 * i, w, wide);
                        }
                    }
                    continue;
                }
#pragma unroll
                for (int cc = 0; cc < D; cc += 32) {
                    uint32_t o[32];
                    tc05::tmem_ld32(tw + Sh::col_o(t) + cc, o);
                    if (cc == D - 32) {
                        tc05::fence_before_sync();
                        warp_arrive(o_empty(t));
                    }
                    if (!row_ok) continue;
                    uint16_t *dst = static_cast<uint16_t *>(p.out) + at * D + cc;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            w[e] = pack_bf16(__uint_as_float(o[16 * i + 2 * e]) * inv,
                                             __uint_as_float(o[16 * i + 2 * e + 1]) * inv);
                        store32(dst + 16 * i, w, wide);
                    }
                }
            }
        }
        if (!ok) {
            if (lane == 0) raise_error(p.err, KF_DEVERR_TIMEOUT);
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

// x [num_tokens, heads, D] bf16, tokens `stride` elements apart, as (64 columns, head, token,
// column half): a box of 128 tokens of one head lands as halves of 128 rows of 128
// swizzled bytes.
bool encode_tokens(tc::EncodeFn fn, CUtensorMap *map, const uint16_t *x, int64_t stride, int heads, int D, int tokens) {
    const cuuint64_t dims[4] = {64, (cuuint64_t)heads, (cuuint64_t)tokens, (cuuint64_t)D / 64};
    const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2, 128};
    const cuuint32_t box[4] = {64, 1, 128, (cuuint32_t)D / 64};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t *>(x), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool F32>
cudaError_t launch(const PromptParams &p, int ctas, cudaStream_t stream, const CUtensorMap &mq, const CUtensorMap &mk,
                   const CUtensorMap &mv) {
    using Sh = PShape<D, F32>;
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done.load() & bit)) {
        e = cudaFuncSetAttribute(prompt_kernel<D, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmemBytes);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit);
    }
    prompt_kernel<D, F32><<<ctas, kThreads, Sh::kSmemBytes, stream>>>(p, mq, mk, mv);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt(const PromptParams &p, int sm_count, cudaStream_t stream, void *encode_fn) {
    tc::EncodeFn fn = reinterpret_cast<tc::EncodeFn>(encode_fn);
    CUtensorMap mq, mk, mv;
    if (!encode_tokens(fn, &mq, p.q, p.q_stride, p.num_q_heads, p.head_dim, p.num_tokens) ||
        !encode_tokens(fn, &mk, p.k, p.k_stride, p.num_kv_heads, p.head_dim, p.num_tokens) ||
        !encode_tokens(fn, &mv, p.v, p.v_stride, p.num_kv_heads, p.head_dim, p.num_tokens))
        return cudaErrorInvalidValue;
    // no more units than the tokens and the bound allow
    const bool grouped = p.num_q_heads > p.num_kv_heads;
    const bool single = single_tile(p.head_dim, p.out_dtype == KF_F32);
    const int64_t block = grouped || single ? kRows : 2 * kRows;
    const int64_t pairs = grouped && !single ? p.num_q_heads / 2 : p.num_q_heads;
    const int64_t blocks = std::min<int64_t>(p.batch * ((p.max_seq_len + block - 1) / block),
                                             p.num_tokens / block + std::min(p.batch, p.num_tokens));
    const int ctas = (int)std::min<int64_t>(blocks * pairs, sm_count);
    const bool f32 = p.out_dtype == KF_F32;
    if (p.head_dim == 128)
        return f32 ? launch<128, true>(p, ctas, stream, mq, mk, mv) : launch<128, false>(p, ctas, stream, mq, mk, mv);
    return f32 ? launch<64, true>(p, ctas, stream, mq, mk, mv) : launch<64, false>(p, ctas, stream, mq, mk, mv);
}

}  // namespace kf
