// kf_tree.cu -- attention for trees of drafted tokens over a paged cache, on tcgen05.
//
// Row (node i, head g of a KV head's group) sees the context, node i and its ancestors:
//   S = scale Q K^T,  P = softmax over what the row sees,  O = P V.
// The rows of a (request, KV head) share its keys and values: node i's rows are
// G i .. G i + G - 1, contiguous in q, and 256 of them at a time are a unit.
//
// Work. Tokens come in tiles of 128. The units' tiles, laid end to end, are cut into equal
// runs, one a CTA, one CTA an SM; the parts of a unit that is cut go to the workspace as
// normalised (o, lse) and a second kernel joins them (kf_runs.cuh). A unit's two query tiles
// of 128 rows are two streams over its tiles; with 128 rows or fewer the streams are its even
// and its odd tiles, joined when the rows are written out. Either way two softmaxes are under
// way, which the cache's bytes need: one alone takes 2900 cycles a tile (score product,
// softmax, value product and their hand-offs), an SM's share of HBM brings one in 1400.
//
//   warps 0-3 / 4-7  softmax of stream 0 / 1: thread r owns row r (kf_row_tile.cuh). Tiles
//                    before the tree need no mask; in the others a thread walks up its node's
//                    parents and sets a bit for each ancestor in the tile.
//   warps 9, 11      issue S_t = Q_t K^T and O_t += P_t V of stream 0 / 1 (S_t at TMEM column
//                    128 t, O_t at 256 + D t);
//   warps 8, 10      TMA producers (keys, values): one box a cache block; warp 10 also finds the
//                    run's parts ahead;
//   warps 12-15      write finished rows out; for E4M3 caches they also widen the codes.
//
// E4M3: the score product takes the keys' codes as they are (kind::f8f6f4) against q as the sum
// of two E4M3 numbers, scaled by a power of two a row; warps 12-15 widen the values' codes to
// fp16 (exact), the type of the weights. The scales multiply scores and output. Widening keys as
// well, for fp16 products of the same cost, took 48 KB more shared-memory traffic a tile.
//
// Precision: scores and sums fp32; weights enter the value product as bf16 (2^-8 of the
// weight at most) or fp16 (2^-11; relative to the maximum less 7, which uses the type's range
// whole); an fp32 output takes them in three pieces of bf16 or two of fp16, as many products
// into one sum, which the tensor cores cut off at every step. Every four tiles the softmax warps
// add it to one of their own, rounded, and clear it. TMEM and shared memory are full, so that sum
// lies in the workspace, a quad of columns of all rows at a time. 64 requests of 4096, 16384 or
// 65536 tokens, 16 nodes, are off by 2.0e-6 (E4M3 1.7e-6) against 64 bits, where one sum a run
// was off by 6e-6, 2.2e-5 and 8e-5; 4096 tokens take 282 us instead of 228 (E4M3 245, 190), 16384 tokens
// 1007 instead of 815. Every eight tiles: 3.6e-6, 947 us.
//
// Bound and measured (32/8 heads of 128). bf16 caches: HBM; 64 requests of 3.5-4K tokens and 16
// nodes 172 us, 0.88 of the measured copy rate (0.95 where contexts of 1K-32K are long enough to
// hide the start and the merge); 61 nodes 248, one request of 32K 38.6, 24/24 heads of 64 282.
// E4M3 caches: 64 of 1K-64K tokens, 32 nodes 520 us, 0.55 of HBM: two streams of 128 rows finish a
// tile each in some 5000 cycles (scores, softmax, widening, value product, hand-offs; 389 tiles a
// CTA), a part's start and end among them; 64 of 3.5-4K, 16 nodes 147. Eight requests of 2-16K, 61
// nodes, 64/8 heads 128 us, half of the tensor rate: 488 rows are two units of 256, whose second
// is not full, and a softmax tile is longer than its products. One issuer for both streams took
// 179 us instead of 172 and 163 instead of 128.
//
// What a row must not see is masked by selection, and value rows past the context are zeroed
// in shared memory (0 * NaN). Every wait is bounded; one that gives up sets
// KF_DEVERR_TIMEOUT and the CTA drains its copies and MMAs and frees its TMEM.
#include <algorithm>
#include <type_traits>

#include "kf_row_tile.cuh"
#include "kf_runs.cuh"
#include "kf_tree.cuh"
#include "kf_wait.cuh"

namespace kf {
namespace {

using namespace rows;

constexpr int kRows = 128, kTok = 128;
// Rows a unit: two query tiles; one where the room of the other holds widened tiles.
__host__ __device__ constexpr int unit_rows(bool kv8) { return kv8 ? kRows : 2 * kRows; }
constexpr int kLoadWarp = 8, kIssuerWarp = 9, kPlanWarp = 10, kIssuerWarp2 = 11, kStoreWarp = 12, kThreads = 512;
constexpr int kPlanned = 2;  // parts found ahead
constexpr int kFlush = 4;    // fp32 outputs: a stream's tiles that the tensor cores sum before their sum is set aside
// Registers a thread, once the four warpgroups have shared out the 128 each that 512
// threads start with: the softmax ones hold a row's 128 scores.
constexpr int kSoftRegs = 176, kOtherRegs = 80;
static_assert(2 * kSoftRegs + 2 * kOtherRegs <= 4 * 128, "no more than the block starts with");

// One part of a run: tiles [tile0, tile0 + n) of a unit.
struct Part {
    int n;  // -1 behind the last
    int tile0, b, head, q0, node0, rows, C, L;
    int slot;  // of the workspace, or -1: the unit lies in this run alone
};

template <int D, bool KV8>
struct TShape {
    static constexpr int kHalves = D / 64;
    static constexpr int kAtomBytes = kHalves * 1024;          // 8 tokens x D, 16 bits
    static constexpr int kTileBytes = kTok / 8 * kAtomBytes;
    static constexpr int kCodeBytes = kTok * D;                // a tile's codes
    static constexpr int kKBytes = KV8 ? kCodeBytes : kTileBytes;
    // (a value tile waits for its softmax, a key tile does not: one more of them)
    static constexpr int kNK = D == 128 ? (KV8 ? 4 : 2) : (KV8 ? 8 : 5);
    static constexpr int kNV = D == 128 ? (KV8 ? 2 : 3) : (KV8 ? 4 : 6);
    static constexpr int kNC = KV8 ? (D == 128 ? 4 : 6) : 0;  // tiles of value codes
    // full and empty of the three rings; two each of q_full, q_empty, s_full, p_half, p_full,
    // o_full, o_empty, l_full, w_free; fin; u_full, u_empty[kPlanned]
    static constexpr int kBars = 2 * (kNK + kNV + kNC) + 19 + 2 * kPlanned;
    static constexpr int kKAt = unit_rows(KV8) / kRows * kTileBytes, kVAt = kKAt + kNK * kKBytes;
    static constexpr int kCAt = kVAt + kNV * kTileBytes, kMlAt = kCAt + kNC * kCodeBytes;
    static constexpr int kBarsAt = kMlAt + 2 * kRows * 8, kPartsAt = kBarsAt + (kBars + 1) / 2 * 16;
    static constexpr int kEndAt = kPartsAt + kPlanned * 48;    // then the TMEM address and the abort flag
    static constexpr int kSmemBytes = kEndAt + 16;
    static_assert(sizeof(Part) <= 48 && 36 * 8 <= 2 * kRows * 8, "parts; the place search borrows m and l's room");
    static_assert(kSmemBytes > 116 * 1024 && kSmemBytes <= 227 * 1024, "one CTA an SM");
    __host__ __device__ static constexpr uint32_t col_s(int t) { return 128u * t; }
    __host__ __device__ static constexpr uint32_t col_o(int t) { return 256u + (uint32_t)D * t; }
};

// A unit cut over the CTAs i, i + 1, ...: its first part is in `slot0`, the others' in the
// first of their CTA's two slots.
struct Cut {
    int token, head, rows, parts, slot0;
};

struct Partials {
    float *o;    // [2 * CTAs][pitch][D]
    float *lse;  // [2 * CTAs][pitch]
    Cut *cuts;   // [CTAs]: the unit that starts in CTA i's run and goes on (parts = 0: none)
    int pitch;   // rows a slot holds
    // fp32 outputs: each CTA's two streams' sums set aside, [2 * CTAs][D / 4][kRows] quads of columns,
    // and the maxima that they are relative to, [2 * CTAs][kRows]
    float4 *sums;
    float *sums_m;
};

struct Request {
    TreeRequest r;
    int64_t n;  // tiles of each unit
    int groups, units;
};

__device__ __forceinline__ Request request_of(const TreeParams &p, int b, bool report) {
    Request q;
    q.r = tree_request(p.q_start, p.ctx_lens, b, p.num_q_tokens, p.max_query_len, p.max_context_len,
                       (int64_t)p.bt_stride * p.block_size, report ? p.err : nullptr);
    const int G = p.num_q_heads / p.num_kv_heads;
    const int unit = unit_rows(p.k_scale != nullptr);
    q.n = (q.r.L + kTok - 1) / kTok;
    q.groups = q.r.q0 < 0 ? 0 : (int)((q.r.C * G + unit - 1) / unit);
    q.units = q.groups * p.num_kv_heads;
    return q;
}

// Tiles of stream t: all, or (`alt`) every second.
__device__ __forceinline__ bool alternate(const Part &s) { return s.rows <= kRows; }
__device__ __forceinline__ int stream_tiles(const Part &s, int t) { return alternate(s) ? (s.n + 1 - t) / 2 : s.n; }

// Instruction descriptor of kind::f8f6f4 with both inputs E4M3 (format 0), fp32 result.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Shared-memory descriptor of K-major rows of D one-byte elements, 8-row atoms one after
// the other: 128-byte swizzle for rows of 128 bytes, 64-byte swizzle (mode 4) for 64.
template <int D>
__device__ __forceinline__ uint64_t sdesc_codes(uint32_t addr) {
    const uint64_t d = tc05::sdesc_sw128(addr, 16, 8 * D);
    return D == 128 ? d : (d & ~(7ull << 61)) | (4ull << 61);
}

// D[tmem] (+)= A[smem] * B[smem]^T, E4M3 inputs, K = 32.
__device__ __forceinline__ void mma_ss_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// What other threads of the CTA have left in the workspace, past the first-level cache.
__device__ __forceinline__ float4 load_l2(const float4 *p) {
    float4 v;
    asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}
__device__ __forceinline__ float load_l2(const float *p) {
    float v;
    asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
    return v;
}

// Four E4M3 codes (lowest byte first) to two fp16 pairs, exactly.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t x, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
}

template <int D, bool F32, bool KV8>
__global__ void __launch_bounds__(kThreads, 1)
tree_kernel(const TreeParams p, const Partials part, const __grid_constant__ CUtensorMap tmap_q,
            const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v) {
    using Sh = TShape<D, KV8>;
    constexpr int NK = Sh::kNK, NV = Sh::kNV, NC = KV8 ? Sh::kNC : 1;
    constexpr int NP = !F32 ? 1 : KV8 ? 2 : 3;  // pieces of a weight
    // (all shared memory is this array: the tiles come first, on the 1024-byte border that
    // their swizzle needs)
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = smem_u32(smem_raw);
    const uint32_t sQ = base, sK = base + Sh::kKAt, sV = base + Sh::kVAt, sC = base + Sh::kCAt;
    float2 *const sm_ml = reinterpret_cast<float2 *>(smem_raw + Sh::kMlAt);  // [2][kRows]
    Part *const sm_part = reinterpret_cast<Part *>(smem_raw + Sh::kPartsAt);
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + Sh::kEndAt);
    volatile int &abort_flag = *reinterpret_cast<volatile int *>(smem_raw + Sh::kEndAt + 4);
    const uint32_t bars = base + Sh::kBarsAt;
    auto kfull = [&](uint32_t i) { return bars + 8u * i; };
    auto kempty = [&](uint32_t i) { return bars + 8u * (NK + i); };
    auto vfull = [&](uint32_t i) { return bars + 8u * (2 * NK + i); };
    auto vempty = [&](uint32_t i) { return bars + 8u * (2 * NK + NV + i); };
    auto cfull = [&](uint32_t i) { return bars + 8u * (2 * (NK + NV) + i); };
    auto cempty = [&](uint32_t i) { return bars + 8u * (2 * (NK + NV) + NC + i); };
    const uint32_t rest = bars + 8u * (2 * (NK + NV + Sh::kNC));
    auto q_full = [&](int t) { return rest + 8u * t; };
    auto q_empty = [&](int t) { return rest + 16u + 8u * t; };
    auto s_full = [&](int t) { return rest + 32u + 8u * t; };
    auto p_half = [&](int t) { return rest + 48u + 8u * t; };
    auto p_full = [&](int t) { return rest + 64u + 8u * t; };
    auto o_full = [&](int t) { return rest + 80u + 8u * t; };
    auto o_empty = [&](int t) { return rest + 96u + 8u * t; };
    auto l_full = [&](int t) { return rest + 112u + 8u * t; };
    auto w_free = [&](int t) { return rest + 128u + 8u * t; };  // three pieces: a half tile's weights have been read
    const uint32_t fin = rest + 144u;
    auto u_full = [&](uint32_t i) { return rest + 152u + 8u * i; };
    auto u_empty = [&](uint32_t i) { return rest + 152u + 8u * (kPlanned + i); };
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (base & 1023u) {  // (never: the array's own alignment)
        if (threadIdx.x == 0) {
            raise_error(p.err, KF_DEVERR_TIMEOUT);
            part.cuts[blockIdx.x] = Cut{};
        }
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < NK; ++i) {
            mbar_init(kfull(i), 1);
            mbar_init(kempty(i), 2);  // (both issuers)
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(vfull(i), KV8 ? 4 : 1);
            mbar_init(vempty(i), 2);
        }
        for (int i = 0; i < Sh::kNC; ++i) {
            mbar_init(cfull(i), 1);
            mbar_init(cempty(i), 4);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(q_full(t), KV8 ? 4 : 1);
            mbar_init(q_empty(t), 2);
            mbar_init(s_full(t), 1);
            mbar_init(p_half(t), 4);  // (a warp arrives once)
            mbar_init(p_full(t), 4);
            mbar_init(o_full(t), 1);
            mbar_init(o_empty(t), 4);
            mbar_init(l_full(t), 4);
            mbar_init(w_free(t), 1);
        }
        mbar_init(fin, 2);
        for (int i = 0; i < kPlanned; ++i) {
            mbar_init(u_full(i), 1);
            mbar_init(u_empty(i), 16);  // eight softmax and four storing warps, the issuers, the producers
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kLoadWarp && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_k)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_v)) : "memory");
        if (!KV8) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_q)) : "memory");
    }
    // what ran before on the stream (an append, say) is complete from here on
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == kIssuerWarp) tc05::tmem_alloc(base + Sh::kEndAt, 512);
    if (threadIdx.x == 0) abort_flag = (*(volatile unsigned int *)p.err & KF_DEVERR_TIMEOUT) ? 1 : 0;
    Place at;
    int64_t slot0;
    const int run = blockIdx.x, runs = gridDim.x;
    const int64_t total = locate(
        p.batch,
        [&](int b) {
            const Request q = request_of(p, b, run == 0);
            return q.n * q.units;
        },
        reinterpret_cast<int64_t *>(sm_ml), [&](int64_t T) { return cut_at(run, runs, T); }, at, slot0);
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    const uint32_t tm = *tmem_slot;
    const int G = p.num_q_heads / p.num_kv_heads, g_shift = 31 - __clz(G);
    const int bs_shift = block_shift(p.block_size);

    auto warp_arrive = [&](uint32_t bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    // A wait that may last as long as a part does; given up early if another role has (kf_wait.cuh).
    auto long_wait = [&](uint32_t bar, uint32_t parity) {
        KF_WAIT_IN_SLICES(__all_sync(0xffffffffu, mbar_wait(bar, parity, kPollsASlice)),
                          __any_sync(0xffffffffu, abort_flag != 0));
    };
    // The k-th part of this run; false behind the last one, or where a wait gave up (`ok`).
    auto next_part = [&](int k, Part &s, bool &ok) {
        const uint32_t e = k % kPlanned;
        ok = ok && long_wait(u_full(e), (k / kPlanned) & 1);
        if (!ok) return false;
        s = sm_part[e];
        warp_arrive(u_empty(e));
        return s.n >= 0;
    };
    // F32: stream t's sum set aside for row r
    auto sums_of = [&](int t, int r) { return part.sums + (int64_t)(2 * run + t) * (D / 4) * kRows + r; };
    auto give_up = [&] {
        if (lane == 0) raise_error(p.err, KF_DEVERR_TIMEOUT);
        abort_flag = 1;
    };

    if (warp >= kLoadWarp && warp < kStoreWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        // ------------------------------- planner --------------------------------
        int64_t pos = slot0, left = cut_at(run + 1, runs, total) - slot0, off = at.off;
        int b = at.b, planned = 0;
        bool loaded = false, first = true, last = false;
        Request q;
        Cut cut{};
        // Finds and publishes the run's next part; false where a wait gave up.
        auto plan_next = [&]() {
            if (last) return true;
            Part s;
            s.n = -1;
            while (left > 0 && b < p.batch) {
                if (!loaded) {
                    q = request_of(p, b, false);
                    loaded = true;
                }
                if (off >= q.n * q.units) {  // on to the next request (some have no units)
                    ++b;
                    off = 0;
                    loaded = false;
                    continue;
                }
                const int64_t unit = off / q.n, tile = off - unit * q.n;
                const int64_t len = left < q.n - tile ? left : q.n - tile;
                const int group = (int)(unit % q.groups);
                const int row0 = group * unit_rows(KV8), all = (int)q.r.C * G;
                s.n = (int)len;
                s.tile0 = (int)tile;
                s.b = b;
                s.head = (int)(unit / q.groups);
                s.q0 = (int)q.r.q0;
                s.node0 = row0 >> g_shift;
                s.rows = min(all - row0, unit_rows(KV8));
                s.C = (int)q.r.C;
                s.L = (int)q.r.L;
                s.slot = len == q.n ? -1 : 2 * run + (first ? 0 : 1);
                if (tile == 0 && len < q.n) {
                    const int64_t P = runs < total ? runs : total, end = pos + q.n;
                    const int64_t last_run = (end * P - 1) / total;  // of the unit's last tile
                    cut = Cut{s.q0 + s.node0, s.head, s.rows, (int)(last_run - run) + 1, s.slot};
                }
                off += len;
                pos += len;
                left -= len;
                first = false;
                break;
            }
            const uint32_t e = planned % kPlanned;
            if (!long_wait(u_empty(e), ((planned / kPlanned) & 1) ^ 1)) return false;
            if (lane == 0) {
                sm_part[e] = s;
                mbar_arrive(u_full(e));
            }
            __syncwarp();
            ++planned;
            last = s.n < 0;
            return true;
        };
        if (warp == kLoadWarp || warp == kPlanWarp) {
            // ---------------------------- producers -----------------------------
            const uint32_t box_bytes = (uint32_t)p.block_size * D * (KV8 ? 1 : 2);
            const int per = kTok >> bs_shift;  // blocks a tile
            uint32_t count = 0, q_loads[2] = {0, 0};
            bool ok = true;
            Part s;
            // (the value loads' warp plans as well, a part ahead)
            const bool plans = warp == kPlanWarp;
            if (plans) ok = plan_next();
            for (int k = 0; next_part(k, s, ok); ++k) {
                if (plans && !plan_next()) {
                    ok = false;
                    break;
                }
                const int32_t *const table = p.block_tables + (int64_t)s.b * p.bt_stride;
                const int lb0 = s.tile0 * per;
                auto entries = [&](int chunk) {  // 32 blocks of the part, one a lane
                    const int e = lb0 + 32 * chunk + lane;
                    return e < p.bt_stride ? __ldg(table + e) : -1;
                };
                // (32 entries at a time, the next ones asked for before they are needed)
                int chunk = 0, cur = entries(0), nxt = entries(1);
                const bool keys = warp == kLoadWarp;
                const CUtensorMap *const map = keys ? &tmap_k : &tmap_v;
                for (int j = 0; j < s.n && ok; ++j) {
                    const bool codes = KV8 && !keys;  // values of E4M3 caches; their keys are used as they are
                    const uint32_t ring = keys ? NK : codes ? NC : NV, st = count % ring;
                    const uint32_t dst = keys ? sK + st * Sh::kKBytes
                                              : codes ? sC + st * Sh::kCodeBytes : sV + st * Sh::kTileBytes;
                    const uint32_t bar = keys ? kfull(st) : codes ? cfull(st) : vfull(st);
                    ok = long_wait(keys ? kempty(st) : codes ? cempty(st) : vempty(st), ((count / ring) & 1) ^ 1);
                    if (!ok) break;
                    ++count;
                    const int t0 = (s.tile0 + j) * kTok;
                    const int nblk = (min(s.L - t0, kTok) + p.block_size - 1) >> bs_shift;
                    if (j * per >> 5 != chunk) {
                        ++chunk;
                        cur = nxt;
                        nxt = entries(chunk + 1);
                    }
                    int phys = __shfl_sync(0xffffffffu, cur, (j * per & 31) + (lane < nblk ? lane : 0));
                    if (lane == 0) mbar_arrive_expect_tx(bar, nblk * box_bytes);
                    __syncwarp();
                    if (lane < nblk) {
                        if (phys < 0 || phys >= p.num_blocks) {
                            raise_error(p.err, KF_DEVERR_BLOCK_ID);
                            phys = 0;
                        }
                        if (KV8) tma_load_4d(dst + lane * box_bytes, map, 0, s.head, 0, phys, bar);
                        else
                            tma_load_4d(dst + lane * box_bytes, map, 0, 0, s.head * Sh::kHalves,
                                        phys * (p.block_size / 8), bar);
                    }
                    __syncwarp();
                    if (KV8 || !keys || j > 0) continue;
                    for (int t = 0; t < (alternate(s) ? 1 : 2) && ok; ++t) {
                        ok = long_wait(q_empty(t), (q_loads[t] & 1) ^ 1);
                        if (!ok) break;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(q_full(t), Sh::kTileBytes);
                            tma_load_4d(sQ + t * Sh::kTileBytes, &tmap_q, 0, s.head * G,
                                        s.q0 + s.node0 + t * (kRows >> g_shift), 0, q_full(t));
                        }
                        __syncwarp();
                        ++q_loads[t];
                    }
                }
            }
            if (!ok) {
                give_up();
                cut.parts = 0;
            }
            if (plans && lane == 0) part.cuts[run] = cut;
            if (lane == 0) {
                // drain: the last use of every slot has landed before the CTA can exit
                const uint32_t ring = warp == kLoadWarp ? NK : KV8 ? NC : NV;
                bool done = true;
                for (uint32_t i = count > ring ? count - ring : 0; i < count; ++i) {
                    const uint32_t st = i % ring;
                    const uint32_t bar = warp == kLoadWarp ? kfull(st) : KV8 ? cfull(st) : vfull(st);
                    done = mbar_wait(bar, (i / ring) & 1) && done;
                }
                for (int t = 0; t < 2; ++t)
                    if (q_loads[t] > 0) done = mbar_wait(q_full(t), (q_loads[t] - 1) & 1) && done;
                if (!done) raise_error(p.err, KF_DEVERR_TIMEOUT);
            }
            __syncwarp();
        } else if (warp == kIssuerWarp || warp == kIssuerWarp2) {
            // --------------------- MMA issuers, one a stream ---------------------
            // (A wait behind issued MMAs is served once the tensor pipe has taken them: one
            // warp for both streams spent 2500 cycles a tile on 1024 cycles of MMAs.)
            const int t = warp == kIssuerWarp ? 0 : 1;
            {
                const uint32_t id_s = KV8 ? idesc_e4m3(kRows, kTok) : tc05::idesc_bf16(kRows, kTok, false, false);
                const uint32_t id_o = KV8 ? tc05::idesc_f16(kRows, D, false, true) : tc05::idesc_bf16(kRows, D, false, true);
                const uint64_t qd0 = KV8 ? sdesc_codes<D>(sQ) : tc05::sdesc_sw128(sQ, 16, 1024);
                const uint64_t kd0 = KV8 ? sdesc_codes<D>(sK) : tc05::sdesc_sw128(sK, 16, Sh::kAtomBytes);
                const uint64_t vd0 = tc05::sdesc_sw128(sV, 1024, Sh::kAtomBytes);
                constexpr uint64_t kStep = Sh::kTileBytes / 16;
                const uint32_t ts = tm + Sh::col_s(t), to = tm + Sh::col_o(t);
                uint32_t tile_base = 0;               // the ring's tiles before this part
                uint32_t qc[2] = {0, 0}, pc = 0, oc = 0;  // query tiles, weights and parts so far
                bool ok = true;
                Part s;
                for (int k = 0; next_part(k, s, ok); ++k) {
                    const int n = s.n;
                    const bool alt = alternate(s);
                    const int tiles = alt ? (n + 1 - t) / 2 : n, qt = alt ? 0 : t;
                    const uint64_t qd = qd0 + qt * kStep;
                    // Both issuers wait for every tile of the rings, in order (a parity wait that
                    // skipped a phase could take the one before for it), and release it: the one
                    // whose stream has no use for it by a plain arrival.
                    auto pass_k = [&](int j) {
                        const uint32_t st = (tile_base + j) % NK;
                        if (!long_wait(kfull(st), ((tile_base + j) / NK) & 1)) return false;
                        if (lane == 0) mbar_arrive(kempty(st));
                        return true;
                    };
                    auto pass_v = [&](int j) {
                        const uint32_t st = (tile_base + j) % NV;
                        if (!long_wait(vfull(st), ((tile_base + j) / NV) & 1)) return false;
                        if (lane == 0) mbar_arrive(vempty(st));
                        return true;
                    };
                    ok = long_wait(q_full(0), qc[0] & 1);
                    if (!ok) break;
                    if (t == 1 && (!alt || tiles == 0) && lane == 0) mbar_arrive(q_empty(0));
                    if (alt && t == 1) ok = pass_k(0) && (tiles > 0 || pass_v(0));
                    for (int i = 0; ok && i <= tiles && tiles > 0; ++i) {
                        if (i > 0) {
                            // O += P V of the tile before
                            const int j = alt ? 2 * (i - 1) + t : i - 1;
                            if (alt && j == 1) ok = pass_v(0);
                            const uint32_t st = (tile_base + j) % NV;
                            const uint64_t vd = vd0 + st * kStep;
                            ok = ok && long_wait(vfull(st), ((tile_base + j) / NV) & 1);
                            // the last part's rows have been read out of O
                            if (i == 1) ok = ok && long_wait(o_empty(t), (oc & 1) ^ 1);
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                ok = ok && long_wait(half ? p_full(t) : p_half(t), pc & 1);
                                if (!ok) break;
                                tc05::fence_after_sync();
                                if (tc05::elect_one()) {
#pragma unroll
                                    for (int kk = 4 * half; kk < 4 * half + 4; ++kk) {
                                        const uint32_t w = ts + (NP == 3 ? 0 : 64 * half) + 8 * (kk & 3);
                                        const uint64_t v = vd + (uint64_t)(kk * 2 * Sh::kAtomBytes / 16);
#pragma unroll
                                        for (int n = 0; n < NP; ++n)
                                            tc05::mma_ts(to, w + 32 * n, v, id_o, i == 1 && kk == 0 && n == 0 ? 0u : 1u);
                                    }
                                    if (NP == 3 && !half) tc05::commit(w_free(t));
                                    if (half && i == tiles) tc05::commit(o_full(t));
                                    if (half) tc05::commit(vempty(st));
                                }
                                __syncwarp();
                            }
                            if (!ok) break;
                            ++pc;
                            oc += i == tiles;
                            if (i == tiles && alt && j + 1 < n) ok = pass_v(j + 1);
                        }
                        if (i < tiles) {
                            // S = Q K^T
                            const int j = alt ? 2 * i + t : i;
                            const uint32_t st = (tile_base + j) % NK;
                            const uint64_t kd = kd0 + st * (uint64_t)(Sh::kKBytes / 16);
                            if (i == 0 && qt == 1) ok = ok && long_wait(q_full(1), qc[1] & 1);
                            ok = ok && long_wait(kfull(st), ((tile_base + j) / NK) & 1);
                            if (!ok) break;
                            tc05::fence_after_sync();
                            if (tc05::elect_one()) {
#pragma unroll
                                for (int kk = 0; KV8 && kk < 2 * (D / 32); ++kk)  // q's high parts, then its low parts
                                    mma_ss_e4m3(ts, qd + (uint64_t)((kk / (D / 32) * kRows * D + 32 * (kk % (D / 32))) / 16),
                                                kd + (uint64_t)(32 * (kk % (D / 32)) / 16), id_s, kk > 0 ? 1u : 0u);
#pragma unroll
                                for (int kk = 0; !KV8 && kk < D / 16; ++kk)
                                    tc05::mma_ss(ts, qd + (uint64_t)(((kk >> 2) * 16384 + 32 * (kk & 3)) / 16),
                                                 kd + (uint64_t)(((kk >> 2) * 1024 + 32 * (kk & 3)) / 16), id_s,
                                                 kk > 0 ? 1u : 0u);
                                tc05::commit(s_full(t));
                                tc05::commit(kempty(st));
                                if (i == tiles - 1) {
                                    tc05::commit(q_empty(qt));
                                    if (qt == 1) tc05::commit(q_empty(1));  // (its only reader)
                                }
                            }
                            __syncwarp();
                            if (alt && j > 1) ok = pass_v(j - 1);
                            if (alt && j + 1 < n) ok = ok && pass_k(j + 1);
                        }
                    }
                    if (!ok) break;
                    ++qc[0];  // (a part uses query tile 0, and tile 1 where it has one)
                    if (!alt) ++qc[1];
                    tile_base += n;
                }
                if (!ok) give_up();
                if (tc05::elect_one()) {
                    tc05::commit(fin);  // every MMA has completed before TMEM is freed
                    if (!mbar_wait(fin, 0)) raise_error(p.err, KF_DEVERR_TIMEOUT);
                }
                __syncwarp();
            }
        }
    } else if (warp < 8) {
        // ------------------------------- softmax --------------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        const int t = warp >> 2, r = threadIdx.x & (kRows - 1);
        const uint32_t tw = tm + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t ts = tw + Sh::col_s(t), to = tw + Sh::col_o(t);
        uint32_t sc = 0, oc = 0, qc = 0;  // score tiles, parts, query tiles so far
        uint32_t vbase = 0;               // value tiles before this part
        bool ok = true;
        Part s;
        for (int k = 0; next_part(k, s, ok); ++k) {
            const bool alt = alternate(s);
            const int tiles = stream_tiles(s, t), row = r + (alt ? 0 : kRows * t);
            const bool row_ok = row < s.rows;
            const int node = s.node0 + (row >> g_shift);
            const int first = s.L - s.C;  // the context's tokens
            float c = p.scale_log2;
            bool bad_row = false;
            if (KV8) {
                // The row of q as two E4M3 numbers each, high part and rest, so that the scores
                // come from the cache's codes as they are: times the power of two that brings the
                // row's largest number below 2^8, a bf16 number (8 bits) is the sum of the two (4
                // bits each) exactly from 2^-2 on; below that it is off by at most 2^-10, which is
                // 2^-17 of the row's largest.
                const uint16_t *q = p.q + ((int64_t)(s.q0 + (row_ok ? node : 0)) * p.num_q_heads + s.head * G +
                                           (r & (G - 1))) * D;
                uint32_t x[D / 2];
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const uint4 v = row_ok ? __ldg(reinterpret_cast<const uint4 *>(q) + i) : make_uint4(0, 0, 0, 0);
                    x[4 * i] = v.x;
                    x[4 * i + 1] = v.y;
                    x[4 * i + 2] = v.z;
                    x[4 * i + 3] = v.w;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t w = x[4 * i + e];
                        top = max(top, max(w & 0x7fff, (w >> 16) & 0x7fff));
                    }
                }
                // |q| < 2^(e - 126), e the largest exponent field (subnormal rows: 1). A row with an
                // infinity or a NaN: its scores are made NaN below
                const int e = max((int)(top >> 7), 1);
                bad_row = e == 255;
                const int up = bad_row ? 0 : 8 - (e - 126);  // q * 2^up < 2^8
                c *= p.k_scale[s.head];
                // (2^up and 2^-up each as two factors: one alone can leave fp32's exponents)
                const float f1 = __uint_as_float((uint32_t)(127 + up / 2) << 23);
                const float f2 = __uint_as_float((uint32_t)(127 + up - up / 2) << 23);
                c = c * __uint_as_float((uint32_t)(127 - up / 2) << 23) * __uint_as_float((uint32_t)(127 - (up - up / 2)) << 23);
                if (t == 0) {
                    if (!long_wait(q_empty(0), (qc & 1) ^ 1)) {
                        ok = false;
                        break;
                    }
                    ++qc;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            hi[h] = lo[h] = 0;
#pragma unroll
                            for (int g = 0; g < 2; ++g) {
                                const uint32_t w = x[8 * i + 2 * h + g];
                                const float a = bf16_lo(w) * f1 * f2, b = bf16_hi(w) * f1 * f2;
                                const uint32_t two = f32x2_to_e4m3x2(a, b), back = e4m3x2_to_f16x2(two);
                                hi[h] |= two << (16 * g);
                                lo[h] |= f32x2_to_e4m3x2(a - f16_lo(back), b - f16_hi(back)) << (16 * g);
                            }
                        }
                        const uint32_t at_q = sQ + swz<D>(r, i);
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at_q), "r"(hi[0]), "r"(hi[1]),
                                     "r"(hi[2]), "r"(hi[3])
                                     : "memory");
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at_q + kRows * D), "r"(lo[0]),
                                     "r"(lo[1]), "r"(lo[2]), "r"(lo[3])
                                     : "memory");
                    }
                    fence_proxy_async_smem();
                    warp_arrive(q_full(0));
                }
            }
            if (bad_row) c = NAN;
            const float cs = c > 0.f ? c : 1.f;  // (a scale of zero or less is applied first)
            float m = -INFINITY, l = 0.f;
            float aside = -INFINITY;  // F32: the maximum that the sums set aside are relative to
            for (int i = 0; i < tiles; ++i, ++sc) {
                const int j = alt ? 2 * i + t : i, t0 = (s.tile0 + j) * kTok;
                if (!long_wait(s_full(t), sc & 1)) {
                    ok = false;
                    break;
                }
                tc05::fence_after_sync();
                if (!KV8 && s.L - t0 < kTok) {  // zero the value rows past the context (every stream that reads them)
                    const uint32_t vi = vbase + j, vst = vi % NV;
                    if (!warp_wait(vfull(vst), (vi / NV) & 1)) {
                        ok = false;
                        break;
                    }
                    const int ntok = s.L - t0, chunks = (kTok - ntok) * 8;  // 16-byte chunks a half
                    for (int z = r; z < chunks * Sh::kHalves; z += kRows) {
                        const int hf = z / chunks, q = z % chunks, tok = ntok + (q >> 3);
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                         sV + vst * Sh::kTileBytes + (tok >> 3) * Sh::kAtomBytes + hf * 1024 +
                                         (tok & 7) * 128 + (q & 7) * 16),
                                     "r"(0u)
                                     : "memory");
                    }
                    fence_proxy_async_smem();
                }
                // (constexpr: a plain condition costs the other forms; E4M3, 64 columns 218 -> 222 us)
                if constexpr (F32) if (i > 0 && i % kFlush == 0) {  // O, complete up to the tile before, is set aside
                    float4 *const sums = sums_of(t, r);
                    auto quad = [&](int at) {
                        return i > kFlush ? load_l2(sums + at * kRows) : make_float4(0.f, 0.f, 0.f, 0.f);
                    };
                    float4 set[16];  // (64 columns on their way at a time)
#pragma unroll
                    for (int e = 0; e < 16; ++e) set[e] = quad(e);
                    const float keep = aside == m ? 1.f : exp2f(aside - m);
                    aside = m;
                    const uint32_t zero[16] = {};
#pragma unroll
                    for (int cc = 0; cc < D; cc += 16) {
                        uint32_t o[16];
                        tmem_ld16(to + cc, o);
                        tmem_st16_async(to + cc, zero);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float4 &v = set[(cc / 4 + e) % 16];
                            v.x = fmaf(v.x, keep, __uint_as_float(o[4 * e]));
                            v.y = fmaf(v.y, keep, __uint_as_float(o[4 * e + 1]));
                            v.z = fmaf(v.z, keep, __uint_as_float(o[4 * e + 2]));
                            v.w = fmaf(v.w, keep, __uint_as_float(o[4 * e + 3]));
                            __stcg(sums + (cc / 4 + e) * kRows, v);
                            if (cc + 64 < D) v = quad(cc / 4 + e + 16);
                        }
                    }
                    __stcg(part.sums_m + (2 * run + t) * kRows + r, m);
                    tmem_wait_st();
                }
                uint32_t x[2][64];
                tmem_ld64_async(ts, x[0]);
                tmem_ld64_async(ts + 64, x[1]);
                tmem_landed(x[0]);
                tmem_landed(x[1]);
                if (!(c > 0.f)) {  // (the maximum is one of unscaled scores)
#pragma unroll
                    for (int e = 0; e < 128; ++e)
                        x[e >> 6][e & 63] = __float_as_uint(__uint_as_float(x[e >> 6][e & 63]) * c);
                }
                int most = kTok;
                if (t0 + kTok > first) {  // nodes in the tile: the context before them, and the row's ancestors
                    uint32_t w[4];
                    const int ctx = first - t0;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        w[q] = ctx >= 32 * q + 32 ? 0xffffffffu : ctx <= 32 * q ? 0u : (1u << (ctx - 32 * q)) - 1;
                    for (int a = row_ok ? node : -1; a >= 0;) {
                        const int at_tok = ctx + a;
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (at_tok >> 5 == q) w[q] |= 1u << (at_tok & 31);
                        const int up = __ldg(p.parents + s.q0 + a);
                        if (up < -1 || up >= a) {  // no earlier node: taken as none
                            raise_error(p.err, KF_DEVERR_TREE);
                            break;
                        }
                        a = up;
                    }
                    most = 0;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (__any_sync(0xffffffffu, w[q] != 0)) most = 32 * q + 32;
                        if (__all_sync(0xffffffffu, w[q] == 0xffffffffu)) continue;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(w[q] >> e & 1)) x[q >> 1][32 * (q & 1) + e] = 0xff800000u;  // -inf
                    }
                }
                ok = row_tile<D, NP, KV8>(
                    ts, to, 0, x, most, cs, i > 0, m, l, [&](int half) { warp_arrive(half ? p_full(t) : p_half(t)); },
                    [&] { return long_wait(w_free(t), sc & 1); });
                if (!ok) break;
            }
            vbase += s.n;
            if (!ok) break;
            if (tiles == 0) continue;
            // (the last part's have been read)
            if (!long_wait(o_empty(t), (oc & 1) ^ 1)) {
                ok = false;
                break;
            }
            sm_ml[t * kRows + r] = make_float2(m, l);
            warp_arrive(l_full(t));
            ++oc;
        }
        if (!ok) give_up();
    } else {
        // ------------------- rows out; E4M3 codes to fp16 -----------------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        const int r = threadIdx.x & (kRows - 1);
        const uint32_t tw = tm + ((uint32_t)(32 * (warp & 3)) << 16);
        const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
        const bool part_wide = (reinterpret_cast<uintptr_t>(part.o) & 31) == 0;
        uint32_t oc[2] = {0, 0};
        bool ok = true;

        auto store_rows = [&](const Part &s) {
            const bool alt = alternate(s);
            // stream 1's rows are tile 1's, or (alt) the same rows over the odd tiles
            const int count = alt ? 1 : 2;
            float f[2], lse = -INFINITY;  // factors of O_0 and O_1
            auto wait_for = [&](int t) {
                ok = ok && long_wait(l_full(t), oc[t] & 1) && long_wait(o_full(t), oc[t] & 1);
                ++oc[t];
                return ok;
            };
            const float vs = KV8 ? p.v_scale[s.head] : 1.f;
            auto finish = [&](float m, float l) { return l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY; };
            for (int t = 0; t < count && ok; ++t) {
                const int row = r + kRows * t;
                const bool row_ok = row < s.rows;
                bool both = false;
                if (!wait_for(t)) return;
                if (alt && s.n > 1) {
                    if (!wait_for(1)) return;
                    both = true;
                }
                tc05::fence_after_sync();
                const float2 a = sm_ml[t * kRows + r];
                if (both) {
                    const float2 b = sm_ml[kRows + r];
                    // (a maximum of -inf: nothing seen, weight 0; a NaN stays one)
                    const float M = a.x > b.x ? a.x : b.x;
                    const float wa = a.x == -INFINITY && a.y == 0.f ? 0.f : exp2f(a.x - M);
                    const float wb = b.x == -INFINITY && b.y == 0.f ? 0.f : exp2f(b.x - M);
                    const float l = a.y * wa + b.y * wb, inv = l != 0.f ? vs / l : 0.f;
                    f[0] = wa * inv;
                    f[1] = wb * inv;
                    lse = finish(M, l);
                } else {
                    f[0] = a.y != 0.f ? vs / a.y : 0.f;
                    f[1] = 0.f;
                    lse = finish(a.x, a.y);
                }
                // F32: what to multiply the sums set aside by (those of the other row tile's rows
                // lie with stream 1; 0: none)
                float keep[2] = {0.f, 0.f};
                if constexpr (F32) {
                    if (stream_tiles(s, t) > kFlush) {
                        const float from = load_l2(part.sums_m + (2 * run + t) * kRows + r);
                        keep[0] = from == a.x ? 1.f : exp2f(from - a.x);
                    }
                    if (both && stream_tiles(s, 1) > kFlush) {
                        const float m = sm_ml[kRows + r].x, from = load_l2(part.sums_m + (2 * run + 1) * kRows + r);
                        keep[1] = from == m ? 1.f : exp2f(from - m);
                    }
                }
                const int64_t at_row = (int64_t)(s.q0 + s.node0 + (row >> g_shift)) * p.num_q_heads + s.head * G + (r & (G - 1));
                const int64_t at_part = (int64_t)s.slot * part.pitch + row;
                if (row_ok) {
                    if (s.slot >= 0) part.lse[at_part] = lse;
                    else if (p.lse_out) p.lse_out[at_row] = lse;
                }
#pragma unroll 1
                for (int cc = 0; cc < D; cc += 16) {
                    uint32_t o[16], o2[16];
                    tmem_ld16(tw + Sh::col_o(t) + cc, o);
                    if (both) tmem_ld16(tw + Sh::col_o(1) + cc, o2);
                    auto add_sums = [&](int u, float k, uint32_t (&to)[16]) {
                        const float4 *const sums = sums_of(u, r) + cc / 4 * kRows;
                        float4 v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = load_l2(sums + e * kRows);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            to[e] = __float_as_uint(
                                fmaf(reinterpret_cast<const float *>(v)[e], k, __uint_as_float(to[e])));
                    };
                    if constexpr (F32) if (keep[0] != 0.f) add_sums(t, keep[0], o);
                    if constexpr (F32) if (keep[1] != 0.f) add_sums(1, keep[1], o2);
                    if (cc == D - 16) {
                        tc05::fence_before_sync();
                        warp_arrive(o_empty(t));
                        if (both) warp_arrive(o_empty(1));
                    }
                    if (!row_ok) continue;
                    float v[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        // (a stream whose weights are all zero says nothing, whatever its values)
                        v[e] = f[0] != 0.f ? __uint_as_float(o[e]) * f[0] : 0.f;
                        if (both && f[1] != 0.f) v[e] = fmaf(__uint_as_float(o2[e]), f[1], v[e]);
                    }
                    if (s.slot >= 0 || F32) {
                        float *dst = s.slot >= 0 ? part.o + at_part * D + cc : static_cast<float *>(p.out) + at_row * D + cc;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t w[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(v[8 * i + e]);
                            store32(dst + 8 * i, w, s.slot >= 0 ? part_wide : wide);
                        }
                    } else {
                        uint32_t w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) w[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
                        store32(static_cast<uint16_t *>(p.out) + at_row * D + cc, w, wide);
                    }
                }
            }
        };

        Part s, prev;
        prev.n = -1;
        // E4M3: these warps widen the values' codes. A thread takes 16 codes a step, always the
        // same columns of the same token of 16 (D = 128) or 32 (64), so that source and
        // destination step by constants. Of the 8 lanes that store together half are at an even
        // token and half at the odd one behind it, whose swizzle differs by one, in opposite
        // column halves, whose codes lie in different banks.
        const int tok0 = D == 128 ? r / 16 * 2 + (r >> 2 & 1) : r >> 2;
        const int ch = D == 128 ? (r & 3) + 4 * ((r >> 2 & 1) ^ (r >> 3 & 1)) : r & 3;
        const uint32_t code_at = tok0 * D + ch * 16;
        const uint32_t wide_at = (tok0 >> 3) * Sh::kAtomBytes + (ch >> 2) * 1024 + (tok0 & 7) * 128 +
                                 ((2 * (ch & 3) ^ (tok0 & 7)) << 4);
        uint32_t vc = 0;  // tiles so far
        auto widen = [&](const Part &s, int j) {
            constexpr int kTokStep = D == 128 ? 16 : 32, kPer = kTok / kTokStep;
            const uint32_t cst = vc % NC, st = vc % NV;
            if (!long_wait(cfull(cst), (vc / NC) & 1) || !long_wait(vempty(st), ((vc / NV) & 1) ^ 1)) return false;
            const uint32_t src = sC + cst * Sh::kCodeBytes + code_at, dst = sV + st * Sh::kTileBytes + wide_at;
            const int live = s.L - (s.tile0 + j) * kTok - tok0;  // steps of the context, times kTokStep
            uint4 x[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(x[i].x), "=r"(x[i].y), "=r"(x[i].z), "=r"(x[i].w)
                             : "r"(src + i * 2048));
            if (live < kTok) {
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (i * kTokStep >= live) x[i] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                uint32_t y[8];
                e4m3x4_to_f16x4(x[i].x, y[0], y[1]);
                e4m3x4_to_f16x4(x[i].y, y[2], y[3]);
                e4m3x4_to_f16x4(x[i].z, y[4], y[5]);
                e4m3x4_to_f16x4(x[i].w, y[6], y[7]);
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst + i * 4096), "r"(y[0]), "r"(y[1]),
                             "r"(y[2]), "r"(y[3]));
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"((dst ^ 16) + i * 4096), "r"(y[4]),
                             "r"(y[5]), "r"(y[6]), "r"(y[7]));
            }
            fence_proxy_async_smem();
            warp_arrive(vfull(st));
            if (lane == 0) mbar_arrive(cempty(cst));
            ++vc;
            return true;
        };
        for (int k = 0; next_part(k, s, ok); ++k) {
            if (KV8) {
                for (int j = 0; j < s.n && ok; ++j) {
                    ok = widen(s, j);
                    // the part before is written out once this one's first tiles are under way
                    if (ok && j == 0 && prev.n >= 0) store_rows(prev);
                }
                prev = s;
            } else {
                store_rows(s);
            }
            if (!ok) break;
        }
        if (KV8 && ok && prev.n >= 0) store_rows(prev);
        if (!ok) give_up();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge may be set up
    tc05::fence_before_sync();
    __syncthreads();
    if (warp == kIssuerWarp) {
        tc05::fence_after_sync();
        tc05::tmem_dealloc(tm, 512);
    }
}

// ---------------------------------------------------------------------------
// Merge of the units that more than one CTA worked on: block x takes the one that CTA x
// began, RPB rows a block, 8 / RPB warps a row, each over every (8 / RPB)-th part:
//   M = max lse_i, w_i = e^{lse_i - M}, out = sum w_i o_i / sum w_i.
// With a warp a row and at most FEW parts all loads go out at once and every lane computes
// the same weights. Instruction issue bounds it (59 % of its slots over 32 MB, 12.7 us, cold).
// ---------------------------------------------------------------------------
template <int D, int RPB, int FEW>
__global__ void __launch_bounds__(256)
tree_merge_kernel(const TreeParams p, const Partials part) {
    constexpr int WPR = 8 / RPB, V = D / 32;  // warps a row; a lane's columns, side by side
    using Vec = typename std::conditional<V == 4, float4, float2>::type;
    __shared__ float sm_o[WPR > 1 ? 8 : 1][D];
    __shared__ float sm_w[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the attention kernel's writes are there
    const Cut cut = part.cuts[blockIdx.x];
    const int n = cut.parts, rows = cut.rows;
    if (n == 0 || blockIdx.y * RPB >= rows) return;
    auto slot_at = [&](int i) { return i == 0 ? (int64_t)cut.slot0 : 2 * ((int64_t)blockIdx.x + i); };
    const int sub = warp % WPR;
    const int row = blockIdx.y * RPB + warp / WPR;
    const bool live = row < rows;
    float M = -INFINITY, W = 0.f, acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
    if (live && WPR == 1 && n <= FEW) {
        // the usual case: all loads at once, every lane the same weights, no exchange
        float x[FEW];
        Vec o[FEW];
#pragma unroll
        for (int i = 0; i < FEW; ++i) {
            if (i >= n) {
                x[i] = -INFINITY;
                continue;
            }
            const int64_t at_row = slot_at(i) * part.pitch + row;
            x[i] = part.lse[at_row];
            o[i] = reinterpret_cast<const Vec *>(part.o + at_row * D)[lane];
        }
        bool nan = false;
#pragma unroll
        for (int i = 0; i < FEW; ++i) {
            nan = nan || x[i] != x[i];
            M = fmaxf(M, x[i]);
        }
        if (nan) M = NAN;  // a NaN row's weights, and so the row, are NaN
        if (M != -INFINITY) {
#pragma unroll
            for (int i = 0; i < FEW; ++i) {
                if (i >= n) continue;
                const float w = exp2f((x[i] - M) * 1.4426950408889634f);
                const float *const e = reinterpret_cast<const float *>(&o[i]);
                W += w;
#pragma unroll
                for (int v = 0; v < V; ++v) acc[v] = fmaf(w, e[v], acc[v]);
            }
        }
    } else if (live) {
        bool nan = false;
        for (int i = lane; i < n; i += 32) {
            const float x = part.lse[slot_at(i) * part.pitch + row];
            nan = nan || x != x;
            M = fmaxf(M, x);
        }
        for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        if (__any_sync(0xffffffffu, nan)) M = NAN;  // a NaN row's weights, and so the row, are NaN
        if (M != -INFINITY) {
#pragma unroll 4
            for (int i = sub; i < n; i += WPR) {
                const int64_t at_row = slot_at(i) * part.pitch + row;
                const float w = exp2f((part.lse[at_row] - M) * 1.4426950408889634f);
                W += w;
                const Vec o = reinterpret_cast<const Vec *>(part.o + at_row * D)[lane];
                const float *const e = reinterpret_cast<const float *>(&o);
#pragma unroll
                for (int v = 0; v < V; ++v) acc[v] = fmaf(w, e[v], acc[v]);  // (an empty part holds zeros)
            }
        }
    }
    if (WPR > 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) sm_o[WPR > 1 ? warp : 0][V * lane + v] = acc[v];
        if (lane == 0) sm_w[warp] = W;
        __syncthreads();
        if (sub != 0 || !live) return;
        for (int k = 1; k < WPR; ++k) {
            W += sm_w[warp + k];
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] += sm_o[WPR > 1 ? warp + k : 0][V * lane + v];
        }
    }
    if (!live) return;
    const int G = p.num_q_heads / p.num_kv_heads, g_shift = 31 - __clz(G);
    const int64_t at = (int64_t)(cut.token + (row >> g_shift)) * p.num_q_heads + cut.head * G + (row & (G - 1));
    const float inv = W != 0.f ? 1.f / W : 0.f;
    Vec x;
    float *const e = reinterpret_cast<float *>(&x);
#pragma unroll
    for (int v = 0; v < V; ++v) e[v] = acc[v] * inv;
    if (p.out_dtype == KF_F32) {
        reinterpret_cast<Vec *>(static_cast<float *>(p.out) + at * D)[lane] = x;
    } else {
        uint32_t w[V / 2];
#pragma unroll
        for (int v = 0; v < V / 2; ++v) w[v] = pack_bf16(e[2 * v], e[2 * v + 1]);
        uint32_t *const dst = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.out) + at * D) + V / 2 * lane;
        if (V == 4) *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[V / 2 - 1]);
        else dst[0] = w[0];
    }
    if (lane == 0 && p.lse_out) p.lse_out[at] = W != 0.f ? M + logf(W) : -INFINITY;
}

// q [num_q_tokens, Hq, D] as (64 columns, head, token, column half): 128 rows of (token,
// head of the group) pairs land as halves of 128 swizzled 128-byte rows.
bool encode_q(tc::EncodeFn fn, CUtensorMap *map, const TreeParams &p) {
    const int G = p.num_q_heads / p.num_kv_heads;
    const cuuint64_t head = (cuuint64_t)p.head_dim * 2;
    const cuuint64_t dims[4] = {64, (cuuint64_t)p.num_q_heads, (cuuint64_t)p.num_q_tokens, (cuuint64_t)p.head_dim / 64};
    const cuuint64_t strides[3] = {head, head * p.num_q_heads, 128};
    const cuuint32_t box[4] = {64, (cuuint32_t)G, (cuuint32_t)(kRows / G), (cuuint32_t)p.head_dim / 64};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t *>(p.q), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16 cache as (64 columns, 8 slots, (head, half), 8-slot groups): a box of one block of one
// head lands as 8-token atoms, each half by half, of swizzled 128-byte rows. E4M3 cache as (D
// columns, head, slot, block): a box lands as rows of D codes, swizzled where products read
// them (keys).
bool encode_cache(tc::EncodeFn fn, CUtensorMap *map, const void *cache, const TreeParams &p, bool kv8, bool keys) {
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    // L2 fetches no more around a token than this head's row of it: with 256 bytes for rows of
    // 128 the neighbouring head came along, whose turn is long after (E4M3, 64 requests of
    // 1K-64K tokens: 555 us, the DRAM busy with twice the bytes; 522 now).
    const int bytes = p.head_dim * (kv8 ? 1 : 2);
    const CUtensorMapL2promotion promote = bytes >= 256   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                           : bytes == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                          : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
    const int bs = p.block_size, D = p.head_dim;
    const cuuint64_t row = (cuuint64_t)p.num_kv_heads * D * (kv8 ? 1 : 2);  // bytes between slots
    if (kv8) {
        const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)p.num_kv_heads, (cuuint64_t)bs, (cuuint64_t)p.num_blocks};
        const cuuint64_t strides[3] = {(cuuint64_t)D, row, row * bs};
        const cuuint32_t box[4] = {(cuuint32_t)D, 1, (cuuint32_t)bs, 1};
        return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(cache), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE,
                  !keys ? CU_TENSOR_MAP_SWIZZLE_NONE : D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  promote,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    }
    const int halves = D / 64;
    const cuuint64_t dims[4] = {64, 8, (cuuint64_t)p.num_kv_heads * halves, (cuuint64_t)p.num_blocks * (bs / 8)};
    const cuuint64_t strides[3] = {row, 128, 8 * row};
    const cuuint32_t box[4] = {64, 8, (cuuint32_t)halves, (cuuint32_t)bs / 8};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(cache), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, promote,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool F32, bool KV8>
cudaError_t launch(const TreeParams &p, const Partials &part, int ctas, int64_t units, cudaStream_t stream,
                   tc::EncodeFn fn) {
    using Sh = TShape<D, KV8>;
    CUtensorMap mq, mk, mv;
    if (!encode_q(fn, &mq, p) || !encode_cache(fn, &mk, p.k_cache, p, KV8, true) ||
        !encode_cache(fn, &mv, p.v_cache, p, KV8, false))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done.load() & bit)) {
        e = cudaFuncSetAttribute(tree_kernel<D, F32, KV8>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmemBytes);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Sh::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    // both kernels are set up while their predecessor ends, and wait for it themselves
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, tree_kernel<D, F32, KV8>, p, part, mq, mk, mv);
    if (e != cudaSuccess || ctas == 1) return e;  // (one run: nothing is cut)
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    // Few units are cut over many CTAs each: one row a merge block, its warps share the parts.
    // Else a warp a row, all parts' loads at once where there are no more than 4 or 8: 8 where
    // units have as many (one request of 777 tokens 15.7 -> 14.5 us); their registers cost
    // occupancy where rows are many (8 requests, 4000 rows: 128 us with 4, 132 with 8).
    if (units * 8 < ctas) {
        cfg.gridDim = dim3(ctas - 1, part.pitch);
        return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, 1, 4>, p, part);
    }
    cfg.gridDim = dim3(ctas - 1, (part.pitch + 7) / 8);
    if (units * 3 < ctas) return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, 8, 8>, p, part);
    return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, 8, 4>, p, part);
}

size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

// Tiles of n tokens, at least one.
int64_t tiles_of(int64_t n) { return std::max<int64_t>(1, (n + kTok - 1) / kTok); }

int row_pitch(int max_query_len, int num_q_heads, int num_kv_heads) {
    return std::min(max_query_len * (num_q_heads / num_kv_heads), unit_rows(false));
}

}  // namespace

size_t tree_workspace_bytes(int max_query_len, int num_q_heads, int num_kv_heads, int head_dim, bool f32,
                            int sm_count) {
    const int pitch = row_pitch(max_query_len, num_q_heads, num_kv_heads);
    const size_t rows = 2 * (size_t)sm_count * pitch;
    const size_t parts = al256(rows * head_dim * 4) + al256(rows * 4) + sm_count * sizeof(Cut);
    return f32 ? al256(parts) + 2 * (size_t)sm_count * (head_dim + 1) * kRows * sizeof(float) : parts;
}

cudaError_t launch_tree(const TreeParams &p, void *workspace, int sm_count, cudaStream_t stream, void *encode_fn) {
    tc::EncodeFn fn = reinterpret_cast<tc::EncodeFn>(encode_fn);
    const int G = p.num_q_heads / p.num_kv_heads;
    // no more units than the bound, and than all rows, allow; no more runs than these have tiles
    const int64_t rows_max = (int64_t)p.max_query_len * G;
    const int unit = unit_rows(p.k_scale != nullptr);
    const int64_t units = p.num_kv_heads * std::min<int64_t>((int64_t)p.batch * ((rows_max + unit - 1) / unit),
                                                             p.batch + (int64_t)p.num_q_tokens * G / unit);
    const int64_t tokens = std::min<int64_t>(p.max_context_len, (int64_t)p.bt_stride * p.block_size);
    const int64_t tiles = units * tiles_of(tokens);
    const int ctas = (int)std::min<int64_t>(sm_count, tiles);
    Partials part;
    part.pitch = row_pitch(p.max_query_len, p.num_q_heads, p.num_kv_heads);
    part.o = static_cast<float *>(workspace);
    const size_t rows = 2 * (size_t)sm_count * part.pitch;
    uint8_t *ws = static_cast<uint8_t *>(workspace) + al256(rows * p.head_dim * 4);
    part.lse = reinterpret_cast<float *>(ws);
    ws += al256(rows * 4);
    part.cuts = reinterpret_cast<Cut *>(ws);
    part.sums = reinterpret_cast<float4 *>(ws + al256(sm_count * sizeof(Cut)));  // (fp32 outputs only)
    part.sums_m = reinterpret_cast<float *>(part.sums + 2 * (size_t)sm_count * (p.head_dim / 4) * kRows);
    const bool f32 = p.out_dtype == KF_F32;
    if (p.k_scale) {
        if (p.head_dim == 128)
            return f32 ? launch<128, true, true>(p, part, ctas, units, stream, fn)
                       : launch<128, false, true>(p, part, ctas, units, stream, fn);
        return f32 ? launch<64, true, true>(p, part, ctas, units, stream, fn)
                   : launch<64, false, true>(p, part, ctas, units, stream, fn);
    }
    if (p.head_dim == 128)
        return f32 ? launch<128, true, false>(p, part, ctas, units, stream, fn)
                   : launch<128, false, false>(p, part, ctas, units, stream, fn);
    return f32 ? launch<64, true, false>(p, part, ctas, units, stream, fn)
               : launch<64, false, false>(p, part, ctas, units, stream, fn);
}

}  // namespace kf
