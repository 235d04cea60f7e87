// kf_latent_tc05.cu -- latent attention, absorbed form, on tcgen05.
//
// Query rows (query token j, head h) of a request share every key: row r of the
// request is q[q_start + r / H, r % H], contiguous in memory. With the latent
// row x_t = [c_t ; r_t] of R + 64 numbers,
//   S = Q X^T  (K = R + 64),   P = softmax rows,   O = P C  (C = the first R columns of X),
// so one tile of X in shared memory serves both products: keys as they are, values
// as the same bytes read along the other axis.
//
// Work. Rows come in tiles of 64 (R = 512) or 128 (R = 256), tokens in tiles of 32 or
// 64. A unit is one row tile of one request over all its token tiles; the units of the
// batch, laid end to end, are cut into equal runs, one a CTA (one CTA an SM: the
// tile ring fills its shared memory); where nearly all units have a partner in their
// request, one a pair of CTAs, which walk it side by side. A run may start and end
// inside a unit; the parts of such a unit go to the workspace as normalised (o, lse)
// partials and latent_merge joins them. So a batch of any length mix keeps every SM
// busy to the end, at the price of at most two partials a CTA.
//
// One tile: 32 or 64 rows of R + 64 bf16 arrive as TMA boxes of 16 tokens, landing as
// 8-token groups of 128-byte-swizzled atoms (group, 64-column atom, token, column).
//   S[rows x tokens]           = Q X^T          A = Q, B = X, both K-major, M = the row tile
//   O^T[128 columns x rows]   += C^T P^T        A = C^T (M-major: the same tile), B = P
// The value product is taken transposed, R / 128 instructions of M = 128 and N = the
// rows in use (rounded up to 16): its accumulator then takes 256 TMEM columns instead
// of R in every row's lane, which leaves room for two score tiles, and its work
// shrinks with the rows. P goes through shared memory as that product's B.
//   warps 0-3  softmax; 64-row tiles: rows 16 w .. 16 w + 15, four lanes a row (16x256b
//              TMEM loads: lane l holds columns 8 i + 2 (l % 4), + 1 of rows l / 4 and
//              l / 4 + 8); 128-row tiles: a thread a row. Base-2 online softmax with a
//              lazy maximum (it moves only by more than 8, and then O^T's columns are
//              rescaled in TMEM); the epilogue.
//   warp 4     TMA producer;  warp 5  issues S and owns TMEM;  warp 6  issues O^T.
// Score tiles alternate between two TMEM buffers, and the two products have an issuing
// warp each: S of tile g + 1 goes out as soon as its tile has landed, the value
// product of tile g as soon as its weights are there, whichever comes first.
//
// What bounds it: 2 (R + 64) bytes of cache a token. At R = 512 an SM's share of HBM
// brings 64 tokens in 3400 cycles (73.7 KB at 44.6 B/ns). The instructions' operands
// come from shared memory at 128 bytes a cycle: per 32 tokens 36 S instructions of 24
// cycles (3 KB) and 8 O^T ones of 48 (6 KB), 2500 cycles for 64 tokens. So the cache is
// the bound up to 64 rows: 16 requests of 8K-256K tokens and 32 heads take 185 us, 0.88
// of the copy bandwidth with start, epilogues and merge. With more rows what bounds is
// the chain load (1650 cycles for 64 tokens) - S - softmax - O^T over a ring that Q
// (72 KB) leaves 144 KB for: 64 requests of 4K tokens, 128 heads: 110 us. Four slots of
// 32 tokens cost a fifth more operand reads than two of 64 and shorten the chain: 201
// and 116 us with two. The weights of 32 tokens are half of a swizzled 128-byte row,
// so that two tiles' weights fit where 64 tokens' lay, and the softmax of one tile
// writes while the value product of the last reads. More than two score tiles in TMEM
// gain nothing.
//
// P is rounded to bf16, the type of C in the same instruction (l sums the weights before
// that); a lower half beside it would read all of C again, at the bound above. Against 64
// bits the bf16 output is 1.8e-3 to 2.4e-3 off, its own rounding 1.7e-3.
//
// Tokens past a unit's last visible one are masked by selection (never multiplied)
// and their rows zeroed in shared memory (0 * NaN would poison the product).
// Every wait is bounded; one that gives up sets KF_DEVERR_TIMEOUT and the CTA
// drains its copies and MMAs, frees its TMEM and returns.
#include "kf_latent.cuh"
#include "kf_runs.cuh"
#include "kf_tc05_ops.cuh"

#include <algorithm>

namespace kf {
namespace {

using namespace tc;
using namespace mq5;

// Rows a unit: O^T takes R / 128 * (rows a unit) of TMEM's columns, 256 either way.
__host__ __device__ constexpr int unit_rows(int latent_dim) { return latent_dim == 512 ? 64 : 128; }
// Tokens a tile: half as many where a token's row is twice as long.
__host__ __device__ constexpr int tile_tokens(int latent_dim) { return latent_dim == 512 ? 32 : 64; }
// Tiles fetched into L2 ahead of the ring's loads (16 requests of 8K-256K tokens, 32 heads: 185 us
// with one, 186 with two, 189 with three; 48 of 4K, R = 256: 49 / 50 / 51).
constexpr int kAhead = 1;
constexpr int kSoftThreads = 128, kProducerWarp = 4, kScoreWarp = 5, kValueWarp = 6, kThreads = 224;

template <int R>
struct LShape {
    static constexpr int kM = unit_rows(R), kN = tile_tokens(R);
    static constexpr int kAtoms = (R + kRopeDim) / 64;
    static constexpr int kGroupBytes = kAtoms * 1024;         // 8 tokens
    static constexpr int kTileBytes = kN / 8 * kGroupBytes;
    static constexpr int kQAtomBytes = kM * 128;              // the rows x 64 columns
    static constexpr int kQBytes = kAtoms * kQAtomBytes;
    static constexpr int kPBytes = kM * 128;
    static constexpr int kPBuffers = 64 / kN;  // weights of a tile: a row's 128 bytes hold 64 tokens
    static constexpr int kStages = R == 512 ? 4 : 3;
    static constexpr int kSmemBytes = kQBytes + kStages * kTileBytes + kPBytes + 1024;
    static constexpr int kDimTiles = R / 128;
    static constexpr uint32_t kColS = 256;                    // two score tiles; O^T below
    static_assert(kSmemBytes > 116 * 1024 && kSmemBytes <= 225 * 1024, "one CTA an SM");
    static_assert(kDimTiles * kM <= 256, "O^T columns");
};

// ---------------------------------------------------------------------------
// The schedule: units of a request and the run of each CTA.
// ---------------------------------------------------------------------------
struct Request {
    int64_t q0, rows, L, shift;  // query j sees tokens [0, min(shift + j + 1, L))
    int64_t n;                   // token tiles charged to each unit (at least one)
    int units;
};

__device__ __forceinline__ Request request_of(const LatentParams &p, int b, bool report) {
    const LatentRequest r = latent_request(p, b, report);
    if (r.q0 < 0) return {0, 0, 0, 0, 1, 0};
    const int64_t C = r.C < p.max_query_len ? r.C : p.max_query_len;
    Request q;
    q.q0 = r.q0;
    q.rows = C * p.num_heads;
    q.L = r.L < p.max_context_len ? r.L : p.max_context_len;
    q.shift = r.L - r.C;
    const int kN = tile_tokens(p.latent_dim);
    q.n = q.L > 0 ? (q.L + kN - 1) / kN : 1;
    const int M = unit_rows(p.latent_dim);
    q.units = (int)((q.rows + M - 1) / M);
    return q;
}

// Tiles of a request in the list that the runs are cut from: with `twins` = 2, two CTAs
// share a run, one the even, one the odd units, tile by tile at the same time.
__device__ __forceinline__ int64_t cost_of(const LatentParams &p, int b, int twins, bool report) {
    const Request r = request_of(p, b, report);
    return r.n * ((r.units + twins - 1) / twins);
}

// Whether pairs of CTAs pay: of `all` tiles of all units, `lone` are of requests' last, odd
// units, where the second twin has nothing to do. 64 requests of 4K tokens, R = 512, pairs /
// single CTAs: no lone tile, 102 / 111 us (128 rows) and 181 / 200 (256); one in 15, 102 /
// 109; one in 9, 410 / 385; one in 5, 258 / 221; one in 3, 172 / 155; all, 90 / 64.
__host__ __device__ constexpr bool pairs_pay(int64_t all, int64_t lone) { return lone * 12 <= all; }

// CTAs that share a run, from the batch's real query counts.
__device__ __forceinline__ int twins_of(const LatentParams &p, int64_t *sm) {
    int64_t all = 0, lone = 0;
    for (int b = threadIdx.x; b < p.batch; b += blockDim.x) {
        const Request r = request_of(p, b, false);
        all += r.n * r.units;
        lone += r.n * (r.units & 1);
    }
    for (int o = 16; o; o >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, o);
        lone += __shfl_xor_sync(0xffffffffu, lone, o);
    }
    const int warp = threadIdx.x >> 5, warps = blockDim.x / 32;
    if ((threadIdx.x & 31) == 0) {
        sm[2 * warp] = all;
        sm[2 * warp + 1] = lone;
    }
    __syncthreads();
    all = lone = 0;
    for (int w = 0; w < warps; ++w) {
        all += sm[2 * w];
        lone += sm[2 * w + 1];
    }
    __syncthreads();  // `sm` is free again
    return pairs_pay(all, lone) ? 2 : 1;
}

// One unit's part in a CTA's run: token tiles [tile0, tile0 + tiles).
struct Segment {
    int64_t q0, row0, L, shift;
    int rows, tile0, tiles;
    int t_end;          // the last token any row of the unit sees, plus one
    int b;
    bool whole, first;  // the unit lies in this run alone; it is the run's first segment
    bool cut;           // the unit starts here and goes on in the next run
    int64_t unit_end;   // the tile after the unit's last, in the batch's list
};

struct Walker {
    Place at;
    int64_t pos, left;  // the next tile in the batch's list; tiles left of the run
    int twins, twin;  // CTAs that share the run; which of them this is
    bool first = true;
    Request r;
    bool loaded = false;

    __device__ __forceinline__ bool next(const LatentParams &p, Segment &s) {
        while (left > 0) {
            if (!loaded) {
                r = request_of(p, at.b, false);
                loaded = true;
            }
            const int64_t groups = (r.units + twins - 1) / twins;
            if (at.off >= r.n * groups) {  // on to the next request (some have no units)
                ++at.b;
                at.off = 0;
                loaded = false;
                if (at.b >= p.batch) return false;
                continue;
            }
            const int64_t group = at.off / r.n, tile = at.off - group * r.n;
            const int64_t len = left < r.n - tile ? left : r.n - tile;
            const int64_t unit = group * twins + twin;
            if (unit >= r.units) {  // the other twin's unit is the request's last
                at.off += len;
                pos += len;
                left -= len;
                continue;
            }
            s.q0 = r.q0;
            const int M = unit_rows(p.latent_dim);
            s.row0 = unit * M;
            s.rows = (int)(r.rows - s.row0 < M ? r.rows - s.row0 : M);
            s.L = r.L;
            s.shift = r.shift;
            s.b = at.b;
            s.whole = len == r.n;
            s.first = first;
            s.cut = tile == 0 && !s.whole;
            s.unit_end = pos - tile + r.n;
            int64_t end = r.L;
            if (p.causal) {
                const int64_t lim = r.shift + (s.row0 + s.rows - 1) / p.num_heads + 1;
                if (lim < end) end = lim < 0 ? 0 : lim;
            }
            s.t_end = (int)end;
            const int kN = tile_tokens(p.latent_dim);
            const int64_t valid = (end + kN - 1) / kN;  // tiles any row sees
            const int64_t hi = tile + len < valid ? tile + len : valid;
            s.tile0 = (int)tile;
            s.tiles = hi > tile ? (int)(hi - tile) : 0;
            at.off += len;
            pos += len;
            left -= len;
            first = false;
            return true;
        }
        return false;
    }
};

// A unit cut over the CTAs i, i + twins, i + 2 twins, ...: where its partials lie. The
// first CTA's slot is `slot0`; the others' is the first of their two (2 i).
struct Cut {
    int64_t row_out;  // its first row in out and lse_out
    int rows, parts, slot0, twins;
};

struct Partials {
    float *o;    // [2 * CTAs][row pitch][R]
    float *lse;  // [2 * CTAs][row pitch]
    Cut *cuts;   // [CTAs]: the unit that starts in CTA i's run and goes on (parts = 0: none)
    int pitch;   // rows a slot holds
};

// ---------------------------------------------------------------------------
// PTX
// ---------------------------------------------------------------------------
// 16 lanes x 32 columns: lane l gets columns 8 i + 2 (l % 4) + {0, 1} of TMEM lanes
// l / 4 (r[4 i], r[4 i + 1]) and l / 4 + 8 (r[4 i + 2], r[4 i + 3]), waited for.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15"
        "}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// Columns [col, col + 16) of this thread's TMEM lane, waited for.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15"
        "}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// A 4-D box into L2.
__device__ __forceinline__ void prefetch_4d(const CUtensorMap *map, int x, int y, int z, int w) {
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}

// The softmax warps' barrier, and the same with an OR of one predicate.
__device__ __forceinline__ void soft_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ bool soft_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

// put(row, column offset, value) for this thread's column of every 128-column tile
// and the first `rows` rows: O^T times the row's 1 / sum (in `inv`), or zeros.
template <int R, typename F>
__device__ __forceinline__ void store_rows(uint32_t tm, bool any, int rows, const float *inv, F put) {
#pragma unroll 1
    for (int d = 0; d < R / 128; ++d) {
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += 16) {
            uint32_t o[16];
            if (any) tmem_ld16(tm + unit_rows(R) * d + r0, o);
            float v[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float w = inv[r0 + e];
                v[e] = any && w != 0.f ? __uint_as_float(o[e]) * w : 0.f;
            }
            // (a branch a store costs three times the stores: only the last chunk pays it)
            if (r0 + 16 <= rows) {
#pragma unroll
                for (int e = 0; e < 16; ++e) put(r0 + e, 128 * d, v[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (r0 + e < rows) put(r0 + e, 128 * d, v[e]);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Attention
// ---------------------------------------------------------------------------
template <int R>
__global__ void __launch_bounds__(kThreads, 1)
latent_kernel(const LatentParams p, const Partials part, int max_twins, bool decide,
              const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_q) {
    using Sh = LShape<R>;
    constexpr int NS = Sh::kStages, NP = Sh::kPBuffers, KS = (R + kRopeDim) / 16, kN = Sh::kN, KP = kN / 16, kM = Sh::kM;
    // full[NS], empty[NS], q_full, q_empty, s_full[2], s_empty[2], p_full[2], pv_done[2], o_empty, fin[2]
    __shared__ __align__(8) uint64_t bar_mem[2 * NS + 13];
    __shared__ int64_t sm_loc[36];
    // (1 / sum has an array of its own: a warp that still rescales O^T after the unit's last
    // tile reads every row's alpha, and no barrier lies between that and the epilogue's sums)
    __shared__ float sm_alpha[kM], sm_inv[kM], sm_lse[kM];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t sQ = base, sX = base + Sh::kQBytes, sP = sX + NS * Sh::kTileBytes;
    const uint32_t bars = smem_u32(bar_mem);
    auto full = [&](uint32_t i) { return bars + 8u * i; };
    auto empty = [&](uint32_t i) { return bars + 8u * (NS + i); };
    const uint32_t q_full = bars + 8u * (2 * NS), q_empty = q_full + 8;
    auto s_full = [&](uint32_t i) { return q_full + 16 + 8 * i; };
    auto s_empty = [&](uint32_t i) { return q_full + 32 + 8 * i; };
    auto p_full = [&](uint32_t i) { return q_full + 48 + 8 * (i % NP); };   // of tile i
    auto pv_done = [&](uint32_t i) { return q_full + 64 + 8 * (i % NP); };
    const uint32_t o_empty = q_full + 80, fin = q_full + 88;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * NS; ++i) mbar_init(bars + 8 * i, 1);
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full(i), 1);
            mbar_init(s_empty(i), kSoftThreads);
        }
        for (int i = 0; i < NP; ++i) {
            mbar_init(p_full(i), kSoftThreads);
            mbar_init(pv_done(i), 1);
        }
        mbar_init(o_empty, kSoftThreads);
        mbar_init(fin, 1);
        mbar_init(fin + 8, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kProducerWarp && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_x)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_q)) : "memory");
    }
    // what ran before on the stream (an append, say) is complete from here on
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // (TMEM is taken after the wait: a predecessor that still has to allocate its own would
    // wait for this kernel, and this one for it)
    if (warp == kScoreWarp) tc05::tmem_alloc(smem_u32(&tmem_slot), 512);
    if (threadIdx.x == 0) abort_flag = (*(volatile unsigned int *)p.err & KF_DEVERR_TIMEOUT) ? 1 : 0;
    const int twins = decide ? twins_of(p, sm_loc) : max_twins;
    const int run = blockIdx.x / twins, runs = gridDim.x / twins;
    Walker walk;
    walk.twins = twins;
    walk.twin = blockIdx.x - run * twins;
    int64_t slot0;
    const int64_t total = locate(
        p.batch, [&](int b) { return cost_of(p, b, twins, blockIdx.x == 0); }, sm_loc,
        [&](int64_t T) { return cut_at(run, runs, T); }, walk.at, slot0);
    walk.pos = slot0;
    walk.left = cut_at(run + 1, runs, total) - slot0;
    if (abort_flag) walk.left = 0;  // an earlier kernel's wait gave up (no role has started yet)
    tc05::fence_before_sync();
    __syncthreads();
    tc05::fence_after_sync();
    const uint32_t tm = tmem_slot;
    const int bs_shift = block_shift(p.block_size);
    // an issuing warp's end: report a wait that gave up, and see every MMA issued done
    // before TMEM is freed
    auto finish = [&](bool ok, uint32_t bar) {
        if (tc05::elect_one()) {
            if (!ok) {
                raise_error(p.err, KF_DEVERR_TIMEOUT);
                abort_flag = 1;
            }
            tc05::commit(bar);
            if (!mbar_wait(bar, 0)) raise_error(p.err, KF_DEVERR_TIMEOUT);
        }
        __syncwarp();
    };

    if (warp == kProducerWarp) {
        // ------------------------------ producer ------------------------------
        uint32_t g = 0, nseg = 0, q_loads = 0;
        bool ok = true;
        Segment s{};
        // lane e: the cache row group of the tile's e-th 16 tokens, asked for long
        // before the tile's turn; past the last token any valid one
        auto group_of = [&](int tile) -> int {
            const int t = tile * kN + 16 * lane;
            if (lane >= kN / 16 || t >= s.t_end) return -1;
            const int64_t e = t >> bs_shift;
            int64_t phys = e < p.bt_stride ? p.block_tables[(int64_t)s.b * p.bt_stride + e] : -1;
            if (phys < 0 || phys >= p.num_blocks) {
                raise_error(p.err, KF_DEVERR_BLOCK_ID);
                phys = 0;
            }
            return (int)(phys * (p.block_size / 8)) + ((t & (p.block_size - 1)) >> 3);
        };
        while (ok && walk.next(p, s)) {
            if (s.tiles == 0) continue;
            // kAhead tiles beyond the ring are fetched into L2: HBM's latency then passes
            // under their predecessors' turns, and the ring's own loads come from L2
            // (and a tile's table entry is read one turn before that)
            int grp[kAhead + 2];
#pragma unroll
            for (int k = 0; k <= kAhead; ++k) grp[k] = k < s.tiles ? group_of(s.tile0 + k) : -1;
            for (int i = 0; i < s.tiles; ++i, ++g) {
                if (grp[kAhead] >= 0) prefetch_4d(&tmap_x, 0, 0, 0, grp[kAhead]);
                grp[kAhead + 1] = i + kAhead + 1 < s.tiles ? group_of(s.tile0 + i + kAhead + 1) : -1;
                const int t0 = (s.tile0 + i) * kN;
                const int ntok = s.t_end - t0 < kN ? s.t_end - t0 : kN;
                const int nbox = (ntok + 15) / 16;
                const uint32_t st = g % NS;
                int go = 1;
                if (lane == 0) {
                    go = !abort_flag && mbar_wait(empty(st), ((g / NS) & 1) ^ 1);
                    if (go && i == 0) {
                        go = mbar_wait(q_empty, (nseg & 1) ^ 1);
                        if (go) {
                            ++q_loads;
                            mbar_arrive_expect_tx(q_full, Sh::kQBytes);
                            tc05::tma_load_3d(sQ, &tmap_q, 0, (int)(s.q0 * p.num_heads + s.row0), 0, q_full);
                        }
                    }
                    if (go) mbar_arrive_expect_tx(full(st), nbox * 2 * Sh::kGroupBytes);
                    else {
                        raise_error(p.err, KF_DEVERR_TIMEOUT);
                        abort_flag = 1;
                    }
                }
                ok = __shfl_sync(0xffffffffu, go, 0);
                if (!ok) break;
                if (lane < nbox)
                    tma_load_4d(sX + st * Sh::kTileBytes + lane * 2 * Sh::kGroupBytes, &tmap_x, 0, 0, 0, grp[0],
                                full(st));
                __syncwarp();
#pragma unroll
                for (int k = 0; k <= kAhead; ++k) grp[k] = grp[k + 1];
            }
            ++nseg;
        }
        if (lane == 0) {
            // drain: the last use of every slot has landed before the CTA can exit
            for (uint32_t j = g > NS ? g - NS : 0; j < g; ++j)
                if (!mbar_wait(full(j % NS), (j / NS) & 1)) raise_error(p.err, KF_DEVERR_TIMEOUT);
            if (q_loads > 0 && !mbar_wait(q_full, (q_loads - 1) & 1)) raise_error(p.err, KF_DEVERR_TIMEOUT);
        }
    } else if (warp == kScoreWarp) {
        // ----------------------------- score issuer -----------------------------
        // (whole warps walk and wait, one elected lane issues: the descriptors then
        // stay in uniform registers, 36 cycles an instruction instead of 58)
        const uint32_t id_s = tc05::idesc_bf16(kM, kN, false, false);
        const uint64_t qd = tc05::sdesc_sw128(sQ, 16, 1024);
        uint32_t g = 0, nseg = 0;
        bool ok = true;
        Segment s{};
        while (ok && walk.next(p, s)) {
            const int tiles = __shfl_sync(0xffffffffu, s.tiles, 0);
            if (tiles == 0) continue;
            ok = warp_wait(q_full, nseg & 1);
            for (int i = 0; i < tiles && ok; ++i, ++g) {
                const uint32_t st = g % NS, sb = g & 1;
                ok = !__any_sync(0xffffffffu, abort_flag) && warp_wait(s_empty(sb), ((g >> 1) & 1) ^ 1) &&
                     warp_wait(full(st), (g / NS) & 1);
                if (!ok) break;
                tc05::fence_after_sync();
                const uint64_t xd = tc05::sdesc_sw128(sX + st * Sh::kTileBytes, 16, Sh::kGroupBytes);
                if (tc05::elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < KS; ++kk)
                        tc05::mma_ss(tm + Sh::kColS + 64 * sb,
                                     qd + (uint64_t)(((kk >> 2) * Sh::kQAtomBytes + 32 * (kk & 3)) / 16),
                                     xd + (uint64_t)(((kk >> 2) * 1024 + 32 * (kk & 3)) / 16), id_s, kk > 0 ? 1u : 0u);
                    tc05::commit(s_full(sb));
                    if (i == tiles - 1) tc05::commit(q_empty);
                }
                __syncwarp();
            }
            ++nseg;
        }
        finish(ok, fin);
    } else if (warp == kValueWarp) {
        // ----------------------------- value issuer -----------------------------
        const uint64_t pd = tc05::sdesc_sw128(sP, 16, 1024);
        uint32_t g = 0, nseg = 0;
        bool ok = true;
        Segment s{};
        while (ok && walk.next(p, s)) {
            const int tiles = __shfl_sync(0xffffffffu, s.tiles, 0);
            if (tiles == 0) continue;
            const uint32_t id_o =
                tc05::idesc_bf16(128, __shfl_sync(0xffffffffu, (s.rows + 15) / 16 * 16, 0), true, false);
            // the previous segment's O^T has been read out
            ok = warp_wait(o_empty, (nseg & 1) ^ 1);
            for (int i = 0; i < tiles && ok; ++i, ++g) {
                const uint32_t st = g % NS;
                ok = !__any_sync(0xffffffffu, abort_flag) && warp_wait(p_full(g), (g / NP) & 1);
                if (!ok) break;
                tc05::fence_after_sync();
                const uint64_t cd = tc05::sdesc_sw128(sX + st * Sh::kTileBytes, 1024, Sh::kGroupBytes);
                if (tc05::elect_one()) {
                    // (one accumulator after the other: alternating between them costs a fifth)
#pragma unroll
                    for (int d = 0; d < Sh::kDimTiles; ++d)
#pragma unroll
                        for (int kk = 0; kk < KP; ++kk)
                            tc05::mma_ss(tm + kM * d, cd + (uint64_t)((d * 2048 + kk * 2 * Sh::kGroupBytes) / 16),
                                         pd + (uint64_t)(((g % NP) * kN * 2 + 32 * kk) / 16), id_o, (i > 0 || kk > 0) ? 1u : 0u);
                    tc05::commit(empty(st));
                    tc05::commit(pv_done(g));
                }
                __syncwarp();
            }
            ++nseg;
        }
        finish(ok, fin + 8);
    } else {
        // ------------------------------- softmax --------------------------------
        const uint32_t lane_base = (uint32_t)(32 * warp) << 16;
        const float c = p.scale_log2;
        // This lane's rows and how their scores lie: 64 rows a unit, two rows, a quarter of
        // each; 128 rows, one whole row.
        constexpr int NR = kM == 64 ? 2 : 1, NX = kN / (kM == 64 ? 4 : 1);
        const int rr[2] = {kM == 64 ? 16 * warp + (lane >> 2) : (int)threadIdx.x, 16 * warp + (lane >> 2) + 8};
        auto token_of = [&](int e) { return kM == 64 ? 8 * (e >> 1) + 2 * (lane & 3) + (e & 1) : e; };
        uint32_t g = 0;
        bool fail = false, stop = false;  // fail: this warp's wait gave up; stop: all four warps leave
        Cut cut{};
        Segment s{};
        while (!stop && walk.next(p, s)) {
            float m[NR], l[NR];
            int lim[NR];  // tokens these rows see (none: rows past the unit's last)
#pragma unroll
            for (int k = 0; k < NR; ++k) {
                m[k] = -INFINITY;
                l[k] = 0.f;
                int64_t x = s.t_end;
                if (p.causal && s.shift + (s.row0 + rr[k]) / p.num_heads + 1 < x)
                    x = s.shift + (s.row0 + rr[k]) / p.num_heads + 1;
                lim[k] = rr[k] < s.rows && x > 0 ? (int)x : 0;
            }
            for (int i = 0; i < s.tiles; ++i, ++g) {
                const int t0 = (s.tile0 + i) * kN;
                const uint32_t sb = g & 1;
                if (!warp_wait(s_full(sb), (g >> 1) & 1)) fail = true;
                tc05::fence_after_sync();
                float x[NR][NX];  // element e of row k: token token_of(e) of the tile
                if (kM == 64) {
                    uint32_t u[16];
                    tmem_ld_16x256b_x4(tm + lane_base + Sh::kColS + 64 * sb, u);
#pragma unroll
                    for (int e = 0; e < 16; ++e)  // (NR - 1 and NX - 1 are 1 and 7 here)
                        x[(e >> 1) & (NR - 1)][(((e >> 2) << 1) | (e & 1)) & (NX - 1)] = __uint_as_float(u[e]);
                } else {
                    uint32_t u[64];
                    tc05::tmem_ld64(tm + lane_base + Sh::kColS + 64 * sb, u);
#pragma unroll
                    for (int e = 0; e < 64; ++e) x[0][e & (NX - 1)] = __uint_as_float(u[e]);
                }
                tc05::fence_before_sync();
                mbar_arrive(s_empty(sb));
                // tokens past the last visible one: their rows become zeros
                const int ntok = s.t_end - t0;
                if (ntok < kN) {
                    const uint32_t xt = sX + (g % NS) * Sh::kTileBytes;
                    constexpr int CH = R / 8;  // 16-byte chunks of a value row
                    for (int k = threadIdx.x; k < (kN - ntok) * CH; k += kSoftThreads) {
                        const int t = ntok + k / CH, ch = k % CH;
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                         xt + (t >> 3) * Sh::kGroupBytes + (ch >> 3) * 1024 + (t & 7) * 128 +
                                         (ch & 7) * 16),
                                     "r"(0u)
                                     : "memory");
                    }
                }
                float mx[NR];
                // fast path: all rows of the warp see the whole tile and the scale is positive;
                // otherwise scores are scaled and masked first
                bool whole_tile = true;
#pragma unroll
                for (int k = 0; k < NR; ++k) {
                    mx[k] = -INFINITY;
                    whole_tile = whole_tile && t0 + kN <= lim[k];
                }
                const bool fast = c > 0.f && __all_sync(0xffffffffu, whole_tile);
                if (fast) {
#pragma unroll
                    for (int k = 0; k < NR; ++k) {
#pragma unroll
                        for (int e = 0; e < NX; e += 2) mx[k] = max3f(mx[k], x[k][e], x[k][e + 1]);
                        mx[k] *= c;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < NR; ++k)
#pragma unroll
                        for (int e = 0; e < NX; ++e) {
                            x[k][e] = t0 + token_of(e) < lim[k] ? x[k][e] * c : -INFINITY;
                            mx[k] = fmaxf(mx[k], x[k][e]);
                        }
                }
                bool need = false;
                float alpha[NR];
#pragma unroll
                for (int k = 0; k < NR; ++k) {
                    if (kM == 64) {
                        mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 1));
                        mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 2));
                    }
                    const bool up = mx[k] > m[k] + kRescaleSlack;
                    alpha[k] = up ? exp2f(m[k] - mx[k]) : 1.f;  // m = -inf: 0
                    if (up) {
                        l[k] *= alpha[k];
                        m[k] = mx[k];
                        need = need || i > 0;
                    }
                }
                // one barrier a tile in the common case; O^T is rescaled (and a wait that
                // gave up acted on) by all four warps together
                const bool any = soft_any(need || fail);
                // O^T is complete once the previous value product is done (the P buffer is free
                // with the last one that read it)
                if (any && g > 0 && !warp_wait(pv_done(g - 1), ((g - 1) / NP) & 1)) fail = true;
                if (g >= NP && !warp_wait(pv_done(g - NP), ((g / NP) - 1) & 1)) fail = true;
                if (any) {
                    stop = soft_any(fail);
                    if (stop) break;
#pragma unroll
                    for (int k = 0; k < NR; ++k)
                        if (kM == 128 || (lane & 3) == 0) sm_alpha[rr[k]] = alpha[k];
                    soft_sync();
                    tc05::fence_after_sync();
                    for (int d = 0; d < Sh::kDimTiles; ++d)
                        for (int q = 0; q < (s.rows + 15) / 16; ++q) {
                            uint32_t o[16];
                            tmem_ld16(tm + lane_base + kM * d + 16 * q, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * sm_alpha[16 * q + e]);
                            tc05::tmem_st16(tm + lane_base + kM * d + 16 * q, o);
                        }
                }
#pragma unroll
                for (int k = 0; k < NR; ++k) {
                    const float mu = m[k] == -INFINITY ? 0.f : m[k];
                    const float cc = fast ? c : 1.f;  // (scores are scaled already on the slow path)
                    const uint32_t row = sP + rr[k] * 128;
                    float2 ls = make_float2(0.f, 0.f);
                    uint32_t w[NX / 2];
#pragma unroll
                    for (int e = 0; e < NX / 2; ++e) {
                        float2 a = fma_f32x2(make_float2(x[k][2 * e], x[k][2 * e + 1]), make_float2(cc, cc),
                                             make_float2(-mu, -mu));
                        a.x = ex2f(a.x);
                        a.y = ex2f(a.y);
                        ls = add_f32x2(ls, a);
                        w[e] = pack_bf16(a.x, a.y);
                    }
                    l[k] += ls.x + ls.y;
                    if (kM == 64) {
#pragma unroll
                        for (int e = 0; e < NX / 2; ++e)
                            asm volatile("st.shared.u32 [%0], %1;" ::"r"(row + (((e + (g % NP) * (kN / 8)) ^ (rr[k] & 7)) << 4) + (lane & 3) * 4),
                                         "r"(w[e])
                                         : "memory");
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(row + ((e ^ (rr[k] & 7)) << 4)),
                                         "r"(w[(4 * e) % (NX / 2)]), "r"(w[(4 * e + 1) % (NX / 2)]),
                                         "r"(w[(4 * e + 2) % (NX / 2)]), "r"(w[(4 * e + 3) % (NX / 2)])
                                         : "memory");
                    }
                }
                fence_proxy_async_smem();
                tc05::fence_before_sync();
                mbar_arrive(p_full(g));
            }
            if (stop) break;
            // epilogue: row sums (over the lanes of a row), then O^T column by column
#pragma unroll
            for (int k = 0; k < NR; ++k) {
                if (kM == 64) {
                    l[k] += __shfl_xor_sync(0xffffffffu, l[k], 1);
                    l[k] += __shfl_xor_sync(0xffffffffu, l[k], 2);
                }
                if (kM == 128 || (lane & 3) == 0) {
                    // (no token seen: 0 and -inf; a NaN stays one)
                    sm_inv[rr[k]] = l[k] != 0.f ? 1.f / l[k] : 0.f;
                    sm_lse[rr[k]] = l[k] != 0.f ? (m[k] + log2f(l[k])) * 0.6931471805599453f : -INFINITY;
                }
            }
            if (s.tiles > 0 && !warp_wait(pv_done(g - 1), ((g - 1) / NP) & 1)) fail = true;
            stop = soft_any(fail);
            if (stop) break;
            const int64_t slot = 2 * (int64_t)blockIdx.x + (s.first ? 0 : 1);
            const int64_t row_out = s.q0 * p.num_heads + s.row0;
            if (s.cut) {
                const int64_t P = runs < total ? runs : total;
                const int64_t last = (s.unit_end * P - 1) / total;  // the run of the unit's last tile
                cut = Cut{row_out, s.rows, (int)(last - run) + 1, (int)slot, twins};
            }
            if (s.tiles > 0) tc05::fence_after_sync();
            // O^T: thread = column, one row a TMEM column; 32 consecutive numbers a warp and store
            if (!s.whole) {
                float *dst = part.o + slot * part.pitch * R + threadIdx.x;
                store_rows<R>(tm + lane_base, s.tiles > 0, s.rows, sm_inv, [=](int r, int d, float v) { dst[r * R + d] = v; });
            } else if (p.out_dtype == KF_F32) {
                float *dst = static_cast<float *>(p.out) + row_out * R + threadIdx.x;
                store_rows<R>(tm + lane_base, s.tiles > 0, s.rows, sm_inv, [=](int r, int d, float v) { dst[r * R + d] = v; });
            } else {
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + row_out * R + threadIdx.x;
                store_rows<R>(tm + lane_base, s.tiles > 0, s.rows, sm_inv,
                              [=](int r, int d, float v) { dst[r * R + d] = __float2bfloat16(v); });
            }
            if (threadIdx.x < s.rows) {
                if (!s.whole) part.lse[slot * part.pitch + threadIdx.x] = sm_lse[threadIdx.x];
                else if (p.lse_out) p.lse_out[row_out + threadIdx.x] = sm_lse[threadIdx.x];
            }
            tc05::fence_before_sync();
            if (s.tiles > 0) mbar_arrive(o_empty);
            soft_sync();  // sm_inv and sm_lse are free again
        }
        if (threadIdx.x == 0) {
            if (stop) cut.parts = 0;
            part.cuts[blockIdx.x] = cut;
        }
        if (stop) {
            if (threadIdx.x == 0) raise_error(p.err, KF_DEVERR_TIMEOUT);
            abort_flag = 1;
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge may be set up
    tc05::fence_before_sync();
    __syncthreads();
    if (warp == kScoreWarp) {
        tc05::fence_after_sync();
        tc05::tmem_dealloc(tm, 512);
    }
}

// ---------------------------------------------------------------------------
// Merge of the units that more than one CTA worked on: block x takes the one that
// CTA x began, RPB rows a block, 8 / RPB warps a row, each over every (8 / RPB)-th
// partial:
//   M = max lse_i, w_i = e^{lse_i - M}, out = sum w_i o_i / sum w_i.
// ---------------------------------------------------------------------------
template <int R, int RPB>
__global__ void __launch_bounds__(256)
latent_merge_kernel(const LatentParams p, const Partials part) {
    constexpr int WPR = 8 / RPB, V = R / 128;  // warps a row; float4 a lane
    __shared__ float4 sm_o[WPR > 1 ? 8 : 1][V][32];
    __shared__ float sm_w[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the attention kernel's writes are there
    const Cut cut = part.cuts[blockIdx.x];
    const int n = cut.parts, rows = cut.rows;
    if (n == 0 || blockIdx.y * RPB >= rows) return;
    auto slot_at = [&](int i) { return i == 0 ? (int64_t)cut.slot0 : 2 * ((int64_t)blockIdx.x + i * cut.twins); };
    const int sub = warp % WPR;
    const int row = blockIdx.y * RPB + warp / WPR;
    const bool live = row < rows;
    float M = -INFINITY, W = 0.f;
    float4 acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
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
                const float4 *o = reinterpret_cast<const float4 *>(part.o + at_row * R);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float4 x = o[32 * v + lane];
                    // an empty part (w = 0) holds zeros
                    acc[v].x = fmaf(w, x.x, acc[v].x);
                    acc[v].y = fmaf(w, x.y, acc[v].y);
                    acc[v].z = fmaf(w, x.z, acc[v].z);
                    acc[v].w = fmaf(w, x.w, acc[v].w);
                }
            }
        }
    }
    if (WPR > 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) sm_o[warp][v][lane] = acc[v];
        if (lane == 0) sm_w[warp] = W;
        __syncthreads();
        if (sub != 0 || !live) return;
        for (int k = 1; k < WPR; ++k) {
            W += sm_w[warp + k];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float4 x = sm_o[warp + k][v][lane];
                acc[v].x += x.x;
                acc[v].y += x.y;
                acc[v].z += x.z;
                acc[v].w += x.w;
            }
        }
    }
    if (!live) return;
    const int64_t out_row = cut.row_out + row;
    const float inv = W != 0.f ? 1.f / W : 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float4 x = make_float4(acc[v].x * inv, acc[v].y * inv, acc[v].z * inv, acc[v].w * inv);
        const int64_t e = out_row * R + 128 * v + 4 * lane;
        if (p.out_dtype == KF_F32) *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + e) = x;
        else
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + e) =
                make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
    }
    if (lane == 0 && p.lse_out) p.lse_out[out_row] = W != 0.f ? M + logf(W) : -INFINITY;
}

int64_t row_pitch(int max_query_len, int num_heads, int latent_dim) {
    const int64_t rows = (int64_t)max_query_len * num_heads;
    return std::min<int64_t>(rows, unit_rows(latent_dim));
}

// (64 columns, rows, column atoms): a box of a unit's rows x all columns lands as atoms
// of those rows x 128 swizzled bytes.
bool encode_q(tc::EncodeFn fn, CUtensorMap *map, const LatentParams &p) {
    const int width = p.latent_dim + kRopeDim;
    const cuuint64_t dims[3] = {64, (cuuint64_t)p.num_q_tokens * p.num_heads, (cuuint64_t)width / 64};
    const cuuint64_t strides[2] = {(cuuint64_t)width * 2, 128};
    const cuuint32_t box[3] = {64, (cuuint32_t)unit_rows(p.latent_dim), (cuuint32_t)width / 64};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(p.q), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// (64 columns, 8 tokens, column atoms, 8-token groups of all blocks): a box of 16
// tokens (which no block border cuts) lands group by group, each atom by atom.
bool encode_cache(tc::EncodeFn fn, CUtensorMap *map, const LatentParams &p) {
    const cuuint64_t row = (cuuint64_t)(p.latent_dim + kRopeDim) * 2;
    const cuuint64_t dims[4] = {64, 8, row / 128, (cuuint64_t)p.num_blocks * (p.block_size / 8)};
    const cuuint64_t strides[3] = {row, 128, 8 * row};
    const cuuint32_t box[4] = {64, 8, (cuuint32_t)(row / 128), 2};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t *>(p.cache), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int R>
cudaError_t launch(const LatentParams &p, const Partials &part, int ctas, int twins, bool decide, bool long_units,
                   cudaStream_t stream, const CUtensorMap &mx, const CUtensorMap &mq) {
    using Sh = LShape<R>;
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(done.load() & bit)) {
        e = cudaFuncSetAttribute(latent_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmemBytes);
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
    e = cudaLaunchKernelEx(&cfg, latent_kernel<R>, p, part, twins, decide, mx, mq);
    if (e != cudaSuccess || ctas == twins) return e;  // (one run: nothing is cut)
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    const int starts = ctas - (decide ? 1 : twins);  // CTAs where a unit may start that goes on
    if (long_units) {
        cfg.gridDim = dim3(starts, part.pitch);
        return cudaLaunchKernelEx(&cfg, latent_merge_kernel<R, 1>, p, part);
    }
    cfg.gridDim = dim3(starts, (part.pitch + 7) / 8);
    return cudaLaunchKernelEx(&cfg, latent_merge_kernel<R, 8>, p, part);
}

}  // namespace

namespace {
size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }
}  // namespace

size_t latent_workspace_bytes(int max_query_len, int num_heads, int latent_dim, int sm_count) {
    sm_count = std::max(sm_count, 2);
    const size_t rows = 2 * (size_t)sm_count * row_pitch(max_query_len, num_heads, latent_dim);
    return al256(rows * latent_dim * 4) + al256(rows * 4) + sm_count * sizeof(Cut);
}

cudaError_t launch_latent(const LatentParams &p, void *workspace, int sm_count, cudaStream_t stream, void *encode_fn) {
    tc::EncodeFn fn = reinterpret_cast<tc::EncodeFn>(encode_fn);
    sm_count = std::max(sm_count, 2);
    CUtensorMap mx, mq;
    if (!encode_cache(fn, &mx, p) || !encode_q(fn, &mq, p)) return cudaErrorInvalidValue;
    // Requests of more than one unit: two CTAs walk a run together, a unit each, so that
    // one's tiles are the other's L2 hits (64 requests of 4K tokens, 128 heads: 110 us
    // against 119, which read 550 MB from HBM for a cache of 302). With one unit a
    // request there is nothing to share. Where every request has as many queries as the
    // bound (all of q's tokens) that is known here, else the kernel looks (0.8 us).
    const int M = unit_rows(p.latent_dim);
    const int64_t rows_max = (int64_t)p.max_query_len * p.num_heads, units_max = (rows_max + M - 1) / M;
    const bool uniform = (int64_t)p.batch * p.max_query_len == p.num_q_tokens;
    const int twins = units_max > 1 && (!uniform || pairs_pay(units_max, units_max & 1)) ? 2 : 1;
    // No more units (groups of twins) than the bound, and than all query rows, allow; and no
    // more runs than these have pieces of 64 tokens (1 request of 777 tokens, 16 heads:
    // 16.7 us with 13 runs, 18.6 with 25 of 32 tokens).
    auto groups_of = [&](int64_t rows) {
        return std::min<int64_t>((int64_t)p.batch * ((rows_max + rows - 1) / rows),
                                 p.batch + (int64_t)p.num_q_tokens * p.num_heads / rows);
    };
    const int64_t pieces = groups_of(twins * M) * std::max<int64_t>(1, ((int64_t)p.max_context_len + 63) / 64);
    const int ctas = twins * (int)std::min<int64_t>(std::max(1, sm_count / twins), pieces);
    const bool decide = twins == 2 && !uniform && ctas > 2;
    Partials part;
    part.pitch = (int)row_pitch(p.max_query_len, p.num_heads, p.latent_dim);
    part.o = static_cast<float *>(workspace);
    const size_t rows = 2 * (size_t)sm_count * part.pitch;
    uint8_t *ws = static_cast<uint8_t *>(workspace) + al256(rows * p.latent_dim * 4);
    part.lse = reinterpret_cast<float *>(ws);
    part.cuts = reinterpret_cast<Cut *>(ws + al256(rows * 4));
    // few units are cut over many CTAs each: one row a merge block, its warps share
    // the partials; many units have two or three partials: one warp a row (1 request of
    // 30K tokens, 16 heads: 31 us against 76; 32 requests of 8K: 73 against 70)
    const bool long_units = groups_of(M) * 8 < ctas;
    return p.latent_dim == 512 ? launch<512>(p, part, ctas, twins, decide, long_units, stream, mx, mq)
                               : launch<256>(p, part, ctas, twins, decide, long_units, stream, mx, mq);
}

}  // namespace kf
