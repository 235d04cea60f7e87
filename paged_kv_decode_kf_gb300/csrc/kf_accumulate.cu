// kf_accumulate.cu -- attention weight each cached token receives.
//
//   scores_out[b, t] = scores_in[b, t] + sum_{j sees t} sum_h exp(scale <q_jh, k_{h/G, t}> - lse_jh)
//
// The softmax's statistics are known (lse), so one pass over K is enough, with no
// reduction between tokens. Per KV head the queries' rows (j, g) are columns of
//   S[16 tokens x 8 columns] += K[16 x 16] Q^T[16 x 8]   (mma.sync m16n8k16)
// taken 8 at a time; a column's weight is exp2(S * scale * log2 e - lse * log2 e)
// and a token's sum runs over its row of S, then over column groups and heads, in
// one warp: the same order every time, no atomics.
//
// Why mma.sync and not tcgen05: one query token a request gives G <= 8 columns, and
// K is read once. The order of the 16 numbers inside a k step is free as long
// as K and Q agree, so a lane's fragment is 16 consecutive bytes of a K row, loaded
// from global memory straight into registers: no shared memory, no barrier, and the
// four lanes of a row cover 64 contiguous bytes a load. A warp holds 32 tokens of
// one head (64 E4M3 ones; 64 registers at D = 128), twelve warps an SM some 96 KB in
// flight, against the 45-60 KB that cover HBM's latency. Q comes through L1.
// Measured: 64 requests of 4K tokens, 32 / 8 heads, bf16: 89 us, 5.7 TB/s of K.
// E4M3 keys widen to fp16 (exact); q goes to fp16 times a power of two that puts
// the row's largest magnitude just below 2^15 (exact for every number within 2^-29
// of it), undone with the key's scale.
//
// What bounds it: K's bytes (Hkv * D * 2, or 1, a token) for one query token a
// request; with a window of C queries the 2 C G D operations a (token, head),
// from some 16 columns a head on, at mma.sync's rate.
//
// Work: the batch's 16-token tiles, end to end, are cut into equal runs, one a
// warp; a tile never crosses a cache block (16 or 32 tokens).
#include "kf_decode_tc.cuh"
#include "kf_evict.cuh"
#include "kf_runs.cuh"

namespace kf {
namespace {

using namespace tc;

constexpr int kWarps = 4;  // warps a CTA
// 16-token tiles a warp holds, and CTAs an SM: as many keys in flight either way, and
// enough of them a warp to pay for q's conversion (64 requests of 4K, bf16: 90 us with
// 2 tiles x 3 CTAs, 93 with 2 x 4, 96 with 1 x 6 and 4 x 2; ragged E4M3: 146 us with
// 4 x 3, 155 with 2 x 4, 199 with 1 x 6, and 136 once L2 fetches keys by 256 bytes). Three
// CTAs leave a thread 168 registers: E4M3 at D = 128 spills 60 bytes there.
template <bool KV8>
struct Held {
    static constexpr int kTiles = KV8 ? 4 : 2, kCtas = 3;
};

__device__ __forceinline__ uint4 load_stream(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Eight columns (j, g) of one KV head as B fragments: lane (g, t4) holds part t4 of
// column c0 + g; and of its two result columns 2 t4, 2 t4 + 1 the lse, the scale
// and the last token they see.
template <int D>
struct Columns {
    static constexpr int NQ = D / 32;  // 16-byte loads a lane and q row
    uint4 q[NQ];
    float lse2[2], c[2];
    int hide[2];

    template <bool KV8>
    __device__ __forceinline__ void ready(float scale_log2, float kscale) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (lse2[u] == -INFINITY) hide[u] = -1;  // nothing, whatever its scores are
            lse2[u] *= 1.4426950408889634f;
            c[u] = scale_log2;
        }
        if (KV8) {
            const int t4 = threadIdx.x & 3;
            float mx = 0.f;
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            // times 2^(14 - exponent of mx), where both it and its inverse are normal numbers
            int ex = (int)((__float_as_uint(mx) >> 23) & 255) - 127;
            ex = ex < -100 ? -100 : ex;
            const float up = __uint_as_float((uint32_t)(14 - ex + 127) << 23);
            const float unscale = kscale * __uint_as_float((uint32_t)(ex - 14 + 127) << 23);
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = pack_f16(bf16_lo(w[e]) * up, bf16_hi(w[e]) * up);
                q[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            // (column n's scale lives in lanes 4 n .. 4 n + 3)
#pragma unroll
            for (int u = 0; u < 2; ++u) c[u] *= __shfl_sync(0xffffffffu, unscale, 4 * (2 * t4 + u));
        }
    }
};

// Where a lane's columns lie, from column c0 on; `step` columns further at a time.
template <int D, bool KV8>
struct ColumnWalk {
    const uint16_t *q;       // row of column c0 + g, from this lane's part on
    const float *lse[2];     // of columns c0 + 2 t4 and + 1
    int64_t q_stride, lse_stride;
    int hide[2], hide_stride;
    int left;                // columns from c0 on

    __device__ __forceinline__ ColumnWalk(const AccumulateParams &p, const AccRequest &r, int h, int64_t c0,
                                          int64_t cols, int step, int log_g) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
        const int G = 1 << log_g;
        const int64_t col = c0 + g;
        // bf16 K: chunk t4 + 4 i of 8 numbers; E4M3 K: 16 numbers at 16 (t4 + 4 (i / 2))
        q = p.q + (((r.q0 + (col >> log_g)) * p.num_q_heads) + h * G + (col & (G - 1))) * D + (KV8 ? 16 : 8) * t4;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int64_t cc = c0 + 2 * t4 + u;
            lse[u] = p.lse + (r.q0 + (cc >> log_g)) * p.num_q_heads + h * G + (cc & (G - 1));
            hide[u] = (int)(p.causal ? r.shift + (cc >> log_g) : r.L);  // (lengths are 32-bit)
        }
        // (step is a multiple of 8, and so of G)
        lse_stride = (int64_t)(step >> log_g) * p.num_q_heads;
        q_stride = lse_stride * D;
        hide_stride = p.causal ? step >> log_g : 0;
        left = (int)(cols - c0);
    }

    // Asks for eight columns (zeros, with the lse of a row that saw nothing, past the
    // last: zero times an infinite key is no number); Columns::ready makes them fragments. What lies between the two hides the loads.
    __device__ __forceinline__ void load(Columns<D> &x) const {
        const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int i = 0; i < Columns<D>::NQ; ++i) {
            const int e = KV8 ? 64 * (i >> 1) + 8 * (i & 1) : 32 * i;
            x.q[i] = g < left ? __ldg(reinterpret_cast<const uint4 *>(q + e)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            x.lse2[u] = 2 * t4 + u < left ? __ldg(lse[u]) : -INFINITY;
            x.hide[u] = hide[u];
        }
    }

    __device__ __forceinline__ bool next(int step) {
        left -= step;
        q += q_stride;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            lse[u] += lse_stride;
            hide[u] += hide_stride;
        }
        return left > 0;
    }
};

// sum[k][w] += the weights the eight columns give the tokens t0 + 16 k + g + 8 w.
template <int D, bool KV8, int T>
__device__ __forceinline__ void add_columns(const uint4 (&kr)[T][2][KV8 ? D / 64 : D / 32], const Columns<D> &q,
                                            int t0, float (&sum)[T][2]) {
    const int g = (threadIdx.x & 31) >> 2;
    float s[T][4];
#pragma unroll
    for (int k = 0; k < T; ++k) s[k][0] = s[k][1] = s[k][2] = s[k][3] = 0.f;
    // (tiles innermost: T independent chains of products)
#pragma unroll
    for (int i = 0; i < (KV8 ? D / 64 : D / 32); ++i) {
        if (KV8) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint4 qq = q.q[(2 * i + (e >> 1)) % (D / 32)];
#pragma unroll
                for (int k = 0; k < T; ++k) {
                    const uint4 ka = kr[k][0][i], kb = kr[k][1][i];
                    const uint32_t wa = e == 0 ? ka.x : e == 1 ? ka.y : e == 2 ? ka.z : ka.w;
                    const uint32_t wb = e == 0 ? kb.x : e == 1 ? kb.y : e == 2 ? kb.z : kb.w;
                    const uint32_t a[4] = {e4m3x2_to_f16x2(wa), e4m3x2_to_f16x2(wb), e4m3x2_to_f16x2(wa >> 16),
                                           e4m3x2_to_f16x2(wb >> 16)};
                    if (e & 1) mma_f16(s[k], a, qq.z, qq.w);
                    else mma_f16(s[k], a, qq.x, qq.y);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < T; ++k) {
                const uint32_t a[4] = {kr[k][0][i].x, kr[k][1][i].x, kr[k][0][i].y, kr[k][1][i].y};
                mma_bf16(s[k], a, q.q[i].x, q.q[i].y);
            }
#pragma unroll
            for (int k = 0; k < T; ++k) {
                const uint32_t a[4] = {kr[k][0][i].z, kr[k][1][i].z, kr[k][0][i].w, kr[k][1][i].w};
                mma_bf16(s[k], a, q.q[i].z, q.q[i].w);
            }
        }
    }
    // (all the tokens a lane has may be hidden from a column: the newest ones from older
    // queries, all of them from a column that adds nothing)
    if (__all_sync(0xffffffffu, t0 + 16 * T - 1 <= min(q.hide[0], q.hide[1]))) {
#pragma unroll
        for (int k = 0; k < T; ++k)
#pragma unroll
            for (int w = 0; w < 2; ++w)
                sum[k][w] += exp2_approx(fmaf(s[k][2 * w], q.c[0], -q.lse2[0])) +
                             exp2_approx(fmaf(s[k][2 * w + 1], q.c[1], -q.lse2[1]));
    } else {
#pragma unroll
        for (int k = 0; k < T; ++k)
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    if (t0 + 16 * k + g + 8 * w <= q.hide[u])
                        sum[k][w] += exp2_approx(fmaf(s[k][2 * w + u], q.c[u], -q.lse2[u]));
    }
}

// This lane's K rows of T 16-token tiles (rows g and g + 8), from part t4 of KV head 0
// on; tiles past the last repeat it.
template <int D, bool KV8, int T>
__device__ __forceinline__ void key_rows(const AccumulateParams &p, int b, int64_t tile0, int tiles,
                                         const uint8_t *(&row)[T][2]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
#pragma unroll
    for (int k = 0; k < T; ++k) {
        const int t = (int)(tile0 + (k < tiles ? k : tiles - 1)) * 16;
        int64_t phys = p.block_tables[(int64_t)b * p.bt_stride + (t >> block_shift(p.block_size))];
        if (phys < 0 || phys >= p.num_blocks) {
            if (lane == 0) raise_error(p.err, KF_DEVERR_BLOCK_ID);
            phys = 0;
        }
        const int64_t first = phys * p.block_size + (t & (p.block_size - 1));
#pragma unroll
        for (int u = 0; u < 2; ++u)
            row[k][u] = static_cast<const uint8_t *>(p.k_cache) +
                        (first + g + 8 * u) * p.num_kv_heads * (D * (KV8 ? 1 : 2)) + t4 * 16;
    }
}

template <int D, bool KV8>
__global__ void __launch_bounds__(32 * kWarps, Held<KV8>::kCtas)
accumulate_kernel(const AccumulateParams p) {
    constexpr int kTiles = Held<KV8>::kTiles;
    constexpr int NL = KV8 ? D / 64 : D / 32;   // 16-byte loads a lane and K row
    constexpr int EB = KV8 ? 1 : 2;
    __shared__ int64_t sm_loc[36];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t4 = lane & 3;

    // runs are cut for warps; this CTA's first one starts at `at`
    const int64_t runs = (int64_t)gridDim.x * kWarps;
    Place at;
    int64_t cta_first;
    const int64_t total = locate(
        p.batch, [&](int b) { return (acc_request(p, b, blockIdx.x == 0).L + 15) / 16; }, sm_loc,
        [&](int64_t T) { return (int64_t)blockIdx.x * kWarps * T / runs; }, at, cta_first);
    const int64_t run = (int64_t)blockIdx.x * kWarps + warp;
    int64_t idx = run * total / runs;
    const int64_t end = (run + 1) * total / runs;
    if (idx >= end) return;
    int b = at.b;
    int64_t req_first = cta_first - at.off;  // the request's first tile in the batch's list
    AccRequest r = acc_request(p, b, false);
    const int G = p.num_q_heads / p.num_kv_heads;
    const int log_g = 31 - __clz(G);

    while (idx < end) {
        int64_t n = (r.L + 15) / 16;
        while (idx >= req_first + n) {  // on to the request of tile idx (it exists: idx < total)
            req_first += n;
            r = acc_request(p, ++b, false);
            n = (r.L + 15) / 16;
        }
        const int64_t tile0 = idx - req_first;
        int64_t tiles = n - tile0 < end - idx ? n - tile0 : end - idx;
        if (tiles > kTiles) tiles = kTiles;

        const uint8_t *row[kTiles][2];
        key_rows<D, KV8, kTiles>(p, b, tile0, (int)tiles, row);
        float sum[kTiles][2] = {};
        const int64_t cols = r.C << log_g;
        // with a causal window, columns of queries before the first that sees this tile add nothing
        int64_t col0 = 0;
        if (p.causal && tile0 * 16 > r.shift) col0 = ((tile0 * 16 - r.shift) << log_g) & ~7ll;
        for (int h = 0; h < p.num_kv_heads && col0 < cols; ++h) {
            uint4 kr[kTiles][2][NL];
#pragma unroll
            for (int k = 0; k < kTiles; ++k)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < NL; ++i)
                        kr[k][u][i] = load_stream(row[k][u] + (int64_t)h * (D * EB) + i * 64);
            const float kscale = KV8 ? p.k_scale[h] : 1.f;
            ColumnWalk<D, KV8> walk(p, r, h, col0, cols, 8, log_g);
            do {
                Columns<D> q;
                walk.load(q);
                q.template ready<KV8>(p.scale_log2, kscale);
                add_columns<D, KV8, kTiles>(kr, q, (int)tile0 * 16, sum);
            } while (walk.next(8));
        }
#pragma unroll
        for (int k = 0; k < kTiles; ++k) {
            const int64_t t = (tile0 + k) * 16 + g;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                float x = sum[k][w];
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                if (k < tiles && t4 == w && t + 8 * w < r.L) {
                    const int64_t at = b * p.score_stride + t + 8 * w;
                    p.scores_out[at] = (p.scores_in ? p.scores_in[at] : 0.f) + x;
                }
            }
        }
        idx += tiles;
    }
}

// Windows of queries (more than eight columns a KV head) over E4M3 keys: one CTA a run of 64 tokens,
// its eight warps split the (KV head, column group) pairs, so that the tokens' keys
// are held while the columns pass (64 registers at D = 128, of 214: one CTA an SM) and q,
// which every CTA reads whole, is read once per 64 tokens. The next group's q is asked for
// before this one's products. The warps' sums meet in shared memory, in warp order. What
// bounds it: keys widened again for every eight columns, and mma.sync: 4 requests of
// 4K-12K tokens, 32 / 64 queries of 32 / 8 heads: 62 / 110 us (bf16 keys on tcgen05: 22 / 35).
constexpr int kWinWarps = 8, kWinTiles = 4;

template <int D>
__global__ void __launch_bounds__(32 * kWinWarps, 1)
accumulate_window_kernel(const AccumulateParams p) {
    constexpr bool KV8 = true;
    constexpr int NL = D / 64, EB = 1;
    __shared__ int64_t sm_loc[36];
    __shared__ float part[kWinWarps][kWinTiles * 16];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t4 = lane & 3;
    const int log_g = 31 - __clz(p.num_q_heads / p.num_kv_heads);
    auto runs_of = [&](int b, bool report) {
        return (acc_request(p, b, report).L + 16 * kWinTiles - 1) / (16 * kWinTiles);
    };
    Place at;
    int64_t idx;
    const int64_t total = locate(
        p.batch, [&](int b) { return runs_of(b, blockIdx.x == 0); }, sm_loc,
        [&](int64_t T) { return cut_at(blockIdx.x, gridDim.x, T); }, at, idx);
    const int64_t end = cut_at(blockIdx.x + 1, gridDim.x, total);
    int b = at.b;
    int64_t run = at.off, n = idx < end ? runs_of(b, false) : 0;
    // warps of one head share its columns; with more heads than warps, heads take turns
    const int heads = p.num_kv_heads, share = heads < kWinWarps ? kWinWarps / heads : 1;
    for (; idx < end; ++idx, ++run) {
        while (run >= n) {  // on to the next request with tokens (it exists: idx < total)
            run = 0;
            n = runs_of(++b, false);
        }
        const AccRequest r = acc_request(p, b, false);
        const int64_t t0 = run * 16 * kWinTiles;
        const int tiles = (int)(((r.L - t0 < 16 * kWinTiles ? r.L - t0 : 16 * kWinTiles) + 15) / 16);
        const uint8_t *row[kWinTiles][2];
        key_rows<D, KV8, kWinTiles>(p, b, run * kWinTiles, tiles, row);
        float sum[kWinTiles][2] = {};
        const int64_t cols = r.C << log_g;
        // with a causal window, columns of queries before the first that sees this run add nothing
        int64_t col0 = 0;
        if (p.causal && t0 > r.shift) col0 = ((t0 - r.shift) << log_g) & ~7ll;
        const int step = 8 * share;
        for (int h = warp / share; h < heads; h += kWinWarps) {
            int64_t c0 = col0 + 8 * (warp % share);
            if (c0 >= cols) continue;
            const float kscale = p.k_scale[h];
            ColumnWalk<D, KV8> walk(p, r, h, c0, cols, step, log_g);
            Columns<D> q;
            walk.load(q);
            uint4 kr[kWinTiles][2][NL];
#pragma unroll
            for (int k = 0; k < kWinTiles; ++k)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < NL; ++i) kr[k][u][i] = load_stream(row[k][u] + (int64_t)h * (D * EB) + i * 64);
            while (true) {
                Columns<D> next;
                q.template ready<KV8>(p.scale_log2, kscale);
                const bool more = walk.next(step);
                if (more) walk.load(next);
                add_columns<D, KV8, kWinTiles>(kr, q, (int)t0, sum);
                if (!more) break;
                q = next;
            }
        }
#pragma unroll
        for (int k = 0; k < kWinTiles; ++k)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                float x = sum[k][w];
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                if (t4 == w) part[warp][16 * k + g + 8 * w] = x;
            }
        __syncthreads();
        const int64_t t = t0 + threadIdx.x;
        if (threadIdx.x < 16 * kWinTiles && t < r.L) {
            float x = 0.f;
#pragma unroll
            for (int w = 0; w < kWinWarps; ++w) x += part[w][threadIdx.x];
            const int64_t where = b * p.score_stride + t;
            p.scores_out[where] = (p.scores_in ? p.scores_in[where] : 0.f) + x;
        }
        __syncthreads();
    }
}

template <int D, bool KV8>
cudaError_t launch(const AccumulateParams &p, int sm_count, cudaStream_t stream, void *encode_fn) {
    // Columns a KV head: up to eight are one pass of the row kernel; more keep the keys
    // while the columns pass, bf16 ones on tcgen05 (E4M3 ones would have to be widened to
    // bf16 in shared memory for it, which is not built: accumulate_window_kernel). 64
    // requests of 4K tokens, 8 / 16 / 32 columns: 94 / 110 / 152 us with the row kernel, 106
    // / 107 / 107 on tcgen05.
    const int64_t cols = (int64_t)p.max_query_len * (p.num_q_heads / p.num_kv_heads);
    if (!KV8 && cols > 8 && p.num_q_tokens > 0) return launch_accumulate_tc05(p, sm_count, stream, encode_fn);
    const int64_t tiles = (int64_t)p.batch * ((p.max_context_len + 15) / 16);
    // one wave of resident CTAs, no more warps (CTAs) than the batch can have tiles (runs)
    if (cols <= 8) {
        const int64_t wave = (int64_t)Held<KV8>::kCtas * sm_count, need = (tiles + kWarps - 1) / kWarps;
        const int64_t ctas = need < wave ? need : wave;
        accumulate_kernel<D, KV8><<<(unsigned)ctas, 32 * kWarps, 0, stream>>>(p);
    } else {
        const int64_t runs = (int64_t)p.batch * ((p.max_context_len + 16 * kWinTiles - 1) / (16 * kWinTiles));
        accumulate_window_kernel<D><<<(unsigned)(runs < sm_count ? runs : sm_count), 32 * kWinWarps, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_accumulate(const AccumulateParams &p, int sm_count, cudaStream_t stream, void *encode_fn) {
    if (p.k_scale)
        return p.head_dim == 128 ? launch<128, true>(p, sm_count, stream, encode_fn)
                                 : launch<64, true>(p, sm_count, stream, encode_fn);
    return p.head_dim == 128 ? launch<128, false>(p, sm_count, stream, encode_fn)
                             : launch<64, false>(p, sm_count, stream, encode_fn);
}

}  // namespace kf
