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
// one head (64 registers at D = 128), sixteen warps an SM some 128 KB in flight,
// against the 45-60 KB that cover HBM's latency. Q comes through L1.
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

constexpr int kWarps = 4, kTiles = 2;  // warps a CTA; 16-token tiles a warp holds

__device__ __forceinline__ uint4 load_stream(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

struct AccRequest {
    int64_t q0, C, L, shift;  // query j < C sees tokens t <= shift + j (causal)
};

__device__ __forceinline__ AccRequest acc_request(const AccumulateParams &p, int b, bool report) {
    int64_t q0 = b, q1 = b + 1;
    if (p.q_start) {
        q0 = p.q_start[b];
        q1 = p.q_start[b + 1];
    }
    if (q0 < 0 || q1 < q0 || q1 > p.num_q_tokens) {
        if (report) raise_error(p.err, KF_DEVERR_CONTEXT_LEN);
        return {0, 0, 0, 0};
    }
    AccRequest r;
    r.q0 = q0;
    r.C = q1 - q0;
    int64_t L = p.ctx_lens[b];
    const int64_t cap = (int64_t)p.bt_stride * p.block_size;
    if (L < 0 || L > cap) {
        if (report) raise_error(p.err, KF_DEVERR_CONTEXT_LEN);
        L = L < 0 ? 0 : cap;
    }
    r.shift = L - r.C;
    if ((L > p.max_context_len || r.C > p.max_query_len) && report) raise_error(p.err, KF_DEVERR_MAX_CONTEXT);
    r.L = L < p.max_context_len ? L : p.max_context_len;
    if (r.C > p.max_query_len) r.C = p.max_query_len;
    return r;
}

template <int D, bool KV8>
__global__ void __launch_bounds__(32 * kWarps, 4)
accumulate_kernel(const AccumulateParams p) {
    constexpr int NL = KV8 ? D / 64 : D / 32;   // 16-byte loads a lane and K row
    constexpr int NQ = D / 32;                  // 16-byte loads a lane and q row
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

        // rows of this lane's tokens (tile k, rows g and g + 8)
        const uint8_t *row[kTiles][2];
#pragma unroll
        for (int k = 0; k < kTiles; ++k) {
            const int64_t t = (tile0 + (k < tiles ? k : 0)) * 16;
            int64_t phys = p.block_tables[(int64_t)b * p.bt_stride + t / p.block_size];
            if (phys < 0 || phys >= p.num_blocks) {
                if (lane == 0) raise_error(p.err, KF_DEVERR_BLOCK_ID);
                phys = 0;
            }
            const int64_t first = phys * p.block_size + t % p.block_size;
#pragma unroll
            for (int u = 0; u < 2; ++u)
                row[k][u] = static_cast<const uint8_t *>(p.k_cache) +
                            (first + g + 8 * u) * p.num_kv_heads * (D * EB) + t4 * 16;
        }
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
            for (int64_t c0 = col0; c0 < cols; c0 += 8) {
                // this lane's q row: column c0 + g (zeros past the last)
                uint4 q[NQ];
                const int64_t col = c0 + g;
                const uint16_t *qrow =
                    p.q + (((r.q0 + (col >> log_g)) * p.num_q_heads) + h * G + (col & (G - 1))) * D;
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    // bf16 K: chunk t4 + 4 i of 8 numbers; E4M3 K: 16 numbers at 16 (t4 + 4 (i / 2))
                    const int e = KV8 ? 16 * (t4 + 4 * (i >> 1)) + 8 * (i & 1) : 8 * (t4 + 4 * i);
                    q[i] = col < cols ? __ldg(reinterpret_cast<const uint4 *>(qrow + e)) : make_uint4(0, 0, 0, 0);
                }
                float unscale = kscale;  // of column c0 + g
                if (KV8) {
                    float mx = 0.f;
#pragma unroll
                    for (int i = 0; i < NQ; ++i) {
                        const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
                    }
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    // 2^(14 - exponent of mx), its exponent kept where both it and its inverse are normal
                    int ex = (int)((__float_as_uint(mx) >> 23) & 255) - 127;
                    ex = ex < -100 ? -100 : ex;
                    const float up = __uint_as_float((uint32_t)(14 - ex + 127) << 23);
                    unscale *= __uint_as_float((uint32_t)(ex - 14 + 127) << 23);
#pragma unroll
                    for (int i = 0; i < NQ; ++i) {
                        uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] = pack_f16(bf16_lo(w[e]) * up, bf16_hi(w[e]) * up);
                        q[i] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                // the two columns of this lane's results: their lse and scale
                float lse2[2], c[2];
                int64_t hide[2];  // tokens above this are not seen
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int64_t cc = c0 + 2 * t4 + u;
                    float l = INFINITY;  // weight 0
                    if (cc < cols)
                        l = p.lse[(r.q0 + (cc >> log_g)) * p.num_q_heads + h * G + (cc & (G - 1))];
                    lse2[u] = l == -INFINITY ? INFINITY : l * 1.4426950408889634f;
                    // (column n's row maximum lives in lanes 4 n .. 4 n + 3)
                    c[u] = p.scale_log2 * (KV8 ? __shfl_sync(0xffffffffu, unscale, 4 * (2 * t4 + u)) : 1.f);
                    hide[u] = p.causal ? r.shift + (cc >> log_g) : r.L;
                }
#pragma unroll
                for (int k = 0; k < kTiles; ++k) {
                    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < NL; ++i) {
                        const uint4 ka = kr[k][0][i], kb = kr[k][1][i];
                        if (KV8) {
                            const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t a[4] = {e4m3x2_to_f16x2(wa[e]), e4m3x2_to_f16x2(wb[e]),
                                                       e4m3x2_to_f16x2(wa[e] >> 16), e4m3x2_to_f16x2(wb[e] >> 16)};
                                const uint4 qq = q[2 * i + (e >> 1)];
                                if (e & 1) mma_f16(s, a, qq.z, qq.w);
                                else mma_f16(s, a, qq.x, qq.y);
                            }
                        } else {
                            const uint32_t a0[4] = {ka.x, kb.x, ka.y, kb.y}, a1[4] = {ka.z, kb.z, ka.w, kb.w};
                            mma_bf16(s, a0, q[i].x, q[i].y);
                            mma_bf16(s, a1, q[i].z, q[i].w);
                        }
                    }
                    const int64_t t = (tile0 + k) * 16 + g;
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int w = 0; w < 2; ++w)
                            if (t + 8 * w <= hide[u])
                                sum[k][w] += exp2_approx(fmaf(s[2 * w + u], c[u], -lse2[u]));
                }
            }
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

}  // namespace

cudaError_t launch_accumulate(const AccumulateParams &p, int sm_count, cudaStream_t stream) {
    // one wave of resident CTAs, no more warps than the batch can have tiles
    const int64_t tiles = (int64_t)p.batch * ((p.max_context_len + 15) / 16);
    const int64_t ctas = (tiles + kWarps - 1) / kWarps < 4ll * sm_count ? (tiles + kWarps - 1) / kWarps : 4ll * sm_count;
    const dim3 grid((unsigned)ctas), block(32 * kWarps);
    if (p.k_scale) {
        if (p.head_dim == 128) accumulate_kernel<128, true><<<grid, block, 0, stream>>>(p);
        else accumulate_kernel<64, true><<<grid, block, 0, stream>>>(p);
    } else {
        if (p.head_dim == 128) accumulate_kernel<128, false><<<grid, block, 0, stream>>>(p);
        else accumulate_kernel<64, false><<<grid, block, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace kf
