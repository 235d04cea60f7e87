// kf_evict.cuh -- launch functions of the accumulated attention weights and of
// the eviction that uses them.
#pragma once

#include "kf_internal.cuh"

namespace kf {

struct AccumulateParams {
    const uint16_t *q;            // bf16 [num_q_tokens, Hq, D]
    const int32_t *q_start;       // [batch + 1], or null: query token b is request b's
    const void *k_cache;          // bf16 or E4M3 [NB, bs, Hkv, D]
    const float *k_scale;         // E4M3: per-KV-head scales, else null
    const int32_t *block_tables;
    const int32_t *ctx_lens;
    const float *lse;             // f32 [num_q_tokens, Hq]
    const float *scores_in;       // f32 [batch, score_stride] or null
    float *scores_out;            // f32 [batch, score_stride]
    unsigned int *err;
    int64_t num_blocks, score_stride;
    int bt_stride, max_context_len, max_query_len;
    int batch, num_q_tokens, num_q_heads, num_kv_heads, head_dim, block_size, causal;
    float scale_log2;
};

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

cudaError_t launch_accumulate(const AccumulateParams &p, int sm_count, cudaStream_t stream, void *encode_fn);
// bf16 keys and more than eight (query, head) columns a KV head.
cudaError_t launch_accumulate_tc05(const AccumulateParams &p, int sm_count, cudaStream_t stream, void *encode_fn);

struct EvictParams {
    uint4 *cache_a, *cache_b;     // [NB, bs] rows of row_vecs 16-byte vectors; cache_b may be null
    const int32_t *block_tables;
    const int32_t *ctx_lens;
    const float *scores;          // [batch, score_stride]
    float *scores_out;
    const int32_t *positions;     // [batch, score_stride] or null
    int32_t *positions_out;
    const int32_t *seq_lens;      // [batch], with positions
    int32_t *ctx_out;             // [batch]
    unsigned int *err;
    int *counts;                  // workspace: moves of each request
    int *dst, *src;               // workspace: [batch, max_moves] token indices
    int64_t num_blocks, score_stride;
    int row_vecs, bt_stride, max_context_len, batch, block_size;
    int keep, sink, recent, max_moves;
};

cudaError_t launch_evict(const EvictParams &p, int sm_count, cudaStream_t stream);

}  // namespace kf
