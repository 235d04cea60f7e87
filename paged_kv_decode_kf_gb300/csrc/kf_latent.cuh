// kf_latent.cuh -- parameters and helpers shared by the latent-attention
// kernels (append, absorbed form, expanded form).
//
// A latent cache holds one row a token for all heads: [c_t (R) ; k_rope_t (64)]
// in bf16, [num_blocks, block_size, R + 64]. Head h's key is [W_uk_h c_t ;
// k_rope_t] and its value W_uv_h c_t.
#pragma once

#include "kf_internal.cuh"

namespace kf {

constexpr int kRopeDim = 64;

struct LatentParams {
    const uint16_t *q;            // bf16 [num_q_tokens, H, key width]
    const int32_t *q_start;       // [batch + 1], or null: query token b is request b's
    const uint16_t *cache;        // bf16 [NB, bs, R + 64]
    const int32_t *block_tables;
    const int32_t *ctx_lens;      // [batch], tokens in the cache, the queries' own included
    void *out;                    // [num_q_tokens, H, value width] of out_dtype
    float *lse_out;               // [num_q_tokens, H] or null
    unsigned int *err;
    int64_t num_blocks;
    int bt_stride;
    int max_context_len, max_query_len;
    int batch, num_q_tokens, num_heads, latent_dim, block_size;
    int causal, out_dtype;
    float scale_log2;             // scale * log2(e)
};

// The query rows and the tokens of one request. q0 < 0: nothing to do.
struct LatentRequest {
    int64_t q0, C, L;
};

// Reads and checks request b's ranges. A range outside q touches nothing; a
// length outside the table is reported and clamped; tokens and queries above
// the host's bounds are reported and left out. C > L is no error: the first
// C - L queries of a causal call see no token.
__device__ __forceinline__ LatentRequest latent_request(const LatentParams &p, int b, bool report) {
    LatentRequest r;
    int64_t q0 = b, q1 = b + 1;
    if (p.q_start) {
        q0 = p.q_start[b];
        q1 = p.q_start[b + 1];
    }
    if (q0 < 0 || q1 < q0 || q1 > p.num_q_tokens) {
        if (report) raise_error(p.err, KF_DEVERR_CONTEXT_LEN);
        return {-1, 0, 0};
    }
    r.q0 = q0;
    r.C = q1 - q0;
    r.L = p.ctx_lens[b];
    const int64_t cap = (int64_t)p.bt_stride * p.block_size;
    if (r.L < 0 || r.L > cap) {
        if (report) raise_error(p.err, KF_DEVERR_CONTEXT_LEN);
        r.L = r.L < 0 ? 0 : (r.L > cap ? cap : r.L);
    }
    if (r.L > p.max_context_len) {
        if (report) raise_error(p.err, KF_DEVERR_MAX_CONTEXT);
    }
    if (r.C > p.max_query_len) {
        if (report) raise_error(p.err, KF_DEVERR_MAX_CONTEXT);
    }
    return r;
}

cudaError_t launch_append_latent(const uint16_t *rows, const int32_t *row_start, uint16_t *cache,
                                 const int32_t *block_tables, int bt_stride, const int32_t *ctx_before, int batch,
                                 int num_rows, int row_dim, int block_size, int64_t num_blocks, unsigned int *err,
                                 cudaStream_t stream);

// Absorbed form: the partials of cut units in `workspace` (their o, lse and Cut records, two
// slots an SM: kf_latent_tc05.cu).
size_t latent_workspace_bytes(int max_query_len, int num_heads, int latent_dim, int sm_count);
cudaError_t launch_latent(const LatentParams &p, void *workspace, int sm_count, cudaStream_t stream, void *encode_fn);

// Expanded form: K_nope and V of every token in `workspace`.
struct LatentWeights {
    const uint16_t *w_uk;  // bf16 [H, nope, R]
    const uint16_t *w_uv;  // bf16 [H, v, R]
    int nope, v;
};
size_t latent_expanded_workspace_bytes(int batch, int max_context_len, int num_heads, int nope, int v);
cudaError_t launch_latent_expanded(const LatentParams &p, const LatentWeights &w, void *workspace, int sm_count,
                                   cudaStream_t stream, void *encode_fn);

}  // namespace kf
