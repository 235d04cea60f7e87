// kf_tree.cuh -- trees of drafted tokens: attention (kf_tree.cu), the greedy walk and
// the accepted rows' moves (kf_tree_accept.cu).
#pragma once

#include "kf_internal.cuh"

namespace kf {

constexpr int kMaxNodes = 256;  // a request's drafted tokens

struct TreeParams {
    const uint16_t *q;            // bf16 [num_q_tokens, Hq, D]
    const int32_t *q_start;       // [batch + 1], or null: one node a request
    const int32_t *parents;       // [num_q_tokens]
    const void *k_cache, *v_cache;
    const float *k_scale, *v_scale;  // E4M3 caches, else null
    const int32_t *block_tables;
    const int32_t *ctx_lens;      // [batch], the nodes included
    void *out;                    // [num_q_tokens, Hq, D] of out_dtype
    float *lse_out;               // [num_q_tokens, Hq] or null
    unsigned int *err;
    int64_t num_blocks;
    int bt_stride;
    int max_context_len, max_query_len;
    int batch, num_q_tokens, num_q_heads, num_kv_heads, head_dim, block_size;
    int out_dtype;
    float scale_log2;             // scale * log2(e)
};

// The nodes and the tokens of one request. q0 < 0: nothing to do.
struct TreeRequest {
    int64_t q0, C, L;
};

// Reads and checks request b's ranges. A request whose lengths do not fit -- its nodes
// outside q or above the host's bound, fewer cached tokens than nodes, more than the
// table or the host's bound holds -- is reported and left out whole (its window of nodes
// is at its end, so that no part of it would be right).
__device__ __forceinline__ TreeRequest tree_request(const int32_t *q_start, const int32_t *ctx_lens, int b,
                                                    int64_t num_q_tokens, int64_t max_nodes, int64_t max_ctx,
                                                    int64_t cap, unsigned int *err) {
    int64_t q0 = b, q1 = b + 1;
    if (q_start) {
        q0 = q_start[b];
        q1 = q_start[b + 1];
    }
    const int64_t C = q1 - q0, L = ctx_lens[b];
    unsigned int bad = 0;
    if (q0 < 0 || q1 < q0 || q1 > num_q_tokens || L < C || L > cap) bad = KF_DEVERR_CONTEXT_LEN;
    else if (C > max_nodes || L > max_ctx) bad = KF_DEVERR_MAX_CONTEXT;
    if (bad) {
        if (err) raise_error(err, bad);
        return {-1, 0, 0};
    }
    return {q0, C, L};
}

size_t tree_workspace_bytes(int max_query_len, int num_q_heads, int num_kv_heads, int head_dim, bool f32, int sm_count);
cudaError_t launch_tree(const TreeParams &p, void *workspace, int sm_count, cudaStream_t stream, void *encode_fn);

struct AcceptArgs {
    const int32_t *parents, *draft, *target, *q_start, *ctx_lens;
    int32_t *path, *accepted, *next, *ctx_out;
    unsigned int *err;
    int path_stride, max_nodes, batch, num_q_tokens;
};
cudaError_t launch_accept(const AcceptArgs &a, cudaStream_t stream);

struct CommitArgs {
    uint4 *cache[2];          // the second may be null
    const int32_t *block_tables, *ctx_lens, *q_start, *path, *accepted;
    unsigned int *err;
    int64_t num_blocks;
    int row_vecs, bt_stride, path_stride, batch, block_size;
};
cudaError_t launch_commit(const CommitArgs &a, cudaStream_t stream);

}  // namespace kf
