// kf_prompt_tree_api.cu -- the C entry points of prompt attention, draft trees and block
// tables, declared in include/kf.h: argument checks on the host, then one launch
// function each.
#include <math.h>

#include <algorithm>

#include "kf_device.cuh"
#include "kf_prompt.cuh"
#include "kf_tables.cuh"
#include "kf_tree.cuh"

using namespace kf;

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxBatch = 65535;

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool block_ok(int bs) { return bs == 16 || bs == 32; }
bool heads_ok(int q, int kv, int dim) {
    if (q % kv != 0 || (dim != 64 && dim != 128)) return false;
    const int g = q / kv;
    return g == 1 || g == 2 || g == 4 || g == 8;
}

// Token indices, and those a tile or a block's stride further on, stay in 31 bits.
constexpr int64_t kMaxTokens = (int64_t)1 << 30;

// A launch refused for its shape (a grid or tensor map that does not fit) is an
// unsupported shape; anything else is a CUDA error.
kf_status from_launch(cudaError_t e) {
    return e == cudaSuccess ? KF_OK : e == cudaErrorInvalidValue ? KF_ERR_UNSUPPORTED : KF_ERR_CUDA;
}

cudaStream_t as_stream(kf_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

kf_status tree_impl(const void *q, const int32_t *q_start, const int32_t *parents, const void *k_cache,
                    const void *v_cache, bool kv8, const float *k_scale, const float *v_scale,
                    const int32_t *block_tables, int bt_stride, const int32_t *context_lens, int max_context_len,
                    int max_query_len, int batch, int num_q_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                    int block_size, int64_t num_blocks, float scale, void *workspace, size_t workspace_bytes,
                    void *out, kf_dtype out_dtype, float *lse_out, kf_stream_t stream) {
    if (batch < 0 || num_q_tokens < 0 || bt_stride < 1 || num_blocks < 1 || max_context_len < 0 || max_query_len < 0 ||
        num_q_heads < 1 || num_kv_heads < 1 || head_dim < 1 || block_size < 1 || !isfinite(scale) ||
        (out_dtype != KF_BF16 && out_dtype != KF_F32))
        return KF_ERR_INVALID;
    if (!q_start && num_q_tokens != batch) return KF_ERR_INVALID;
    if (batch == 0 || num_q_tokens == 0 || max_query_len == 0) return KF_OK;
    if (!q || !parents || !k_cache || !v_cache || !block_tables || !context_lens || !workspace || !out ||
        (kv8 && (!k_scale || !v_scale)))
        return KF_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(workspace, 16) ||
        !aligned(out, 16) || !aligned(q_start, 4) || !aligned(parents, 4) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4) || !aligned(lse_out, 4) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
        return KF_ERR_INVALID;
    if (!heads_ok(num_q_heads, num_kv_heads, head_dim) || !block_ok(block_size)) return KF_ERR_UNSUPPORTED;
    const int nodes = q_start ? std::min(max_query_len, num_q_tokens) : 1;  // without ranges a request has one
    // q's rows and the cache's 8-token groups fit the 31-bit TMA coordinates
    if (nodes > kMaxNodes || batch > kMaxBatch || num_q_heads > 1024 ||
        (int64_t)num_q_tokens * num_q_heads > 0x7fffffff || num_blocks * (block_size / 8) > 0x7fffffff ||
        std::min<int64_t>(max_context_len, (int64_t)bt_stride * block_size) > kMaxTokens)
        return KF_ERR_UNSUPPORTED;
    TreeParams p;
    int sms = 0;
    if (device_facts(&p.err, &sms) != cudaSuccess) return KF_ERR_CUDA;
    if (workspace_bytes <
        tree_workspace_bytes(nodes, num_q_heads, num_kv_heads, head_dim, out_dtype == KF_F32, sms))
        return KF_ERR_INVALID;
    void *fn = tensor_map_encoder();
    if (!fn) return KF_ERR_CUDA;
    p.q = static_cast<const uint16_t *>(q);
    p.q_start = q_start;
    p.parents = parents;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = kv8 ? k_scale : nullptr;
    p.v_scale = kv8 ? v_scale : nullptr;
    p.block_tables = block_tables;
    p.ctx_lens = context_lens;
    p.out = out;
    p.lse_out = lse_out;
    p.num_blocks = num_blocks;
    p.bt_stride = bt_stride;
    p.max_context_len = max_context_len;
    p.max_query_len = nodes;
    p.batch = batch;
    p.num_q_tokens = num_q_tokens;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.block_size = block_size;
    p.out_dtype = (int)out_dtype;
    p.scale_log2 = scale * kLog2e;
    return from_launch(launch_tree(p, workspace, sms, as_stream(stream), fn));
}

// Checks common to extend and release; fills a but for the arrays of one of them.
kf_status pool_args(PoolArgs *a, int32_t *pool, int64_t num_blocks, int32_t *block_tables, int bt_stride,
                    const int32_t *before, int batch, int block_size) {
    if (num_blocks < 1 || bt_stride < 1 || batch < 0 || block_size < 1) return KF_ERR_INVALID;
    if (batch == 0) return KF_OK;
    if (!pool || !block_tables || !before || !aligned(pool, 4) || !aligned(block_tables, 4) || !aligned(before, 4))
        return KF_ERR_INVALID;
    if (!block_ok(block_size) || batch > kMaxBatch || num_blocks > 0x7fffffff - KF_POOL_HEADER ||
        (int64_t)bt_stride * block_size > 0x7fffffff)
        return KF_ERR_UNSUPPORTED;
    *a = PoolArgs{};
    a->pool = pool;
    a->block_tables = block_tables;
    a->before = before;
    a->num_blocks = num_blocks;
    a->bt_stride = bt_stride;
    a->batch = batch;
    a->block_size = block_size;
    return KF_OK;
}

kf_status rows_impl(const void *k_rows, const void *v_rows, void *k_cache, void *v_cache, bool fp8,
                    const float *k_scale, const float *v_scale, const int64_t *slots, int num_rows, int num_kv_heads,
                    int head_dim, int block_size, int64_t num_blocks, kf_stream_t stream) {
    if (num_rows < 0 || num_kv_heads < 1 || head_dim < 1 || block_size < 1 || num_blocks < 1) return KF_ERR_INVALID;
    if (num_rows == 0) return KF_OK;
    if (!k_rows || !v_rows || !k_cache || !v_cache || !slots || (fp8 && (!k_scale || !v_scale))) return KF_ERR_INVALID;
    if (!aligned(k_rows, 16) || !aligned(v_rows, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(slots, 8) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
        return KF_ERR_INVALID;
    if ((head_dim != 64 && head_dim != 128) || !block_ok(block_size) || num_kv_heads > 1024 ||
        num_blocks > ((int64_t)1 << 48))
        return KF_ERR_UNSUPPORTED;
    RowsArgs a;
    int sms = 0;
    if (device_facts(&a.err, &sms) != cudaSuccess) return KF_ERR_CUDA;
    a.k_rows = static_cast<const uint16_t *>(k_rows);
    a.v_rows = static_cast<const uint16_t *>(v_rows);
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.slots = slots;
    a.num_slots = num_blocks * block_size;
    a.num_rows = num_rows;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    return from_launch(launch_append_rows(a, fp8, as_stream(stream)));
}

}  // namespace

extern "C" {

kf_status kf_prompt_attention(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                              int64_t v_stride, const int32_t *seq_start, int causal, int max_seq_len, int batch,
                              int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, float scale, void *out,
                              kf_dtype out_dtype, float *lse_out, kf_stream_t stream) {
    if (batch < 0 || num_tokens < 0 || max_seq_len < 0 || num_q_heads < 1 || num_kv_heads < 1 || head_dim < 1 ||
        !isfinite(scale) || (causal != 0 && causal != 1) || (out_dtype != KF_BF16 && out_dtype != KF_F32))
        return KF_ERR_INVALID;
    const int64_t q_row = (int64_t)num_q_heads * head_dim, kv_row = (int64_t)num_kv_heads * head_dim;
    if (q_stride < q_row || k_stride < kv_row || v_stride < kv_row) return KF_ERR_INVALID;
    if (batch == 0 || num_tokens == 0 || max_seq_len == 0) return KF_OK;
    if (!q || !k || !v || !seq_start || !out) return KF_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(seq_start, 4) ||
        !aligned(lse_out, 4) || ((q_stride | k_stride | v_stride) & 7))
        return KF_ERR_INVALID;
    if (!heads_ok(num_q_heads, num_kv_heads, head_dim)) return KF_ERR_UNSUPPORTED;
    // (a tensor map's strides stay below 2^40 bytes)
    constexpr int64_t kMaxStride = (int64_t)1 << 31;
    if (batch > kMaxBatch || num_q_heads > 1024 || (int64_t)num_tokens * num_q_heads > 0x7fffffff ||
        num_tokens > kMaxTokens || q_stride > kMaxStride || k_stride > kMaxStride || v_stride > kMaxStride)
        return KF_ERR_UNSUPPORTED;
    PromptParams p;
    int sms = 0;
    if (device_facts(&p.err, &sms) != cudaSuccess) return KF_ERR_CUDA;
    void *fn = tensor_map_encoder();
    if (!fn) return KF_ERR_CUDA;
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.seq_start = seq_start;
    p.out = out;
    p.lse_out = lse_out;
    p.causal = causal;
    p.max_seq_len = std::min(max_seq_len, num_tokens);
    p.batch = batch;
    p.num_tokens = num_tokens;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.out_dtype = (int)out_dtype;
    p.scale_log2 = scale * kLog2e;
    return from_launch(launch_prompt(p, sms, as_stream(stream), fn));
}

kf_status kf_tree_attention(const void *q, const int32_t *q_start, const int32_t *parents, const void *k_cache,
                            const void *v_cache, const int32_t *block_tables, int bt_stride,
                            const int32_t *context_lens, int max_context_len, int max_query_len, int batch,
                            int num_q_tokens, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                            int64_t num_blocks, float scale, void *workspace, size_t workspace_bytes, void *out,
                            kf_dtype out_dtype, float *lse_out, kf_stream_t stream) {
    return tree_impl(q, q_start, parents, k_cache, v_cache, false, nullptr, nullptr, block_tables, bt_stride,
                     context_lens, max_context_len, max_query_len, batch, num_q_tokens, num_q_heads, num_kv_heads,
                     head_dim, block_size, num_blocks, scale, workspace, workspace_bytes, out, out_dtype, lse_out,
                     stream);
}

kf_status kf_tree_attention_fp8(const void *q, const int32_t *q_start, const int32_t *parents, const void *k_cache,
                                const void *v_cache, const float *k_scale, const float *v_scale,
                                const int32_t *block_tables, int bt_stride, const int32_t *context_lens,
                                int max_context_len, int max_query_len, int batch, int num_q_tokens, int num_q_heads,
                                int num_kv_heads, int head_dim, int block_size, int64_t num_blocks, float scale,
                                void *workspace, size_t workspace_bytes, void *out, kf_dtype out_dtype,
                                float *lse_out, kf_stream_t stream) {
    return tree_impl(q, q_start, parents, k_cache, v_cache, true, k_scale, v_scale, block_tables, bt_stride,
                     context_lens, max_context_len, max_query_len, batch, num_q_tokens, num_q_heads, num_kv_heads,
                     head_dim, block_size, num_blocks, scale, workspace, workspace_bytes, out, out_dtype, lse_out,
                     stream);
}

size_t kf_tree_workspace_size(int max_query_len, int num_q_heads, int num_kv_heads, int head_dim) {
    if (max_query_len < 0 || num_q_heads < 1 || num_kv_heads < 1 || !heads_ok(num_q_heads, num_kv_heads, head_dim))
        return 0;
    unsigned int *err = nullptr;
    int sms = 0;
    if (device_facts(&err, &sms) != cudaSuccess) return 0;
    return tree_workspace_bytes(std::min(max_query_len, kMaxNodes), num_q_heads, num_kv_heads, head_dim, true, sms);
}

kf_status kf_accept_tree(const int32_t *parents, const int32_t *draft_tokens, const int32_t *target_tokens,
                         const int32_t *q_start, const int32_t *context_lens, int max_query_len, int batch,
                         int num_q_tokens, int32_t *path, int path_stride, int32_t *accepted, int32_t *next_tokens,
                         int32_t *context_lens_out, kf_stream_t stream) {
    if (batch < 0 || num_q_tokens < 0 || max_query_len < 0 || path_stride < max_query_len) return KF_ERR_INVALID;
    if (!q_start && num_q_tokens != batch) return KF_ERR_INVALID;
    if (batch == 0) return KF_OK;
    if (!context_lens || !accepted || !next_tokens || !context_lens_out || (max_query_len > 0 && !path) ||
        (num_q_tokens > 0 && (!parents || !draft_tokens || !target_tokens)))
        return KF_ERR_INVALID;
    for (const void *x : {static_cast<const void *>(parents), static_cast<const void *>(draft_tokens),
                          static_cast<const void *>(target_tokens), static_cast<const void *>(q_start),
                          static_cast<const void *>(context_lens), static_cast<const void *>(path),
                          static_cast<const void *>(accepted), static_cast<const void *>(next_tokens),
                          static_cast<const void *>(context_lens_out)})
        if (!aligned(x, 4)) return KF_ERR_INVALID;
    if (max_query_len > kMaxNodes || batch > kMaxBatch) return KF_ERR_UNSUPPORTED;
    AcceptArgs a;
    int sms = 0;
    if (device_facts(&a.err, &sms) != cudaSuccess) return KF_ERR_CUDA;
    a.parents = parents;
    a.draft = draft_tokens;
    a.target = target_tokens;
    a.q_start = q_start;
    a.ctx_lens = context_lens;
    a.path = path;
    a.accepted = accepted;
    a.next = next_tokens;
    a.ctx_out = context_lens_out;
    a.path_stride = path_stride;
    a.max_nodes = max_query_len;
    a.batch = batch;
    a.num_q_tokens = num_q_tokens;
    return from_launch(launch_accept(a, as_stream(stream)));
}

kf_status kf_commit_tree(void *cache_a, void *cache_b, int64_t row_bytes, const int32_t *block_tables, int bt_stride,
                         const int32_t *context_lens, const int32_t *q_start, const int32_t *path, int path_stride,
                         const int32_t *accepted, int batch, int block_size, int64_t num_blocks, kf_stream_t stream) {
    if (row_bytes < 1 || bt_stride < 1 || path_stride < 0 || batch < 0 || block_size < 1 || num_blocks < 1)
        return KF_ERR_INVALID;
    if (batch == 0 || path_stride == 0) return KF_OK;
    if (!cache_a || !block_tables || !context_lens || !path || !accepted) return KF_ERR_INVALID;
    if (!aligned(cache_a, 16) || !aligned(cache_b, 16) || !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
        !aligned(q_start, 4) || !aligned(path, 4) || !aligned(accepted, 4))
        return KF_ERR_INVALID;
    if (row_bytes % 16 != 0 || row_bytes > (1 << 20) || !block_ok(block_size) || batch > kMaxBatch ||
        num_blocks > 0x7fffffff || (int64_t)bt_stride * block_size > 0x7fffffff)
        return KF_ERR_UNSUPPORTED;
    if (cache_a == cache_b) return KF_ERR_INVALID;  // each is moved by CTAs of its own
    CommitArgs a;
    int sms = 0;
    if (device_facts(&a.err, &sms) != cudaSuccess) return KF_ERR_CUDA;
    a.cache[0] = static_cast<uint4 *>(cache_a);
    a.cache[1] = static_cast<uint4 *>(cache_b);
    a.block_tables = block_tables;
    a.ctx_lens = context_lens;
    a.q_start = q_start;
    a.path = path;
    a.accepted = accepted;
    a.num_blocks = num_blocks;
    a.row_vecs = (int)(row_bytes / 16);
    a.bt_stride = bt_stride;
    a.path_stride = path_stride;
    a.batch = batch;
    a.block_size = block_size;
    return from_launch(launch_commit(a, as_stream(stream)));
}

kf_status kf_init_block_pool(int32_t *pool, int64_t num_blocks, kf_stream_t stream) {
    if (!pool || !aligned(pool, 4) || num_blocks < 1) return KF_ERR_INVALID;
    if (num_blocks > 0x7fffffff - KF_POOL_HEADER) return KF_ERR_UNSUPPORTED;
    return from_launch(launch_pool_init(pool, num_blocks, as_stream(stream)));
}

kf_status kf_extend_block_tables(int32_t *pool, int64_t num_blocks, int32_t *block_tables, int bt_stride,
                                 const int32_t *context_lens_before, const int32_t *row_start, int batch, int num_rows,
                                 int block_size, int64_t *slots, int32_t *positions, int32_t *context_lens_after,
                                 kf_stream_t stream) {
    PoolArgs a;
    if (num_rows < 0 || (!row_start && num_rows != batch)) return KF_ERR_INVALID;
    const kf_status st = pool_args(&a, pool, num_blocks, block_tables, bt_stride, context_lens_before, batch, block_size);
    if (st != KF_OK || batch == 0) return st;
    if (!context_lens_after || (num_rows > 0 && !slots) || !aligned(row_start, 4) || !aligned(slots, 8) ||
        !aligned(positions, 4) || !aligned(context_lens_after, 4))
        return KF_ERR_INVALID;
    int sms = 0;
    if (device_facts(&a.err, &sms) != cudaSuccess) return KF_ERR_CUDA;
    a.row_start = row_start;
    a.after = context_lens_after;
    a.slots = slots;
    a.positions = positions;
    a.num_rows = num_rows;
    return from_launch(launch_extend(a, sms, as_stream(stream)));
}

kf_status kf_release_blocks(int32_t *pool, int64_t num_blocks, int32_t *block_tables, int bt_stride,
                            const int32_t *context_lens_before, const int32_t *context_lens_after, int batch,
                            int block_size, kf_stream_t stream) {
    PoolArgs a;
    const kf_status st = pool_args(&a, pool, num_blocks, block_tables, bt_stride, context_lens_before, batch, block_size);
    if (st != KF_OK || batch == 0) return st;
    if (!aligned(context_lens_after, 4)) return KF_ERR_INVALID;
    int sms = 0;
    if (device_facts(&a.err, &sms) != cudaSuccess) return KF_ERR_CUDA;
    a.target = context_lens_after;
    return from_launch(launch_release(a, sms, as_stream(stream)));
}

kf_status kf_append_rows(const void *k_rows, const void *v_rows, void *k_cache, void *v_cache, const int64_t *slots,
                         int num_rows, int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                         kf_stream_t stream) {
    return rows_impl(k_rows, v_rows, k_cache, v_cache, false, nullptr, nullptr, slots, num_rows, num_kv_heads, head_dim,
                     block_size, num_blocks, stream);
}

kf_status kf_append_rows_fp8(const void *k_rows, const void *v_rows, void *k_cache, void *v_cache,
                             const float *k_scale, const float *v_scale, const int64_t *slots, int num_rows,
                             int num_kv_heads, int head_dim, int block_size, int64_t num_blocks, kf_stream_t stream) {
    return rows_impl(k_rows, v_rows, k_cache, v_cache, true, k_scale, v_scale, slots, num_rows, num_kv_heads, head_dim,
                     block_size, num_blocks, stream);
}

}  // extern "C"
