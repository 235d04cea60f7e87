// kf_latent_api.cu -- the C entry points of latent attention and of eviction
// by accumulated attention weight, declared in include/kf.h: argument checks on
// the host, then one launch function each.
#include <math.h>

#include <algorithm>

#include "kf_device.cuh"
#include "kf_evict.cuh"
#include "kf_latent.cuh"

using namespace kf;

namespace {

constexpr float kLog2e = 1.4426950408889634f;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool block_ok(int bs) { return bs == 16 || bs == 32; }
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Token indices, and those a tile or a block's stride further on, stay in 31 bits.
constexpr int64_t kMaxTokens = (int64_t)1 << 30;

// A launch refused for its shape (a grid or tensor map that does not fit) is an
// unsupported shape; anything else is a CUDA error.
kf_status from_launch(cudaError_t e) {
    return e == cudaSuccess ? KF_OK : e == cudaErrorInvalidValue ? KF_ERR_UNSUPPORTED : KF_ERR_CUDA;
}

// Checks common to the two attention forms; fills p but for err.
kf_status latent_args(LatentParams *p, const void *q, const int32_t *q_start, const void *latent_cache,
                      const int32_t *block_tables, int bt_stride, const int32_t *context_lens, int causal,
                      int max_context_len, int max_query_len, int batch, int num_q_tokens, int num_heads,
                      int latent_dim, int rope_dim, int block_size, int64_t num_blocks, float scale,
                      const void *workspace, void *out, kf_dtype out_dtype, float *lse_out) {
    if (batch < 0 || num_q_tokens < 0 || bt_stride < 1 || num_blocks < 1 || max_context_len < 0 ||
        max_query_len < 0 || num_heads < 1 || latent_dim < 1 || rope_dim < 0 || block_size < 1 || !isfinite(scale) ||
        (causal != 0 && causal != 1) || (out_dtype != KF_BF16 && out_dtype != KF_F32))
        return KF_ERR_INVALID;
    if (!q_start && num_q_tokens != batch) return KF_ERR_INVALID;
    if (batch == 0 || num_q_tokens == 0 || max_query_len == 0) return KF_OK;
    if (!q || !latent_cache || !block_tables || !context_lens || !workspace || !out) return KF_ERR_INVALID;
    if (!aligned16(q) || !aligned16(latent_cache) || !aligned16(workspace) || !aligned16(out) ||
        !aligned4(q_start) || !aligned4(block_tables) || !aligned4(context_lens) || !aligned4(lse_out))
        return KF_ERR_INVALID;
    if ((latent_dim != 256 && latent_dim != 512) || rope_dim != kRopeDim || !block_ok(block_size))
        return KF_ERR_UNSUPPORTED;
    // one row index of q, and one 8-token group of the cache, fit the 31-bit TMA coordinates
    if (batch > 65535 || num_heads > 1024 || (int64_t)num_q_tokens * num_heads > 0x7fffffff ||
        num_blocks * (block_size / 8) > 0x7fffffff || (int64_t)bt_stride * block_size > 0x7fffffff ||
        std::min<int64_t>(max_context_len, (int64_t)bt_stride * block_size) > kMaxTokens)
        return KF_ERR_UNSUPPORTED;
    p->q = static_cast<const uint16_t *>(q);
    p->q_start = q_start;
    p->cache = static_cast<const uint16_t *>(latent_cache);
    p->block_tables = block_tables;
    p->ctx_lens = context_lens;
    p->out = out;
    p->lse_out = lse_out;
    p->num_blocks = num_blocks;
    p->bt_stride = bt_stride;
    p->max_context_len = max_context_len;
    // (what follows is sized by it; without ranges every request has one query)
    p->max_query_len = q_start ? std::min(max_query_len, num_q_tokens) : 1;
    p->batch = batch;
    p->num_q_tokens = num_q_tokens;
    p->num_heads = num_heads;
    p->latent_dim = latent_dim;
    p->block_size = block_size;
    p->causal = causal;
    p->out_dtype = (int)out_dtype;
    p->scale_log2 = scale * kLog2e;
    return KF_OK;
}

kf_status accumulate_impl(const void *q, const int32_t *q_start, const void *k_cache, const float *k_scale, bool kv8,
                          const int32_t *block_tables, int bt_stride, const int32_t *context_lens, int causal,
                          int max_context_len, int max_query_len, int batch, int num_q_tokens, int num_q_heads,
                          int num_kv_heads, int head_dim, int block_size, int64_t num_blocks, float scale,
                          const float *lse, const float *scores_in, float *scores_out, int64_t score_stride,
                          kf_stream_t stream) {
    if (batch < 0 || num_q_tokens < 0 || bt_stride < 1 || num_blocks < 1 || max_context_len < 0 ||
        max_query_len < 0 || num_q_heads < 1 || num_kv_heads < 1 || head_dim < 1 || block_size < 1 ||
        !isfinite(scale) || (causal != 0 && causal != 1) || score_stride < max_context_len)
        return KF_ERR_INVALID;
    if (!q_start && num_q_tokens != batch) return KF_ERR_INVALID;
    if (batch == 0 || max_context_len == 0) return KF_OK;
    if (!k_cache || !block_tables || !context_lens || !scores_out || (num_q_tokens > 0 && (!q || !lse)) ||
        (kv8 && !k_scale))
        return KF_ERR_INVALID;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned4(lse) || !aligned4(scores_in) || !aligned4(scores_out) ||
        !aligned4(q_start) || !aligned4(block_tables) || !aligned4(context_lens) || !aligned4(k_scale))
        return KF_ERR_INVALID;
    const int group = num_q_heads / num_kv_heads;
    if ((head_dim != 64 && head_dim != 128) || !block_ok(block_size) || num_q_heads % num_kv_heads != 0 ||
        (group != 1 && group != 2 && group != 4 && group != 8))
        return KF_ERR_UNSUPPORTED;
    // q's rows and the cache's 8-token groups fit 31 bits (TMA coordinates, column counts)
    if (batch > 65535 || (int64_t)num_q_tokens * num_q_heads > 0x7fffffff ||
        num_blocks * (block_size / 8) > 0x7fffffff || max_context_len > kMaxTokens)
        return KF_ERR_UNSUPPORTED;
    AccumulateParams p;
    int sms = 0;
    if (device_facts(&p.err, &sms) != cudaSuccess) return KF_ERR_CUDA;
    p.q = static_cast<const uint16_t *>(q);
    p.q_start = q_start;
    p.k_cache = k_cache;
    p.k_scale = kv8 ? k_scale : nullptr;
    p.block_tables = block_tables;
    p.ctx_lens = context_lens;
    p.lse = lse;
    p.scores_in = scores_in;
    p.scores_out = scores_out;
    p.num_blocks = num_blocks;
    p.score_stride = score_stride;
    p.bt_stride = bt_stride;
    p.max_context_len = max_context_len;
    // (without ranges every request has one query)
    p.max_query_len = q_start ? std::min(max_query_len, num_q_tokens) : std::min(max_query_len, 1);
    p.batch = batch;
    p.num_q_tokens = num_q_tokens;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.block_size = block_size;
    p.causal = causal;
    p.scale_log2 = scale * kLog2e;
    void *fn = tensor_map_encoder();
    if (!fn) return KF_ERR_CUDA;
    return from_launch(launch_accumulate(p, sms, reinterpret_cast<cudaStream_t>(stream), fn));
}

// Rows that can move: into slots below `keep`, from indices at or above it.
int max_moves(int max_context_len, int keep) { return std::max(0, std::min(keep, max_context_len - keep)); }

}  // namespace

extern "C" {

kf_status kf_append_latent(const void *latent_new, const int32_t *row_start, void *latent_cache,
                           const int32_t *block_tables, int bt_stride, const int32_t *context_lens_before, int batch,
                           int num_rows, int latent_dim, int rope_dim, int block_size, int64_t num_blocks,
                           kf_stream_t stream) {
    if (batch < 0 || num_rows < 0 || latent_dim < 1 || rope_dim < 0 || bt_stride < 1 || num_blocks < 1 ||
        block_size < 1)
        return KF_ERR_INVALID;
    if (!row_start && num_rows != batch) return KF_ERR_INVALID;
    if (batch == 0 || num_rows == 0) return KF_OK;
    if (!latent_new || !latent_cache || !block_tables || !context_lens_before) return KF_ERR_INVALID;
    if (!aligned16(latent_new) || !aligned16(latent_cache) || !aligned4(row_start) || !aligned4(block_tables) ||
        !aligned4(context_lens_before))
        return KF_ERR_INVALID;
    if ((latent_dim != 256 && latent_dim != 512) || rope_dim != kRopeDim || !block_ok(block_size))
        return KF_ERR_UNSUPPORTED;
    unsigned int *err = nullptr;
    int sms = 0;
    if (device_facts(&err, &sms) != cudaSuccess) return KF_ERR_CUDA;
    return from_launch(launch_append_latent(
        static_cast<const uint16_t *>(latent_new), row_start, static_cast<uint16_t *>(latent_cache), block_tables,
        bt_stride, context_lens_before, batch, num_rows, latent_dim + rope_dim, block_size, num_blocks, err,
        reinterpret_cast<cudaStream_t>(stream)));
}

size_t kf_latent_workspace_size(int batch, int max_query_len, int num_heads, int latent_dim) {
    if (batch < 0 || max_query_len < 0 || num_heads < 1 || (latent_dim != 256 && latent_dim != 512)) return 0;
    unsigned int *err = nullptr;
    int sms = 0;
    if (device_facts(&err, &sms) != cudaSuccess) return 0;
    return latent_workspace_bytes(max_query_len, num_heads, latent_dim, sms);
}

kf_status kf_latent_attention(const void *q, const int32_t *q_start, const void *latent_cache,
                              const int32_t *block_tables, int bt_stride, const int32_t *context_lens, int causal,
                              int max_context_len, int max_query_len, int batch, int num_q_tokens, int num_heads,
                              int latent_dim, int rope_dim, int block_size, int64_t num_blocks, float scale,
                              void *workspace, size_t workspace_bytes, void *out, kf_dtype out_dtype, float *lse_out,
                              kf_stream_t stream) {
    LatentParams p;
    const kf_status st = latent_args(&p, q, q_start, latent_cache, block_tables, bt_stride, context_lens, causal,
                                     max_context_len, max_query_len, batch, num_q_tokens, num_heads, latent_dim,
                                     rope_dim, block_size, num_blocks, scale, workspace, out, out_dtype, lse_out);
    if (st != KF_OK || batch == 0 || num_q_tokens == 0 || max_query_len == 0) return st;
    int sms = 0;
    if (device_facts(&p.err, &sms) != cudaSuccess) return KF_ERR_CUDA;
    if (workspace_bytes < latent_workspace_bytes(max_query_len, num_heads, latent_dim, sms))
        return KF_ERR_INVALID;
    void *fn = tensor_map_encoder();
    if (!fn) return KF_ERR_CUDA;
    return from_launch(launch_latent(p, workspace, sms, reinterpret_cast<cudaStream_t>(stream), fn));
}

size_t kf_latent_expanded_workspace_size(int batch, int num_q_tokens, int max_context_len, int num_heads, int nope_dim,
                                         int v_dim) {
    if (batch < 0 || num_q_tokens < 0 || max_context_len < 0 || num_heads < 1 || nope_dim < 1 || v_dim < 1) return 0;
    return latent_expanded_workspace_bytes(batch, max_context_len, num_heads, nope_dim, v_dim);
}

kf_status kf_latent_attention_expanded(const void *q, const int32_t *q_start, const void *latent_cache,
                                       const void *w_uk, const void *w_uv, const int32_t *block_tables, int bt_stride,
                                       const int32_t *context_lens, int causal, int max_context_len, int max_query_len,
                                       int batch, int num_q_tokens, int num_heads, int latent_dim, int rope_dim,
                                       int nope_dim, int v_dim, int block_size, int64_t num_blocks, float scale,
                                       void *workspace, size_t workspace_bytes, void *out, kf_dtype out_dtype,
                                       float *lse_out, kf_stream_t stream) {
    if (nope_dim < 1 || v_dim < 1) return KF_ERR_INVALID;
    LatentParams p;
    const kf_status st = latent_args(&p, q, q_start, latent_cache, block_tables, bt_stride, context_lens, causal,
                                     max_context_len, max_query_len, batch, num_q_tokens, num_heads, latent_dim,
                                     rope_dim, block_size, num_blocks, scale, workspace, out, out_dtype, lse_out);
    if (st != KF_OK || batch == 0 || num_q_tokens == 0 || max_query_len == 0) return st;
    if (!w_uk || !w_uv || !aligned16(w_uk) || !aligned16(w_uv)) return KF_ERR_INVALID;
    if (!((nope_dim == 64 && v_dim == 64) || (nope_dim == 128 && v_dim == 128))) return KF_ERR_UNSUPPORTED;
    // rows of the expanded keys and values fit the 31-bit TMA coordinates
    if (((int64_t)max_context_len + 127) / 128 * 128 * batch * num_heads > 0x7fffffff) return KF_ERR_UNSUPPORTED;
    if (workspace_bytes < latent_expanded_workspace_bytes(batch, max_context_len, num_heads, nope_dim, v_dim))
        return KF_ERR_INVALID;
    int sms = 0;
    if (device_facts(&p.err, &sms) != cudaSuccess) return KF_ERR_CUDA;
    void *fn = tensor_map_encoder();
    if (!fn) return KF_ERR_CUDA;
    LatentWeights w{static_cast<const uint16_t *>(w_uk), static_cast<const uint16_t *>(w_uv), nope_dim, v_dim};
    return from_launch(launch_latent_expanded(p, w, workspace, sms, reinterpret_cast<cudaStream_t>(stream), fn));
}

kf_status kf_accumulate_attention(const void *q, const int32_t *q_start, const void *k_cache,
                                  const int32_t *block_tables, int bt_stride, const int32_t *context_lens, int causal,
                                  int max_context_len, int max_query_len, int batch, int num_q_tokens, int num_q_heads,
                                  int num_kv_heads, int head_dim, int block_size, int64_t num_blocks, float scale,
                                  const float *lse, const float *scores_in, float *scores_out, int64_t score_stride,
                                  kf_stream_t stream) {
    return accumulate_impl(q, q_start, k_cache, nullptr, false, block_tables, bt_stride, context_lens, causal,
                           max_context_len, max_query_len, batch, num_q_tokens, num_q_heads, num_kv_heads, head_dim,
                           block_size, num_blocks, scale, lse, scores_in, scores_out, score_stride, stream);
}

kf_status kf_accumulate_attention_fp8(const void *q, const int32_t *q_start, const void *k_cache,
                                      const float *k_scale, const int32_t *block_tables, int bt_stride,
                                      const int32_t *context_lens, int causal, int max_context_len, int max_query_len,
                                      int batch, int num_q_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                      int block_size, int64_t num_blocks, float scale, const float *lse,
                                      const float *scores_in, float *scores_out, int64_t score_stride,
                                      kf_stream_t stream) {
    return accumulate_impl(q, q_start, k_cache, k_scale, true, block_tables, bt_stride, context_lens, causal,
                           max_context_len, max_query_len, batch, num_q_tokens, num_q_heads, num_kv_heads, head_dim,
                           block_size, num_blocks, scale, lse, scores_in, scores_out, score_stride, stream);
}

size_t kf_evict_workspace_size(int batch, int max_context_len, int keep) {
    if (batch < 0 || max_context_len < 0 || keep < 1) return 0;
    return align256((size_t)batch * 4) + 2 * align256((size_t)batch * max_moves(max_context_len, keep) * 4);
}

kf_status kf_evict_tokens(void *cache_a, void *cache_b, int64_t row_bytes, const int32_t *block_tables, int bt_stride,
                          const int32_t *context_lens, int max_context_len, int batch, int block_size,
                          int64_t num_blocks, const float *scores, float *scores_out, int64_t score_stride,
                          const int32_t *positions, int32_t *positions_out, const int32_t *seq_lens, int keep, int sink,
                          int recent, int32_t *context_lens_out, void *workspace, size_t workspace_bytes,
                          kf_stream_t stream) {
    if (batch < 0 || bt_stride < 1 || num_blocks < 1 || max_context_len < 0 || block_size < 1 || row_bytes < 1 ||
        keep < 1 || sink < 0 || recent < 0 || (int64_t)sink + recent > keep || score_stride < max_context_len)
        return KF_ERR_INVALID;
    if (batch == 0) return KF_OK;
    if (!cache_a || !block_tables || !context_lens || !scores || !scores_out || !context_lens_out || !workspace)
        return KF_ERR_INVALID;
    if ((positions != nullptr) != (positions_out != nullptr) || (positions != nullptr) != (seq_lens != nullptr))
        return KF_ERR_INVALID;
    if (!aligned16(cache_a) || !aligned16(cache_b) || !aligned16(workspace) || !aligned4(scores) ||
        !aligned4(scores_out) || !aligned4(positions) || !aligned4(positions_out) || !aligned4(seq_lens) ||
        !aligned4(context_lens) || !aligned4(context_lens_out) || !aligned4(block_tables))
        return KF_ERR_INVALID;
    if (row_bytes % 16 != 0 || row_bytes > (1 << 20) || !block_ok(block_size) || batch > 65535 ||
        max_context_len > kMaxTokens)
        return KF_ERR_UNSUPPORTED;
    if (workspace_bytes < kf_evict_workspace_size(batch, max_context_len, keep)) return KF_ERR_INVALID;
    EvictParams p;
    int sms = 0;
    if (device_facts(&p.err, &sms) != cudaSuccess) return KF_ERR_CUDA;
    p.cache_a = static_cast<uint4 *>(cache_a);
    p.cache_b = static_cast<uint4 *>(cache_b);
    p.block_tables = block_tables;
    p.ctx_lens = context_lens;
    p.scores = scores;
    p.scores_out = scores_out;
    p.positions = positions;
    p.positions_out = positions_out;
    p.seq_lens = seq_lens;
    p.ctx_out = context_lens_out;
    p.max_moves = max_moves(max_context_len, keep);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.counts = reinterpret_cast<int *>(ws);
    p.dst = reinterpret_cast<int *>(ws + align256((size_t)batch * 4));
    p.src = reinterpret_cast<int *>(reinterpret_cast<uint8_t *>(p.dst) + align256((size_t)batch * p.max_moves * 4));
    p.num_blocks = num_blocks;
    p.score_stride = score_stride;
    p.row_vecs = (int)(row_bytes / 16);
    p.bt_stride = bt_stride;
    p.max_context_len = max_context_len;
    p.batch = batch;
    p.block_size = block_size;
    p.keep = keep;
    p.sink = sink;
    p.recent = recent;
    return from_launch(launch_evict(p, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
