// kf_accumulate.cu -- attention weight each cached token receives.
//
// scores_out[b, t] = scores_in[b, t] + sum over the request's queries j that
// see t and over all query heads h of exp(scale <q_jh, k_{h/G, t}> - lse_jh).
// Every sum runs in one thread in one order, so a call's result does not
// depend on scheduling. One warp a token; the lanes split the head dimension.
#include "kf_evict.cuh"

#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace kf {
namespace {

template <int D, bool KV8>
__global__ void __launch_bounds__(128)
accumulate_simple_kernel(const AccumulateParams p) {
    constexpr int E = D / 32;
    const int b = blockIdx.y, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const bool report = t == 0 && lane == 0;
    int64_t q0 = b, q1 = b + 1;
    if (p.q_start) {
        q0 = p.q_start[b];
        q1 = p.q_start[b + 1];
    }
    if (q0 < 0 || q1 < q0 || q1 > p.num_q_tokens) {
        if (report) raise_error(p.err, KF_DEVERR_CONTEXT_LEN);
        return;
    }
    int64_t C = q1 - q0, L = p.ctx_lens[b];
    const int64_t cap = (int64_t)p.bt_stride * p.block_size;
    if (L < 0 || L > cap) {
        if (report) raise_error(p.err, KF_DEVERR_CONTEXT_LEN);
        L = L < 0 ? 0 : (L > cap ? cap : L);
    }
    if ((L > p.max_context_len || C > p.max_query_len) && report) raise_error(p.err, KF_DEVERR_MAX_CONTEXT);
    const int64_t end = L < p.max_context_len ? L : p.max_context_len;
    if (t >= end) return;
    int64_t phys = p.block_tables[(int64_t)b * p.bt_stride + t / p.block_size];
    if (phys < 0 || phys >= p.num_blocks) {
        if (lane == 0) raise_error(p.err, KF_DEVERR_BLOCK_ID);
        phys = 0;
    }
    const int64_t row = (phys * p.block_size + t % p.block_size) * p.num_kv_heads;
    const int G = p.num_q_heads / p.num_kv_heads;
    const int64_t j0 = p.causal && t > L - C ? t - (L - C) : 0;  // the first query that sees t
    const int64_t jn = C < p.max_query_len ? C : p.max_query_len;
    float sum = 0.f;
    for (int h = 0; h < p.num_kv_heads; ++h) {
        float k[E];
        for (int e = 0; e < E; ++e) {
            const int64_t at = (row + h) * D + e * 32 + lane;
            if (KV8) {
                const __nv_fp8_storage_t c = static_cast<const uint8_t *>(p.k_cache)[at];
                k[e] = __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3))) * p.k_scale[h];
            } else {
                k[e] = bf16_lo(static_cast<const uint16_t *>(p.k_cache)[at]);
            }
        }
        for (int64_t j = j0; j < jn; ++j)
            for (int g = 0; g < G; ++g) {
                const int64_t qr = (q0 + j) * p.num_q_heads + h * G + g;
                float s = 0.f;
                for (int e = 0; e < E; ++e) s = fmaf(k[e], bf16_lo(p.q[qr * D + e * 32 + lane]), s);
                for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                const float l = p.lse[qr];
                if (l != -INFINITY) sum += exp2f(s * p.scale_log2 - l * 1.4426950408889634f);
            }
    }
    if (lane == 0) {
        const int64_t at = b * p.score_stride + t;
        p.scores_out[at] = (p.scores_in ? p.scores_in[at] : 0.f) + sum;
    }
}

}  // namespace

cudaError_t launch_accumulate(const AccumulateParams &p, int sm_count, cudaStream_t stream) {
    const dim3 grid((p.max_context_len + 3) / 4, p.batch);
    if (p.k_scale) {
        if (p.head_dim == 128) accumulate_simple_kernel<128, true><<<grid, 128, 0, stream>>>(p);
        else accumulate_simple_kernel<64, true><<<grid, 128, 0, stream>>>(p);
    } else {
        if (p.head_dim == 128) accumulate_simple_kernel<128, false><<<grid, 128, 0, stream>>>(p);
        else accumulate_simple_kernel<64, false><<<grid, 128, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace kf
