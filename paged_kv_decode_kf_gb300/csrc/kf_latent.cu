// kf_latent.cu -- latent attention, absorbed and expanded forms, CUDA cores.
//
// One CTA owns 16 query rows of one request and walks its tokens 32 at a time:
// keys as fp32 in shared memory, 16 x 32 scores, the online softmax, then each
// thread adds the weighted values of its columns. Rows of the absorbed form are
// (query token, head) pairs, which share every key; rows of the expanded form
// are the query tokens of one head.
#include "kf_latent.cuh"

#include <cuda_fp16.h>

namespace kf {
namespace {

constexpr int kRows = 16, kTok = 32, kThreads = 256;

__host__ __device__ inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Expanded keys (fp32) and values (fp16) in the workspace: [H][batch * cap][width].
struct ExpandedKV {
    const float *k;
    const __half *v;
    int64_t cap;  // token rows a request
    int nope, v_dim;
};

template <bool EXPANDED>
__global__ void __launch_bounds__(kThreads)
latent_simple_kernel(const LatentParams p, const ExpandedKV kv) {
    extern __shared__ float sm[];
    const int R = p.latent_dim;
    const int KD = (EXPANDED ? kv.nope : R) + kRopeDim, VD = EXPANDED ? kv.v_dim : R;
    const int KS = KD + 1;
    float *sq = sm, *sk = sq + kRows * KS, *sv = sk + kTok * KS, *sp = sv + (EXPANDED ? kTok * VD : 0);
    float *s_m = sp + kRows * kTok, *s_l = s_m + kRows, *s_a = s_l + kRows;
    const int b = blockIdx.y, h = EXPANDED ? blockIdx.z : 0;
    const int tid = threadIdx.x;
    const LatentRequest rq = latent_request(p, b, blockIdx.x == 0 && blockIdx.z == 0 && tid == 0);
    if (rq.q0 < 0) return;
    const int64_t nrows = (rq.C < p.max_query_len ? rq.C : p.max_query_len) * (EXPANDED ? 1 : p.num_heads);
    const int64_t row0 = (int64_t)blockIdx.x * kRows;
    if (row0 >= nrows) return;
    const int64_t L = rq.L < p.max_context_len ? rq.L : p.max_context_len;
    const int64_t shift = rq.L - rq.C;  // query j sees tokens [0, shift + j]
    // the row's place in q, out and lse, as a (token, head) index
    auto place = [&](int64_t row) {
        return EXPANDED ? (rq.q0 + row) * p.num_heads + h : rq.q0 * p.num_heads + row;
    };
    auto limit = [&](int64_t row) {
        const int64_t j = EXPANDED ? row : row / p.num_heads;
        const int64_t n = p.causal ? shift + j + 1 : L;
        return n < L ? n : L;
    };
    for (int i = tid; i < kRows * KD; i += kThreads) {
        const int r = i / KD, d = i % KD;
        sq[r * KS + d] = row0 + r < nrows ? bf16_lo(p.q[place(row0 + r) * KD + d]) : 0.f;
    }
    if (tid < kRows) {
        s_m[tid] = -INFINITY;
        s_l[tid] = 0.f;
    }
    // this thread's output columns: d = tid, tid + 256 of every row
    float acc[2][kRows];
    for (int r = 0; r < kRows; ++r) acc[0][r] = acc[1][r] = 0.f;
    const int64_t last = row0 + kRows < nrows ? row0 + kRows - 1 : nrows - 1;
    const int64_t t_end = limit(last);
    for (int64_t t0 = 0; t0 < t_end; t0 += kTok) {
        __syncthreads();
        for (int i = tid; i < kTok * KD; i += kThreads) {
            const int t = i / KD, d = i % KD;
            float x = 0.f;
            if (t0 + t < t_end) {
                int64_t phys = p.block_tables[(int64_t)b * p.bt_stride + (t0 + t) / p.block_size];
                if (phys < 0 || phys >= p.num_blocks) {
                    raise_error(p.err, KF_DEVERR_BLOCK_ID);
                    phys = 0;
                }
                const int64_t row = (phys * p.block_size + (t0 + t) % p.block_size) * (R + kRopeDim);
                if (EXPANDED)
                    x = d < kv.nope ? kv.k[(((int64_t)h * p.batch + b) * kv.cap + t0 + t) * kv.nope + d]
                                    : bf16_lo(p.cache[row + R + d - kv.nope]);
                else
                    x = bf16_lo(p.cache[row + d]);
            }
            sk[t * KS + d] = x;
        }
        if (EXPANDED)
            for (int i = tid; i < kTok * VD; i += kThreads) {
                const int t = i / VD, d = i % VD;
                sv[i] = t0 + t < t_end
                            ? __half2float(kv.v[(((int64_t)h * p.batch + b) * kv.cap + t0 + t) * VD + d])
                            : 0.f;
            }
        __syncthreads();
        for (int i = tid; i < kRows * kTok; i += kThreads) {
            const int r = i / kTok, t = i % kTok;
            float s = 0.f;
            for (int d = 0; d < KD; ++d) s = fmaf(sq[r * KS + d], sk[t * KS + d], s);
            sp[i] = row0 + r < nrows && t0 + t < limit(row0 + r) ? s * p.scale_log2 : -INFINITY;
        }
        __syncthreads();
        if (tid < kRows) {
            float m = s_m[tid];
            for (int t = 0; t < kTok; ++t) m = fmaxf(m, sp[tid * kTok + t]);
            const float mu = m == -INFINITY ? 0.f : m;
            float l = 0.f;
            for (int t = 0; t < kTok; ++t) {
                const float e = exp2f(sp[tid * kTok + t] - mu);
                sp[tid * kTok + t] = e;
                l += e;
            }
            const float a = exp2f(s_m[tid] - mu);
            s_a[tid] = a;
            s_l[tid] = s_l[tid] * a + l;
            s_m[tid] = m;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int d = tid + c * kThreads;
            if (d >= VD) break;
            for (int r = 0; r < kRows; ++r) acc[c][r] *= s_a[r];
            for (int t = 0; t < kTok; ++t) {
                const float x = EXPANDED ? sv[t * VD + d] : sk[t * KS + d];
                for (int r = 0; r < kRows; ++r) acc[c][r] = fmaf(sp[r * kTok + t], x, acc[c][r]);
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int d = tid + c * kThreads;
        if (d >= VD) break;
        for (int r = 0; r < kRows && row0 + r < nrows; ++r) {
            const float o = s_l[r] > 0.f ? acc[c][r] / s_l[r] : 0.f;
            const int64_t at = place(row0 + r) * VD + d;
            if (p.out_dtype == KF_F32) static_cast<float *>(p.out)[at] = o;
            else static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16(o);
        }
    }
    if (p.lse_out && tid < kRows && row0 + tid < nrows)
        p.lse_out[place(row0 + tid)] =
            s_l[tid] > 0.f ? (s_m[tid] + log2f(s_l[tid])) * 0.6931471805599453f : -INFINITY;
}

__device__ __forceinline__ void put(const LatentParams &p, float *at, float x) { *at = x; }
__device__ __forceinline__ void put(const LatentParams &p, __half *at, float x) {
    if (!(fabsf(x) <= 65504.f)) raise_error(p.err, KF_DEVERR_RANGE);
    *at = __float2half(x);
}

// K_nope or V of every token: out[h][b * cap + t][i] = <w[h][i], c_t>.
template <typename T>
__global__ void __launch_bounds__(256)
expand_simple_kernel(const LatentParams p, const uint16_t *__restrict__ w, T *__restrict__ out, int width,
                     int64_t cap) {
    extern __shared__ float sc[];  // 16 latent rows
    const int R = p.latent_dim, b = blockIdx.y, h = blockIdx.z;
    const int64_t t0 = (int64_t)blockIdx.x * 16;
    const LatentRequest rq = latent_request(p, b, false);
    const int64_t L = rq.L < p.max_context_len ? rq.L : p.max_context_len;
    if (rq.q0 < 0 || t0 >= L) return;
    for (int i = threadIdx.x; i < 16 * R; i += 256) {
        const int t = i / R, d = i % R;
        float x = 0.f;
        if (t0 + t < L) {
            int64_t phys = p.block_tables[(int64_t)b * p.bt_stride + (t0 + t) / p.block_size];
            if (phys < 0 || phys >= p.num_blocks) {
                raise_error(p.err, KF_DEVERR_BLOCK_ID);
                phys = 0;
            }
            x = bf16_lo(p.cache[(phys * p.block_size + (t0 + t) % p.block_size) * (R + kRopeDim) + d]);
        }
        sc[i] = x;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * width; i += 256) {
        const int t = i / width, n = i % width;
        if (t0 + t >= L) continue;
        const uint16_t *row = w + ((int64_t)h * width + n) * R;
        float s = 0.f;
        for (int d = 0; d < R; ++d) s = fmaf(sc[t * R + d], bf16_lo(row[d]), s);
        put(p, out + (((int64_t)h * p.batch + b) * cap + t0 + t) * width + n, s);
    }
}

}  // namespace

size_t latent_expanded_workspace_bytes(int batch, int num_q_tokens, int max_context_len, int num_heads, int nope,
                                       int v) {
    const size_t cap = ((size_t)max_context_len + 127) / 128 * 128;
    return align256(batch * cap * num_heads * nope * 4) + align256(batch * cap * num_heads * v * 2);
}

cudaError_t launch_latent_expanded(const LatentParams &p, const LatentWeights &w, void *workspace, int sm_count,
                                   cudaStream_t stream, void *encode_fn) {
    const int64_t cap = ((int64_t)p.max_context_len + 127) / 128 * 128;
    float *k = static_cast<float *>(workspace);
    __half *v = reinterpret_cast<__half *>(static_cast<uint8_t *>(workspace) +
                                           align256((size_t)p.batch * cap * p.num_heads * w.nope * 4));
    const dim3 grid((unsigned)((p.max_context_len + 15) / 16), p.batch, p.num_heads);
    if (p.max_context_len > 0) {
        expand_simple_kernel<<<grid, 256, 16 * p.latent_dim * 4, stream>>>(p, w.w_uk, k, w.nope, cap);
        expand_simple_kernel<<<grid, 256, 16 * p.latent_dim * 4, stream>>>(p, w.w_uv, v, w.v, cap);
    }
    const int KS = w.nope + kRopeDim + 1;
    const size_t smem = (size_t)(kRows * KS + kTok * KS + kTok * w.v + kRows * kTok + 3 * kRows) * 4;
    cudaError_t e = cudaFuncSetAttribute(latent_simple_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    latent_simple_kernel<true>
        <<<dim3((unsigned)((p.max_query_len + kRows - 1) / kRows), p.batch, p.num_heads), kThreads, smem, stream>>>(
            p, ExpandedKV{k, v, cap, w.nope, w.v});
    return cudaGetLastError();
}

}  // namespace kf
