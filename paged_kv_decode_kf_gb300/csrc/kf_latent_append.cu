// kf_latent_append.cu -- new latent rows into the paged latent cache.
//
// Request b's rows go to positions ctx_before[b], ctx_before[b] + 1, ... in
// order: block block_tables[b][p / bs], slot p % bs. A row is row_dim bf16
// values, copied bit for bit as 16-byte vectors.
//
// One warp a row, four rows a CTA: a decode step writes one row of 640 or 1152
// bytes a request (the launch is the cost), a prompt's rows are a plain copy.
#include "kf_latent.cuh"

namespace kf {
namespace {

struct AppendArgs {
    const uint4 *rows;
    const int32_t *row_start;   // [batch + 1] or null
    uint4 *cache;
    const int32_t *block_tables, *ctx_before;
    unsigned int *err;
    int64_t num_blocks;
    int bt_stride, batch, num_rows, row_vecs, block_size;
};

__device__ __forceinline__ void append_row(const AppendArgs &a, int64_t row) {
    const int lane = threadIdx.x & 31;
    if (row >= a.num_rows) return;
    // the request that owns the row, row_start[b] <= row < row_start[b + 1] (one of them
    // where ranges overlap)
    int b = (int)row;
    int64_t j = 0;
    if (a.row_start) {
        int lo = 0, hi = a.batch;
        if (row < a.row_start[0] || row >= a.row_start[a.batch]) return;  // owned by no request
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.row_start[mid] <= row) lo = mid;
            else hi = mid;
        }
        b = lo;
        j = row - a.row_start[b];
    }
    const int64_t first = a.ctx_before[b];
    const int64_t pos = first + j;
    if (first < 0 || pos >= (int64_t)a.bt_stride * a.block_size) {
        if (lane == 0) raise_error(a.err, KF_DEVERR_APPEND_POS);
        return;
    }
    const int64_t phys = a.block_tables[(int64_t)b * a.bt_stride + pos / a.block_size];
    if (phys < 0 || phys >= a.num_blocks) {
        if (lane == 0) raise_error(a.err, KF_DEVERR_BLOCK_ID);
        return;
    }
    const int64_t dst = (phys * a.block_size + pos % a.block_size) * a.row_vecs;
    for (int i = lane; i < a.row_vecs; i += 32) a.cache[dst + i] = __ldg(a.rows + row * a.row_vecs + i);
}

__global__ void __launch_bounds__(128)
append_latent_kernel(const AppendArgs a) {
    // (an attention kernel that follows sets itself up meanwhile, and waits for this one
    // before it reads anything)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    append_row(a, (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5));
    // ranges in order and inside the rows: a few starts a thread of the whole grid
    if (a.row_start) {
        for (int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x; i <= a.batch; i += (int64_t)gridDim.x * 128) {
            const int s = a.row_start[i];
            if (s < 0 || s > a.num_rows || (i < a.batch && a.row_start[i + 1] < s))
                raise_error(a.err, KF_DEVERR_CONTEXT_LEN);
        }
    }
}

}  // namespace

cudaError_t launch_append_latent(const uint16_t *rows, const int32_t *row_start, uint16_t *cache,
                                 const int32_t *block_tables, int bt_stride, const int32_t *ctx_before, int batch,
                                 int num_rows, int row_dim, int block_size, int64_t num_blocks, unsigned int *err,
                                 cudaStream_t stream) {
    const AppendArgs a{reinterpret_cast<const uint4 *>(rows), row_start, reinterpret_cast<uint4 *>(cache),
                       block_tables, ctx_before, err, num_blocks, bt_stride, batch, num_rows, row_dim / 8, block_size};
    append_latent_kernel<<<(unsigned)(((int64_t)num_rows + 3) / 4), 128, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kf
