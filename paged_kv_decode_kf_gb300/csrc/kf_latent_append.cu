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

__global__ void __launch_bounds__(128)
append_latent_kernel(const uint4 *__restrict__ rows, const int32_t *__restrict__ row_start, uint4 *__restrict__ cache,
                     const int32_t *__restrict__ block_tables, int bt_stride, const int32_t *__restrict__ ctx_before,
                     int batch, int num_rows, int row_vecs, int block_size, int64_t num_blocks, unsigned int *err) {
    // (an attention kernel that follows sets itself up meanwhile, and waits for this one
    // before it reads anything)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= num_rows) return;
    // the request that owns the row: the last b with row_start[b] <= row
    int b = (int)row;
    int64_t j = 0;
    if (row_start) {
        int lo = 0, hi = batch;  // row_start[lo] <= row < row_start[hi] where the starts ascend
        if (row < row_start[0] || row >= row_start[batch]) return;  // owned by no request
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (row_start[mid] <= row) lo = mid;
            else hi = mid;
        }
        b = lo;
        j = row - row_start[b];
        if (j < 0 || row >= row_start[b + 1]) {  // starts that do not ascend
            if (lane == 0) raise_error(err, KF_DEVERR_CONTEXT_LEN);
            return;
        }
    }
    const int64_t first = ctx_before[b];
    const int64_t pos = first + j;
    if (first < 0 || pos >= (int64_t)bt_stride * block_size) {
        if (lane == 0) raise_error(err, KF_DEVERR_APPEND_POS);
        return;
    }
    const int64_t phys = block_tables[(int64_t)b * bt_stride + pos / block_size];
    if (phys < 0 || phys >= num_blocks) {
        if (lane == 0) raise_error(err, KF_DEVERR_BLOCK_ID);
        return;
    }
    const int64_t dst = (phys * block_size + pos % block_size) * row_vecs;
    for (int i = lane; i < row_vecs; i += 32) cache[dst + i] = rows[row * row_vecs + i];
}

}  // namespace

cudaError_t launch_append_latent(const uint16_t *rows, const int32_t *row_start, uint16_t *cache,
                                 const int32_t *block_tables, int bt_stride, const int32_t *ctx_before, int batch,
                                 int num_rows, int row_dim, int block_size, int64_t num_blocks, unsigned int *err,
                                 cudaStream_t stream) {
    append_latent_kernel<<<(num_rows + 3) / 4, 128, 0, stream>>>(
        reinterpret_cast<const uint4 *>(rows), row_start, reinterpret_cast<uint4 *>(cache), block_tables, bt_stride,
        ctx_before, batch, num_rows, row_dim / 8, block_size, num_blocks, err);
    return cudaGetLastError();
}

}  // namespace kf
