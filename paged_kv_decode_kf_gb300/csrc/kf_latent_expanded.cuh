// kf_latent_expanded.cuh -- what the expanded form's two kernels share: the
// workspace's layout.
//
//   K  bf16 [H][batch * cap][2 * nope]: each key as a pair hi = bf16(k), lo =
//      bf16(k - hi): 16 bits of significand together
//   V  fp16 [H][batch * cap][v]
// cap = the token bound rounded up to 128; request b's token t is row b * cap + t.
// The rotary keys stay in the cache.
#pragma once

#include "kf_latent.cuh"
#include "kf_runs.cuh"
#include "kf_tc05_ops.cuh"

namespace kf {

struct ExpandedKV {
    uint16_t *k, *v;
    int64_t cap, rows;  // token rows a request, a head
};

// out[h][b * cap + t] = W_uk_h c_t (as hi, lo) and W_uv_h c_t for every token t < L_b.
cudaError_t launch_latent_expand(const LatentParams &p, const LatentWeights &w, const ExpandedKV &kv, int sm_count,
                                 cudaStream_t stream, tc::EncodeFn fn);

// A [rows][cols] 16-bit matrix as (64 columns, rows, column atoms): a box of `box_rows`
// rows x all columns lands as atoms of box_rows x 128 swizzled bytes.
inline bool encode_rows(tc::EncodeFn fn, CUtensorMap *map, const void *data, int64_t rows, int cols, int box_rows,
                        int box_atoms) {
    const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)cols / 64};
    const cuuint64_t strides[2] = {(cuuint64_t)cols * 2, 128};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_atoms};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(data), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The latent cache as (64 columns, 8 tokens, column atoms, 8-token groups of all
// blocks): a box of one block and `box_atoms` column atoms lands group by group,
// each group atom by atom.
inline bool encode_latent_cache(tc::EncodeFn fn, CUtensorMap *map, const LatentParams &p, int box_atoms) {
    const cuuint64_t row = (cuuint64_t)(p.latent_dim + kRopeDim) * 2;
    const cuuint64_t dims[4] = {64, 8, row / 128, (cuuint64_t)p.num_blocks * (p.block_size / 8)};
    const cuuint64_t strides[3] = {row, 128, 8 * row};
    const cuuint32_t box[4] = {64, 8, (cuuint32_t)box_atoms, (cuuint32_t)p.block_size / 8};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t *>(p.cache), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace kf
