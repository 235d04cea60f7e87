// kf_tc05_ops.cuh -- further building blocks of tcgen05 kernels: an elected lane, a
// 3-D TMA box, the fp16 instruction descriptor.
#pragma once

#include "kf_mq_tc05.cuh"

namespace kf {
namespace tc05 {

// idesc_bf16 with both inputs fp16 (format 0).
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn_major, bool b_mn_major) {
    return idesc_bf16(M, N, a_mn_major, b_mn_major) & ~((1u << 7) | (1u << 10));
}

// One lane of a converged warp (the same one every time). Instructions that only it
// issues keep their operands in uniform registers: an MMA's descriptors then cost 36
// cycles an instruction instead of 58 (measured, M = 64, N = 64).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// A 3-D box into shared memory.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

}  // namespace tc05
}  // namespace kf
