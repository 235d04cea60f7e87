// kf_row_tile.cuh -- what the kernels with a thread a query row and 128-token key tiles
// share: TMEM accesses without a wait of their own, 32-byte stores, and the online-softmax
// step of a row over one tile.
#pragma once

#include "kf_tc05_ops.cuh"

namespace kf {
namespace rows {

using namespace tc;
using namespace mq5;

// Columns [col, col + 64) of this thread's TMEM lane, not waited for; what lands in r is
// used only behind tmem_landed(r).
__device__ __forceinline__ void tmem_ld64_async(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63"
        "}, [%64];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr)
        : "memory");
}

// Every TMEM load so far has landed; r passes through, so that no use moves ahead of it.
__device__ __forceinline__ void tmem_landed(uint32_t (&r)[64]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]),
                   "+r"(r[32]), "+r"(r[33]), "+r"(r[34]), "+r"(r[35]), "+r"(r[36]), "+r"(r[37]), "+r"(r[38]), "+r"(r[39]),
                   "+r"(r[40]), "+r"(r[41]), "+r"(r[42]), "+r"(r[43]), "+r"(r[44]), "+r"(r[45]), "+r"(r[46]), "+r"(r[47]),
                   "+r"(r[48]), "+r"(r[49]), "+r"(r[50]), "+r"(r[51]), "+r"(r[52]), "+r"(r[53]), "+r"(r[54]), "+r"(r[55]),
                   "+r"(r[56]), "+r"(r[57]), "+r"(r[58]), "+r"(r[59]), "+r"(r[60]), "+r"(r[61]), "+r"(r[62]), "+r"(r[63])
                 :
                 : "memory");
}

// Columns [col, col + 16), waited for.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15"
        "}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// Stores r into columns [col, col + 16) of this thread's TMEM lane, complete behind
// tmem_wait_st().
__device__ __forceinline__ void tmem_st16_async(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {"
        "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16"
        "};"
        :
        : "r"(taddr),
          "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// A 4-D box into L2.
__device__ __forceinline__ void prefetch_4d(const CUtensorMap *map, int x, int y, int z, int w) {
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 bytes of a row: one store where the output's base allows it (whole sectors).
__device__ __forceinline__ void store32(void *dst, const uint32_t (&w)[8], bool wide) {
    if (!wide) {
        static_cast<uint4 *>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4 *>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        return;
    }
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// One row's online-softmax step over a tile of 128 tokens. x: its scores, unscaled, -inf
// where the row must not see the token; columns from `most` on are -inf in all rows of the
// warp. The weights 2^(cs x - m) go over the scores in TMEM (at ts) as NP 16-bit pieces each,
// the first rounded, the next ones what it and its predecessors left; m and l, the running
// maximum and the (unrounded) weights' sum, are updated. `arrive(half)` announces a half
// tile's 64 weights: 32 columns a piece, one piece behind the other, a half over its own
// scores; three pieces do not fit there, so both halves take the first 96 columns in turn and
// `reuse()` waits until the value product has read the first (false where that gave up).
// Two pieces of bf16 are off by up to 2^-17 of the weight (1 + 2^-9 + 2^-17: the rest of 1 lies half-way
// between bf16 numbers 2^-16 apart; outputs of 1-1261 tokens were off by 1.8e-6, four times what three
// take), three hold its 24 bits; two of fp16 are off by up to 2^-23, its last bit.
// The maximum moves only by more than 8 (base 2); then the row of O (at `to`, if has_o),
// complete up to the tile before, is rescaled, and that of its low parts (at `to_lo`, if not 0).
// F16: the weights are fp16, relative to the maximum less 7, so that they use the type's range
// whole: at most 2^15, their least step 2^-31 of the row's largest or less.
template <bool F16>
__device__ __forceinline__ constexpr float weight_lift() { return F16 ? 7.f : 0.f; }

template <int D, int NP, bool F16, typename Arrive, typename Reuse>
__device__ __forceinline__ bool row_tile(uint32_t ts, uint32_t to, uint32_t to_lo, uint32_t (&x)[2][64], int most, float cs,
                                         bool has_o, float &m, float &l, Arrive arrive, Reuse reuse) {
    constexpr float kLift = weight_lift<F16>();
    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < 128; i += 2)
        m4[(i >> 1) & 3] = max3f(m4[(i >> 1) & 3], __uint_as_float(x[i >> 6][i & 63]),
                                 __uint_as_float(x[i >> 6][(i + 1) & 63]));
    const float mx = fmaxf(max3f(m4[0], m4[1], m4[2]), m4[3]) * cs;
    const bool need = mx > m + (kLift + kRescaleSlack);
    const float alpha = need ? exp2f(m - (mx - kLift)) : 1.f;  // m = -inf: 0
    if (need) {
        l *= alpha;
        m = mx - kLift;
    }
    if (has_o && __any_sync(0xffffffffu, need)) {
#pragma unroll 1
        for (int cc = 0; cc < (to_lo ? 2 * D : D); cc += 16) {
            const uint32_t at = cc < D ? to + cc : to_lo + cc - D;
            uint32_t o[16];
            tmem_ld16(at, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st16_async(at, o);
        }
        tmem_wait_st();
    }
    const float mu = m == -INFINITY ? 0.f : m;
    const float2 c2 = make_float2(cs, cs), nm = make_float2(-mu, -mu);
    float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t w[NP][16];
        if (32 * q < most) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t *e = x[q >> 1] + 32 * (q & 1) + 2 * i;
                float2 a = fma_f32x2(make_float2(__uint_as_float(e[0]), __uint_as_float(e[1])), c2, nm);
                a.x = ex2f(a.x);
                a.y = ex2f(a.y);
                ls[i & 1] = add_f32x2(ls[i & 1], a);
#pragma unroll
                for (int n = 0; n < NP; ++n) {
                    w[n][i] = F16 ? pack_f16(a.x, a.y) : pack_bf16(a.x, a.y);
                    a.x -= F16 ? f16_lo(w[n][i]) : bf16_lo(w[n][i]);
                    a.y -= F16 ? f16_hi(w[n][i]) : bf16_hi(w[n][i]);
                }
            }
        } else {
#pragma unroll
            for (int n = 0; n < NP; ++n)
#pragma unroll
                for (int i = 0; i < 16; ++i) w[n][i] = 0;
        }
        if (NP == 3 && q == 2) {
            if (!reuse()) return false;
            tc05::fence_after_sync();
        }
#pragma unroll
        for (int n = 0; n < NP; ++n) tmem_st16_async(ts + (NP == 3 ? 0 : 64 * (q >> 1)) + 32 * n + 16 * (q & 1), w[n]);
        if (q & 1) {
            tmem_wait_st();
            tc05::fence_before_sync();
            arrive(q >> 1);
        }
    }
    ls[0] = add_f32x2(ls[0], ls[1]);
    l += ls[0].x + ls[0].y;
    return true;
}

}  // namespace rows
}  // namespace kf
