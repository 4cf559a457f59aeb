// What the tensor-core kernels of shared-prefix attention share: products of
// 64 contracted columns issued as one batch, and warp-uniform values.
#pragma once

#include "prefix_internal.h"
#include "tc_common.cuh"

namespace gdpa {
namespace tc {

// A value that every lane of the warp holds, marked as such for the compiler:
// the tensor-core instructions take their operands from uniform registers.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// D[tmem] (+)= A B over 64 columns of K-major 128-byte-swizzled A and B: four
// K = 16 steps 32 bytes apart.  One election for the batch: the issuing warp
// shares its scheduler with four busy ones, and its instructions, not the
// tensor pipe, are what a product waits for.
__device__ __forceinline__ void mma_ss_k64(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e, t;\n\t"
        ".reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.eq.b32 t, 0, 0;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 b1, %2, 2;\n\t"
        "add.s64 a2, %1, 4;\n\tadd.s64 b2, %2, 4;\n\t"
        "add.s64 a3, %1, 6;\n\tadd.s64 b3, %2, 6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// S = A B^T over D columns (halves of 64 columns, 16 KB apart)
template <int D>
__device__ __forceinline__ void mma_scores(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
    mma_ss_k64(d, a, b, idesc, 0);
    if constexpr (D == 128) mma_ss_k64(d, a + (16384 >> 4), b + (16384 >> 4), idesc, 1);
}

// D[tmem] (+)= A B over 32 rows: A from TMEM, two K = 16 steps of 8 packed
// columns; B the MN-major reading of 16-row steps of 128-byte rows.
__device__ __forceinline__ void mma_ts_k32(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e, t;\n\t"
        ".reg .b64 b1;\n\t.reg .b32 a1;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.eq.b32 t, 0, 0;\n\t"
        "add.s64 b1, %2, 128;\n\tadd.s32 a1, %1, 8;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The same over 64 rows in four steps; the second pair's A is `a2`.
__device__ __forceinline__ void mma_ts_k64(uint32_t d, uint32_t a, uint32_t a2, uint64_t b,
                                           uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e, t;\n\t"
        ".reg .b64 b1, b2, b3;\n\t.reg .b32 a1, a3;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "setp.eq.b32 t, 0, 0;\n\t"
        "add.s64 b1, %3, 128;\n\tadd.s64 b2, %3, 256;\n\tadd.s64 b3, %3, 384;\n\t"
        "add.s32 a1, %1, 8;\n\tadd.s32 a3, %2, 8;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %3, %4, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %4, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%2], b2, %4, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %4, t;\n\t}" ::"r"(d),
        "r"(a), "r"(a2), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// D (+)= A B over `steps` (1..4) 16-row steps; A's packed columns of steps 2
// and 3 at a2.
__device__ __forceinline__ void mma_sums(uint32_t d, uint32_t a, uint32_t a2, uint64_t b, uint32_t idesc,
                                         uint32_t steps, uint32_t accumulate) {
    if (steps == 4) {
        mma_ts_k64(d, a, a2, b, idesc, accumulate);
        return;
    }
#pragma unroll 1
    for (uint32_t k = 0; k < steps; ++k)
        mma_ts(d, (k & 2 ? a2 : a) + (k & 1) * 8, b + k * 128, idesc, accumulate | k);
}

__device__ __forceinline__ void tma_load_3d(const CUtensorMap* map, uint64_t* bar, void* dst,
                                            int32_t x, int32_t y, int32_t z, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

__device__ __forceinline__ PrefixPiece load_piece(const PrefixPiece* p) {
    const int4* q = reinterpret_cast<const int4*>(p);
    const int4 a = __ldg(q), b = __ldg(q + 1), c = __ldg(q + 2);
    PrefixPiece t;
    t.tok = a.x; t.nA = a.y; t.nB = a.z; t.hk = a.w;
    t.k0 = b.x; t.nk = b.y; t.flags = b.z; t.i0 = b.w;
    t.j0 = c.x; t.part0 = c.y; t.part1 = c.z; t.pad = 0;
    return t;
}

__device__ __forceinline__ PrefixUnit load_unit(const PrefixUnit* p) {
    const int4* q = reinterpret_cast<const int4*>(p);
    const int4 a = __ldg(q), b = __ldg(q + 1);
    PrefixUnit u;
    u.k0 = a.x; u.nk = a.y; u.tok = a.z; u.ntok = a.w;
    u.hk = b.x; u.flags = b.y; u.i0 = b.z; u.j0 = b.w;
    return u;
}

}  // namespace tc
}  // namespace gdpa
