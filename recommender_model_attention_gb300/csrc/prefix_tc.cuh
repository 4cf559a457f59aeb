// What the tensor-core kernels of shared-prefix attention share: the issue of
// products by one elected lane, and the records they walk.
#pragma once

#include "prefix_internal.h"
#include "tc_common.cuh"

namespace gdpa {
namespace tc {

// The issuing role runs on one elected lane of its warp, inside a branch that
// the election opens: the compiler knows such a branch to hold one lane, so
// the operands need no election or vote of their own.  (Measured on 128 x 128
// products that execute in 64 cycles, sixteen a step with four waits, beside
// eight busy warps: 1222 cycles a step; 1381 with an election a batch and a
// vote a wait; 2061 in a branch on lane 0.)  An issuer's own instructions are
// what a short chain of products waits for, so its loops keep counters rather
// than divide.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, e;\n\t}"
        : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void one_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void one_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void one_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// S = A B^T over D columns of K-major 128-byte-swizzled tiles
template <int D>
__device__ __forceinline__ void one_scores(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) one_mma_ss(d, a + kmajor_step(k), b + kmajor_step(k), idesc, k > 0);
}

// D (+)= A B over `steps` (1 .. 4) 16-row steps: A from TMEM, steps 0 and 1 at
// a, 2 and 3 at a2 (8 packed columns each); B the MN-major reading of 16-row
// steps of 128-byte rows.
__device__ __forceinline__ void one_sums(uint32_t d, uint32_t a, uint32_t a2, uint64_t b, uint32_t idesc,
                                         uint32_t steps, uint32_t accumulate) {
    one_mma_ts(d, a, b, idesc, accumulate);
    if (steps > 1) one_mma_ts(d, a + 8, b + mnmajor_step(1), idesc, 1);
    if (steps > 2) one_mma_ts(d, a2, b + mnmajor_step(2), idesc, 1);
    if (steps > 3) one_mma_ts(d, a2 + 8, b + mnmajor_step(3), idesc, 1);
}

// A place of a ring of N stages and the parity of its current use.
template <int N>
struct RingAt {
    uint32_t st = 0, ph = 0;
    __device__ __forceinline__ void next() {
        if (++st == N) {
            st = 0;
            ph ^= 1;
        }
    }
};

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
