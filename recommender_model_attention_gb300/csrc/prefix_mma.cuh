// Warp-level products of the small own keys of shared-prefix attention: the
// m16n8k16 product, 16-byte loads and byte permutes.  Lane = 4 g + q.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "prefix_internal.h"

namespace gdpa {

// Of the keys of a unit that is a whole sample, those that some row sees (a
// causal row sees its own position's key: all up to the last row's).  The rest
// must not enter dQ, whose contraction runs over all of them, as 0 * inf.
__device__ __forceinline__ int keys_seen(const PrefixUnit& u, int windowed) {
    return windowed ? min(u.nk, u.ntok) : u.nk;
}

// Whether the row at position pos of such a sample sees any key: one behind the
// last key's window does not, and must not enter dK and dV the same way.
__device__ __forceinline__ bool sees_keys(const PrefixUnit& u, int pos, int windowed, int window) {
    return !windowed || pos - window < u.nk - 1;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ldg16(const __nv_bfloat16* p) {
    return __ldg(reinterpret_cast<const uint4*>(p));
}

// element e (0..7) of two 16-byte vectors as a packed pair (first: low half)
__device__ __forceinline__ uint32_t pair_of(const uint4& x, const uint4& y, int e) {
    const uint32_t a = (&x.x)[e >> 1], b = (&y.x)[e >> 1];
    return __byte_perm(a, b, (e & 1) ? 0x7632 : 0x5410);
}

}  // namespace gdpa
