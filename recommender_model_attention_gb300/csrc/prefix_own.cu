// Shared-prefix attention, tensor-core family: the small own keys (the rule is
// the planner's: few packed rows, few keys), forward and backward, for up to 8
// packed rows of a sample at a time.
//
// A warp takes 8 rows of one (sample, key head) and streams the sample's keys
// through registers, 16 a step, with m16n8k16 products in the orientation
// that fills them with 8 rows: S^T = K Q^T (16 keys x 8 rows), then O^T = V^T
// P^T.  The order of a contraction is free, so K's columns are dealt to the
// lanes as 16-byte loads bring them (lane q of a quad takes columns 32 i + 8 q
// .. + 7, the queries alike), and V's 8-column loads make the lane of group g
// own output columns 8 g + e of product e; a weight's 8x8 blocks change from
// accumulator to operand layout by movmatrix.  The work is bounded by reading
// the keys once; a 128-row tile on the fifth-generation tensor core would cost
// every sample its whole chain of latencies for a row or two.  Forward, 16
// warps an SM, keys in registers: 75 MB of keys of 512 candidates in 19 us
// (through shared memory as below the same, and slower for d = 64).
//
// The backward of a unit of at most 8 rows runs in one warp too: each key's
// dK and dV are done in its step, dQ^T = K^T dS^T adds up over the steps, so
// every sum has one owner and one order.  It has registers for 8 warps an SM
// only, so the next step's keys are copied to shared memory meanwhile, and dK
// and dV leave as whole sectors: 44 us for a training batch of 32 users (0.2
// GB in all), 47 with the keys prefetched into L2 as well; beside that, keys
// loaded into registers 54, with 12 warps 54, half sectors 54.
#include "act.cuh"
#include "prefix_internal.h"
#include "prefix_mma.cuh"
#include "tc_common.cuh"

namespace gdpa {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

struct OwnArgs {
    const PrefixUnit* units;   // 8 rows of a sample each (j0: the first packed row)
    int n;
    const PrefixOwn* own;
    const __nv_bfloat16 *q, *k, *v, *d_o;
    __nv_bfloat16 *dk, *dv;
    const float *lse, *delta;
    float* parts;
    float* ml;
    int H, Hkv, r;
    int windowed, window;
    float alpha;
};

// the transpose of an 8x8 block of 16-bit values spread over the warp
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t o;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(o) : "r"(v));
    return o;
}

// A operand of product e of X^T (columns x keys): rows g and g + 8 of the
// operand are columns 8 g + e and, for d = 128, 64 + 8 g + e (d = 64: 8 g + e
// and 8 g + e + 4); x[u][h] are 8 columns of keys 2 q, 2 q + 1, 2 q + 8, 2 q + 9.
template <int D>
__device__ __forceinline__ void operand_t(const uint4 (&x)[4][D / 64], int e, uint32_t& a0, uint32_t& a1,
                                          uint32_t& a2, uint32_t& a3) {
    constexpr int h = D == 128 ? 1 : 0, f = D == 128 ? 0 : 4;
    a0 = pair_of(x[0][0], x[1][0], e);
    a1 = pair_of(x[0][h], x[1][h], e + f);
    a2 = pair_of(x[2][0], x[3][0], e);
    a3 = pair_of(x[2][h], x[3][h], e + f);
}
template <int D>
constexpr int products() { return D / 16; }

// Write X^T's accumulator of rows 2 q + w (w = 0, 1) to a part: columns 8 g ..
// + 7 and, for d = 128, 64 + 8 g .. + 7.
template <int D>
__device__ __forceinline__ void store_part(const float (&acc)[D / 16][4], float scale, float* parts, int64_t part,
                                           int rows, int row0, int nrows, int g, int q) {
    float4* out = reinterpret_cast<float4*>(parts) + part * (D / 4);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const int row = row0 + 2 * q + w;
        if (2 * q + w >= nrows) continue;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {   // float4 column: which products, which half
            const int e = D == 128 ? 4 * (c & 1) : 0, x = D == 128 ? c >> 1 : c;
            const int col = D == 128 ? (c >> 1) * 16 + 2 * g + (c & 1) : 2 * g + c;
            out[(int64_t)col * rows + row] =
                make_float4(acc[e][2 * x + w] * scale, acc[e + 1][2 * x + w] * scale,
                            acc[e + 2][2 * x + w] * scale, acc[e + 3][2 * x + w] * scale);
        }
    }
}

// Bring keys [j0, j1) of K and V (rows of D columns, ks apart) into L2, a 128-
// byte line a lane: the steps' loads then wait for L2 rather than, each in
// turn, for memory.
template <int D>
__device__ __forceinline__ void prefetch_keys(const __nv_bfloat16* K, const __nv_bfloat16* V, int64_t ks, int j0,
                                              int j1, int lane) {
    constexpr int kLines = D / 64;
    for (int i = lane; i < (j1 - j0) * 2 * kLines; i += 32) {
        const int j = j0 + i / (2 * kLines), x = i % (2 * kLines);
        const __nv_bfloat16* p = (x < kLines ? K : V) + j * ks + (x % kLines) * 64;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
    }
}
// Keys ahead.  (500 samples of one row on 100 to 500 keys, 4 heads, d = 128,
// forward: 82 us, 86 with 32, 95 with 64, 128 without.  The backward's copies to
// shared memory run ahead by themselves: 125 us, 132 with a prefetch as well.)
constexpr int kAhead = 16;

struct Rows {   // the unit's rows, as this lane meets them
    int nrows, row0, tok, hk, r, H;
    __device__ __forceinline__ int64_t at(int i) const {   // row of [Tq][H]
        const int x = row0 + i, t = x / r;
        return (int64_t)(tok + t) * H + hk * r + (x - t * r);
    }
};

template <int D, int ACT>
__global__ void __launch_bounds__(kThreads, 4) own_fwd_kernel(const OwnArgs a) {
    constexpr bool kSm = ACT == kSoftmax;
    constexpr int kC = D / 32;
    grid_let_next();
    const int unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (unit >= a.n) return;
    const PrefixUnit u = a.units[unit];
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const Rows rows{min(8, u.ntok * a.r - u.j0), u.j0, u.tok, u.hk, a.r, a.H};
    const int64_t ks = (int64_t)a.Hkv * D, k_at = (int64_t)u.k0 * ks + u.hk * D;
    const __nv_bfloat16 *K = a.k + k_at, *V = a.v + k_at;
    int ja = 0, jb = u.nk;
    if (a.windowed) {   // keys some row sees
        ja = max(0, rows.row0 / a.r - a.window + 1);
        jb = min(jb, (rows.row0 + rows.nrows - 1) / a.r + 1);
    }
    prefetch_keys<D>(K, V, ks, ja, min(jb, ja + kAhead), lane);
    const PrefixOwn ow = a.own[u.tok];
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    uint4 qb[kC];
    {
        const int64_t at = g < rows.nrows ? rows.at(g) * D : 0;
#pragma unroll
        for (int i = 0; i < kC; ++i) qb[i] = g < rows.nrows ? ldg16(a.q + at + 32 * i + 8 * q) : z;
    }
    const ActScale sc = act_scale<ACT>(a.alpha);
    float acc[products<D>()][4];
#pragma unroll
    for (int e = 0; e < products<D>(); ++e) acc[e][0] = acc[e][1] = acc[e][2] = acc[e][3] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};   // rows 2 q, 2 q + 1
    const int pos[2] = {(rows.row0 + min(2 * q, rows.nrows - 1)) / a.r,
                        (rows.row0 + min(2 * q + 1, rows.nrows - 1)) / a.r};
    for (int j0 = ja; j0 < jb; j0 += 16) {
        if (j0 + kAhead < jb) prefetch_keys<D>(K, V, ks, j0 + kAhead, min(jb, j0 + kAhead + 16), lane);
        uint4 ka[kC], kb[kC], vv[4][D / 64];
        {
            const int64_t x = min(j0 + g, jb - 1) * ks, y = min(j0 + g + 8, jb - 1) * ks;
#pragma unroll
            for (int i = 0; i < kC; ++i) {
                ka[i] = ldg16(K + x + 32 * i + 8 * q);
                kb[i] = ldg16(K + y + 32 * i + 8 * q);
            }
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int j = j0 + 2 * q + (w & 1) + (w >> 1) * 8;
#pragma unroll
            for (int h = 0; h < D / 64; ++h)   // (values nobody sees must not enter as 0 * inf)
                vv[w][h] = j < jb ? ldg16(V + j * ks + 64 * h + 8 * g) : z;
        }
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};   // key g: rows 2 q, + 1; key g + 8: the same
#pragma unroll
        for (int i = 0; i < kC; ++i) {
            mma16816(s, ka[i].x, kb[i].x, ka[i].y, kb[i].y, qb[i].x, qb[i].y);
            mma16816(s, ka[i].z, kb[i].z, ka[i].w, kb[i].w, qb[i].z, qb[i].w);
        }
        float p[4];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            bool ok[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int j = j0 + g + 8 * x;
                ok[x] = j < jb;
                if (a.windowed) ok[x] = ok[x] && j <= pos[w] && j > pos[w] - a.window;
            }
            if constexpr (kSm) {
                const float t0 = ok[0] ? s[w] * sc.c0 : -INFINITY, t1 = ok[1] ? s[2 + w] * sc.c0 : -INFINITY;
                float top = fmaxf(t0, t1);
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
                const float mn = fmaxf(m[w], top);
                const float ref = mn == -INFINITY ? 0.0f : mn;
                const float f = ex2_approx(m[w] - ref);
                m[w] = mn;
                p[w] = ex2_approx(t0 - ref);
                p[2 + w] = ex2_approx(t1 - ref);
                l[w] = fmaf(l[w], f, p[w] + p[2 + w]);
                if (f != 1.0f) {
#pragma unroll
                    for (int e = 0; e < products<D>(); ++e) {
                        acc[e][w] *= f;
                        acc[e][2 + w] *= f;
                    }
                }
            } else {
                p[w] = ok[0] ? act_s<ACT>(s[w], sc) : 0.0f;
                p[2 + w] = ok[1] ? act_s<ACT>(s[2 + w], sc) : 0.0f;
            }
        }
        const uint32_t b0 = transposed(tc::pack_bf16x2(p[0], p[1])), b1 = transposed(tc::pack_bf16x2(p[2], p[3]));
#pragma unroll
        for (int e = 0; e < products<D>(); ++e) {
            uint32_t a0, a1, a2, a3;
            operand_t<D>(vv, e, a0, a1, a2, a3);
            mma16816(acc[e], a0, a1, a2, a3, b0, b1);
        }
    }
    const int64_t part = (int64_t)ow.part + (int64_t)u.hk * ow.rows;
    store_part<D>(acc, 1.0f, a.parts, part, ow.rows, rows.row0, rows.nrows, g, q);
    if (kSm) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            for (int o = 4; o < 32; o <<= 1) l[w] += __shfl_xor_sync(~0u, l[w], o);
            if (g == 0 && 2 * q + w < rows.nrows)
                reinterpret_cast<float2*>(a.ml)[part + rows.row0 + 2 * q + w] = make_float2(counted(m[w], l[w]), l[w]);
        }
    }
}

// 16 keys of K, then of V, in shared memory: rows of D + 8 columns, so that
// four rows two apart start in different banks.  A lane's copies of the keys
// from j0 on (rows past the last one hold it again).
template <int D>
struct Stage {
    static constexpr int kRow = D + 8, kKeys = 16 * kRow;   // elements
    static constexpr int kBytes = 2 * kKeys * 2;
};

template <int D>
__device__ __forceinline__ void load_stage(__nv_bfloat16* to, const __nv_bfloat16* K, const __nv_bfloat16* V,
                                           int64_t ks, int j0, int nk, int lane) {
    constexpr int kChunks = D / 8;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int x = lane + 32 * i, row = x / kChunks, c = 8 * (x % kChunks);
        const __nv_bfloat16* src = (row < 16 ? K : V) + min(j0 + (row & 15), nk - 1) * ks + c;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(to + row * Stage<D>::kRow + c)),
                     "l"(src)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// a pair less its rounding to bf16, rounded itself
__device__ __forceinline__ uint32_t rest_of(float x, float y, uint32_t rounded) {
    return tc::pack_bf16x2(x - __uint_as_float(rounded << 16), y - __uint_as_float(rounded & 0xffff0000u));
}

__device__ __forceinline__ uint4 lds16(const __nv_bfloat16* p) { return *reinterpret_cast<const uint4*>(p); }

// Backward of units of at most 8 rows.
template <int D, int ACT>
__global__ void __launch_bounds__(kThreads, 2) own_bwd8_kernel(const OwnArgs a) {
    constexpr bool kSm = ACT == kSoftmax;
    constexpr int kC = D / 32, kW = D / 64;
    grid_let_next();
    const int unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (unit >= a.n) return;
    const PrefixUnit u = a.units[unit];
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const Rows rows{min(8, u.ntok * a.r), 0, u.tok, u.hk, a.r, a.H};
    const int64_t ks = (int64_t)a.Hkv * D, k_at = (int64_t)u.k0 * ks + u.hk * D;
    const __nv_bfloat16 *K = a.k + k_at, *V = a.v + k_at;
    const int seen = keys_seen(u, a.windowed);
    extern __shared__ uint4 own_smem[];   // two stages a warp
    __nv_bfloat16* stage = reinterpret_cast<__nv_bfloat16*>(own_smem) + (threadIdx.x >> 5) * 4 * Stage<D>::kKeys;
    load_stage<D>(stage, K, V, ks, 0, u.nk, lane);
    const PrefixOwn ow = a.own[u.tok];
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    const ActScale sc = act_scale<ACT>(a.alpha);
    // rows as the second operand of the scores (row g) and of dK, dV (rows
    // 2 q, 2 q + 1, twice)
    uint4 qb[kC], ob[kC], qv[2][kW], ov[2][kW];
    float l2[2] = {INFINITY, INFINITY}, dl[2] = {0.0f, 0.0f};
    int pos[2];
    {
        const int64_t at = g < rows.nrows ? rows.at(g) * D : 0;
#pragma unroll
        for (int i = 0; i < kC; ++i) {
            qb[i] = g < rows.nrows ? ldg16(a.q + at + 32 * i + 8 * q) : z;
            ob[i] = g < rows.nrows ? ldg16(a.d_o + at + 32 * i + 8 * q) : z;
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const int i = 2 * q + w;
            const bool real = i < rows.nrows;
            const int64_t x = real ? rows.at(i) : 0;
            pos[w] = i / a.r;
            const bool sees = real && sees_keys(u, pos[w], a.windowed, a.window);
#pragma unroll
            for (int h = 0; h < kW; ++h) {
                qv[w][h] = sees ? ldg16(a.q + x * D + 64 * h + 8 * g) : z;
                ov[w][h] = sees ? ldg16(a.d_o + x * D + 64 * h + 8 * g) : z;
            }
            if (kSm && real) {
                const float y = a.lse[x];
                l2[w] = y == -INFINITY ? INFINITY : y * kLog2e;
                dl[w] = a.delta[x];
            }
        }
    }
    const bool wide = !(((uintptr_t)a.dk | (uintptr_t)a.dv) & 31);
    float acc[products<D>()][4];   // dQ^T
#pragma unroll
    for (int e = 0; e < products<D>(); ++e) acc[e][0] = acc[e][1] = acc[e][2] = acc[e][3] = 0.0f;
#pragma unroll 1
    for (int j0 = 0; j0 < u.nk; j0 += 16) {
        const __nv_bfloat16* kk = stage + (j0 & 16 ? 2 * Stage<D>::kKeys : 0);
        const __nv_bfloat16* vv = kk + Stage<D>::kKeys;
        if (j0 + 16 < u.nk) {   // the next keys' copies fly while these are worked on
            load_stage<D>(stage + (j0 & 16 ? 0 : 2 * Stage<D>::kKeys), K, V, ks, j0 + 16, u.nk, lane);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncwarp();
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f}, dp[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        {
            const int x = g * Stage<D>::kRow + 8 * q, y = x + 8 * Stage<D>::kRow;
#pragma unroll
            for (int i = 0; i < kC; ++i) {
                const uint4 ka = lds16(kk + x + 32 * i), kb = lds16(kk + y + 32 * i);
                const uint4 va = lds16(vv + x + 32 * i), vb = lds16(vv + y + 32 * i);
                mma16816(s, ka.x, kb.x, ka.y, kb.y, qb[i].x, qb[i].y);
                mma16816(dp, va.x, vb.x, va.y, vb.y, ob[i].x, ob[i].y);
                mma16816(s, ka.z, kb.z, ka.w, kb.w, qb[i].z, qb[i].w);
                mma16816(dp, va.z, vb.z, va.w, vb.w, ob[i].z, ob[i].w);
            }
        }
        float p[4], ds[4];
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int j = j0 + g + 8 * x, c = 2 * x + w;
                bool ok = j < u.nk && 2 * q + w < rows.nrows;
                if (a.windowed) ok = ok && j <= pos[w] && j > pos[w] - a.window;
                if constexpr (kSm) {
                    p[c] = ex2_approx(fmaf(s[c], sc.c0, -l2[w]));
                    ds[c] = p[c] * (dp[c] - dl[w]);
                } else {
                    float da;
                    act_dact_s<ACT>(s[c], sc, p[c], da);
                    ds[c] = dp[c] * da;
                }
                if (!ok) p[c] = ds[c] = 0.0f;
            }
        // rows 2 q, 2 q + 1 of keys g and g + 8: the first operand of dV, dK;
        // what bf16 leaves of them takes the contraction's other 8 rows
        const uint32_t p0 = tc::pack_bf16x2(p[0], p[1]), p1 = tc::pack_bf16x2(p[2], p[3]);
        const uint32_t d0 = tc::pack_bf16x2(ds[0], ds[1]), d1 = tc::pack_bf16x2(ds[2], ds[3]);
        const uint32_t p2 = rest_of(p[0], p[1], p0), p3 = rest_of(p[2], p[3], p1);
        const uint32_t d2 = rest_of(ds[0], ds[1], d0), d3 = rest_of(ds[2], ds[3], d1);
#pragma unroll
        for (int i = 0; i < 2; ++i)   // dV, then dK
#pragma unroll
            for (int h = 0; h < kW; ++h) {
                float o[8][4];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    o[e][0] = o[e][1] = o[e][2] = o[e][3] = 0.0f;
                    const uint32_t b = i ? pair_of(qv[0][h], qv[1][h], e) : pair_of(ov[0][h], ov[1][h], e);
                    mma16816(o[e], i ? d0 : p0, i ? d1 : p1, i ? d2 : p2, i ? d3 : p3, b, b);
                }
                // product e: columns 64 h + 16 q + e and + 8 + e of keys g, g + 8
                const float f = i ? a.alpha : 1.0f;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int j = j0 + g + 8 * x;
                    if (j >= u.nk) continue;
                    __nv_bfloat16* dst = (i ? a.dk : a.dv) + k_at + j * ks + 64 * h + 16 * q;
                    uint32_t y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[e] = tc::pack_bf16x2(o[2 * (e & 3)][2 * x + (e >> 2)] * f,
                                               o[2 * (e & 3) + 1][2 * x + (e >> 2)] * f);
                    store_sector(dst, y, wide);
                }
            }
        uint4 kv[4][kW];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int j = 2 * q + (w & 1) + (w >> 1) * 8;
#pragma unroll
            for (int h = 0; h < kW; ++h)
                kv[w][h] = j0 + j < seen ? lds16(kk + j * Stage<D>::kRow + 64 * h + 8 * g) : z;
        }
        __syncwarp();   // (read: the next step's copies may overwrite them)
        const uint32_t b0 = transposed(d0), b1 = transposed(d1);
#pragma unroll
        for (int e = 0; e < products<D>(); ++e) {
            uint32_t a0, a1, a2, a3;
            operand_t<D>(kv, e, a0, a1, a2, a3);
            mma16816(acc[e], a0, a1, a2, a3, b0, b1);
        }
    }
    store_part<D>(acc, a.alpha, a.parts, (int64_t)ow.part + (int64_t)u.hk * ow.rows, ow.rows, 0, rows.nrows, g, q);
}

OwnArgs args_of(const PrefixPlan& p, const PrefixIO& io, const float* delta) {
    OwnArgs a;
    a.units = nullptr;
    a.n = 0;
    a.own = p.dev_own();
    a.q = (const __nv_bfloat16*)io.q;
    a.k = (const __nv_bfloat16*)io.k;
    a.v = (const __nv_bfloat16*)io.v;
    a.d_o = (const __nv_bfloat16*)io.d_o;
    a.dk = (__nv_bfloat16*)io.dk;
    a.dv = (__nv_bfloat16*)io.dv;
    a.lse = io.lse;
    a.delta = delta;
    a.parts = p.d_parts;
    a.ml = p.d_ml;
    a.H = p.H;
    a.Hkv = p.Hkv;
    a.r = p.r;
    a.windowed = p.mask == GDPA_MASK_CAUSAL_WINDOW;
    a.window = p.window;
    a.alpha = io.alpha;
    return a;
}

template <int D, int ACT>
bool go(bool bwd, int device, const OwnArgs& a, cudaStream_t st) {
    const unsigned grid = (unsigned)((a.n + kWarps - 1) / kWarps);
    if (bwd) {
        constexpr int kSmem = kWarps * 2 * Stage<D>::kBytes;
        static std::atomic<uint64_t> done{0};
        if (!allow_smem(own_bwd8_kernel<D, ACT>, kSmem, device, done)) return false;
        own_bwd8_kernel<D, ACT><<<grid, kThreads, kSmem, st>>>(a);
    } else {
        own_fwd_kernel<D, ACT><<<grid, kThreads, 0, st>>>(a);
    }
    return true;
}

gdpa_status dispatch(bool bwd, PrefixPlan& p, const OwnArgs& a, int act, cudaStream_t st) {
    if (a.n == 0) return GDPA_OK;
    bool ok = false;
    if (p.d == 128) {
        if (act == kSoftmax)
            ok = go<128, kSoftmax>(bwd, p.device, a, st);
        else
            GDPA_DISPATCH_ACT(act, A, ok = go<128, A>(bwd, p.device, a, st))
    } else {
        if (act == kSoftmax)
            ok = go<64, kSoftmax>(bwd, p.device, a, st);
        else
            GDPA_DISPATCH_ACT(act, A, ok = go<64, A>(bwd, p.device, a, st))
    }
    p.launches += 1;
    p.chain += 1;
    return ok && cudaGetLastError() == cudaSuccess ? GDPA_OK : GDPA_ERR_CUDA;
}

}  // namespace

gdpa_status launch_prefix_own_fwd(PrefixPlan& p, const PrefixIO& io, cudaStream_t st) {
    OwnArgs a = args_of(p, io, nullptr);
    a.units = p.dev_eights();
    a.n = (int)p.eights.size();
    return dispatch(false, p, a, io.act, st);
}

gdpa_status launch_prefix_own_bwd8(PrefixPlan& p, const PrefixIO& io, const float* delta, cudaStream_t st) {
    OwnArgs a = args_of(p, io, delta);
    a.units = p.dev_smalls();
    a.n = (int)p.n_small8;
    return dispatch(true, p, a, io.act, st);
}

}  // namespace gdpa
