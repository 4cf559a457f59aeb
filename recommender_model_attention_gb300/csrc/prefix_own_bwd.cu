// Shared-prefix attention backward: the small own keys of units of 9 to 64
// packed rows, with warp-level products straight from global memory (as
// prefix_own.cu, which has the units of at most 8 rows).
//
// A block takes one (sample, key head); its 4 warps deal its tasks:
//   key tasks, 16 keys and 64 of the d columns: over the sample's rows 16 at
//     a time, S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q (the
//     accumulator layout of one product is the first operand's of the next);
//   row tasks, 16 rows: over the keys, S = Q K^T, dP = dO V^T, dQ += dS K,
//     into the sample's own part, which the merge adds to the prefix's.
// Every sum has one owner and one order.  Bound by reading K, V and writing
// dK, dV once; the second readings of a task hit the caches.
#include "act.cuh"
#include "prefix_internal.h"
#include "prefix_mma.cuh"
#include "tc_common.cuh"

namespace gdpa {
namespace {

constexpr int kThreads = 128;

struct OwnBwArgs {
    const PrefixUnit* units;
    const PrefixOwn* own;
    const __nv_bfloat16 *q, *k, *v, *d_o;
    __nv_bfloat16 *dk, *dv;
    const float *lse, *delta;
    float* parts;
    int H, Hkv, r;
    int windowed, window;
    float alpha;
};

template <int ACT>
__device__ __forceinline__ void weight(float s, float dp, const ActScale& k, float l2, float delta, float& p,
                                       float& ds) {
    if constexpr (ACT == kSoftmax) {
        p = ex2_approx(fmaf(s, k.c0, -l2));
        ds = p * (dp - delta);
    } else {
        float da;
        act_dact_s<ACT>(s, k, p, da);
        ds = dp * da;
    }
}

template <int D, int ACT>
__global__ void __launch_bounds__(kThreads) own_bwd_kernel(const OwnBwArgs a) {
    constexpr bool kSm = ACT == kSoftmax;
    constexpr int kC = D / 32, kW = D / 64;
    grid_let_next();
    const PrefixUnit u = a.units[blockIdx.x];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, q = lane & 3;
    const int nrows = u.ntok * a.r, seen = keys_seen(u, a.windowed);
    const int64_t ks = (int64_t)a.Hkv * D, k_at = (int64_t)u.k0 * ks + u.hk * D;
    const __nv_bfloat16 *K = a.k + k_at, *V = a.v + k_at;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    const ActScale sc = act_scale<ACT>(a.alpha);
    auto row_at = [&](int x) {   // packed row -> row of [Tq][H]
        const int t = x / a.r;
        return (int64_t)(u.tok + t) * a.H + u.hk * a.r + (x - t * a.r);
    };
    const int key_tasks = (u.nk + 15) / 16 * kW, row_tasks = (nrows + 15) / 16;
    for (int task = warp; task < key_tasks + row_tasks; task += kThreads / 32) {
        float acc[2][8][4];   // key tasks: dV and dK; row tasks: dQ's 64-column halves
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[i][e][0] = acc[i][e][1] = acc[i][e][2] = acc[i][e][3] = 0.0f;
        if (task < key_tasks) {
            const int j0 = task / kW * 16, h = task % kW;
            uint4 ka[kC], kb[kC], va[kC], vb[kC];
#pragma unroll
            for (int i = 0; i < kC; ++i) {
                const bool ga = j0 + g < u.nk, gb = j0 + g + 8 < u.nk;
                ka[i] = ga ? ldg16(K + (j0 + g) * ks + 32 * i + 8 * q) : z;
                va[i] = ga ? ldg16(V + (j0 + g) * ks + 32 * i + 8 * q) : z;
                kb[i] = gb ? ldg16(K + (j0 + g + 8) * ks + 32 * i + 8 * q) : z;
                vb[i] = gb ? ldg16(V + (j0 + g + 8) * ks + 32 * i + 8 * q) : z;
            }
            for (int r0 = 0; r0 < nrows; r0 += 16) {
                float s[2][4], dp[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
                    dp[n][0] = dp[n][1] = dp[n][2] = dp[n][3] = 0.0f;
                    const int x = r0 + 8 * n + g;
                    const int64_t at = x < nrows ? row_at(x) * D : 0;
#pragma unroll
                    for (int i = 0; i < kC; ++i) {
                        const uint4 y = x < nrows ? ldg16(a.q + at + 32 * i + 8 * q) : z;
                        const uint4 w = x < nrows ? ldg16(a.d_o + at + 32 * i + 8 * q) : z;
                        mma16816(s[n], ka[i].x, kb[i].x, ka[i].y, kb[i].y, y.x, y.y);
                        mma16816(s[n], ka[i].z, kb[i].z, ka[i].w, kb[i].w, y.z, y.w);
                        mma16816(dp[n], va[i].x, vb[i].x, va[i].y, vb[i].y, w.x, w.y);
                        mma16816(dp[n], va[i].z, vb[i].z, va[i].w, vb[i].w, w.z, w.w);
                    }
                }
                // rows r0 + 8 n + 2 q + w of keys j0 + g (x = 0) and j0 + g + 8 (x = 1)
                uint32_t pp[2][2], dd[2][2];
                uint4 qv[4], ov[4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    float l2[2] = {INFINITY, INFINITY}, dl[2] = {0.0f, 0.0f};
                    int ip[2] = {0, 0};
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const int x = r0 + 8 * n + 2 * q + w;
                        const bool real = x < nrows;
                        const int64_t at = real ? row_at(x) : 0;
                        if (kSm && real) {
                            const float l = a.lse[at];
                            l2[w] = l == -INFINITY ? INFINITY : l * kLog2e;
                            dl[w] = a.delta[at];
                        }
                        ip[w] = u.i0 + x / a.r;
                        const bool sees = real && sees_keys(u, ip[w], a.windowed, a.window);
                        qv[2 * n + w] = sees ? ldg16(a.q + at * D + 64 * h + 8 * g) : z;
                        ov[2 * n + w] = sees ? ldg16(a.d_o + at * D + 64 * h + 8 * g) : z;
                    }
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float p[2], ds[2];
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            weight<ACT>(s[n][2 * x + w], dp[n][2 * x + w], sc, l2[w], dl[w], p[w], ds[w]);
                            const int j = u.j0 + j0 + g + 8 * x;
                            bool ok = r0 + 8 * n + 2 * q + w < nrows;
                            if (a.windowed) ok = ok && j <= ip[w] && j > ip[w] - a.window;
                            if (!ok) p[w] = ds[w] = 0.0f;
                        }
                        pp[x][n] = tc::pack_bf16x2(p[0], p[1]);
                        dd[x][n] = tc::pack_bf16x2(ds[0], ds[1]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    mma16816(acc[0][e], pp[0][0], pp[1][0], pp[0][1], pp[1][1], pair_of(ov[0], ov[1], e),
                             pair_of(ov[2], ov[3], e));
                    mma16816(acc[1][e], dd[0][0], dd[1][0], dd[0][1], dd[1][1], pair_of(qv[0], qv[1], e),
                             pair_of(qv[2], qv[3], e));
                }
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int j = j0 + g + 8 * x;
                if (j >= u.nk) continue;
                // product e: columns 64 h + 16 q + e (first half) and + 8 + e
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    __nv_bfloat16* dst = (i ? a.dk : a.dv) + k_at + j * ks + 64 * h + 16 * q;
                    const float f = i ? a.alpha : 1.0f;
                    uint32_t o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        o[e] = tc::pack_bf16x2(acc[i][2 * (e & 3)][2 * x + (e >> 2)] * f,
                                               acc[i][2 * (e & 3) + 1][2 * x + (e >> 2)] * f);
                    store_sector(dst, o, !(((uintptr_t)a.dk | (uintptr_t)a.dv) & 31));
                }
            }
        } else {
            const int r0 = (task - key_tasks) * 16;
            uint4 qa[kC], qb[kC], oa[kC], ob[kC];
            float l2[2] = {INFINITY, INFINITY}, dl[2] = {0.0f, 0.0f};
            int ip[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int row = r0 + g + 8 * x;
                const bool real = row < nrows;
                const int64_t at = real ? row_at(row) : 0;
                ip[x] = u.i0 + row / a.r;
                if (kSm && real) {
                    const float l = a.lse[at];
                    l2[x] = l == -INFINITY ? INFINITY : l * kLog2e;
                    dl[x] = a.delta[at];
                }
#pragma unroll
                for (int i = 0; i < kC; ++i) {
                    (x ? qb : qa)[i] = real ? ldg16(a.q + at * D + 32 * i + 8 * q) : z;
                    (x ? ob : oa)[i] = real ? ldg16(a.d_o + at * D + 32 * i + 8 * q) : z;
                }
            }
            for (int j0 = 0; j0 < u.nk; j0 += 16) {
                float s[2][4], dp[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
                    dp[n][0] = dp[n][1] = dp[n][2] = dp[n][3] = 0.0f;
                    const int64_t j = min(j0 + 8 * n + g, u.nk - 1);
#pragma unroll
                    for (int i = 0; i < kC; ++i) {
                        const uint4 y = ldg16(K + j * ks + 32 * i + 8 * q);
                        const uint4 w = ldg16(V + j * ks + 32 * i + 8 * q);
                        mma16816(s[n], qa[i].x, qb[i].x, qa[i].y, qb[i].y, y.x, y.y);
                        mma16816(s[n], qa[i].z, qb[i].z, qa[i].w, qb[i].w, y.z, y.w);
                        mma16816(dp[n], oa[i].x, ob[i].x, oa[i].y, ob[i].y, w.x, w.y);
                        mma16816(dp[n], oa[i].z, ob[i].z, oa[i].w, ob[i].w, w.z, w.w);
                    }
                }
                uint32_t dd[2][2];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float p, ds[2];
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            weight<ACT>(s[n][2 * x + w], dp[n][2 * x + w], sc, l2[x], dl[x], p, ds[w]);
                            const int j = j0 + 8 * n + 2 * q + w;
                            bool ok = j < u.nk;
                            if (a.windowed) ok = ok && u.j0 + j <= ip[x] && u.j0 + j > ip[x] - a.window;
                            if (!ok) ds[w] = 0.0f;
                        }
                        dd[x][n] = tc::pack_bf16x2(ds[0], ds[1]);
                    }
#pragma unroll
                for (int h = 0; h < kW; ++h) {
                    uint4 kv[4];
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int j = j0 + 2 * q + (w & 1) + (w >> 1) * 8;
                        kv[w] = j < seen ? ldg16(K + j * ks + 64 * h + 8 * g) : z;
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        mma16816(acc[h][e], dd[0][0], dd[1][0], dd[0][1], dd[1][1], pair_of(kv[0], kv[1], e),
                                 pair_of(kv[2], kv[3], e));
                }
            }
            const PrefixOwn ow = a.own[u.tok];
            const int64_t part = (int64_t)ow.part + (int64_t)u.hk * ow.rows;
            float4* out = reinterpret_cast<float4*>(a.parts) + part * (D / 4);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int row = r0 + g + 8 * x;
                if (row >= nrows) continue;
#pragma unroll
                for (int h = 0; h < kW; ++h)
#pragma unroll
                    for (int w = 0; w < 2; ++w)
#pragma unroll
                        for (int e = 0; e < 8; e += 4)
                            out[(16 * h + 4 * q + 2 * w + e / 4) * ow.rows + row] =
                                make_float4(acc[h][e][2 * x + w] * a.alpha, acc[h][e + 1][2 * x + w] * a.alpha,
                                            acc[h][e + 2][2 * x + w] * a.alpha, acc[h][e + 3][2 * x + w] * a.alpha);
            }
        }
    }
}

}  // namespace

gdpa_status launch_prefix_own_bwd(PrefixPlan& p, const PrefixIO& io, const float* delta, cudaStream_t st) {
    if ((int64_t)p.smalls.size() == p.n_small8) return GDPA_OK;
    OwnBwArgs a;
    a.units = p.dev_smalls() + p.n_small8;
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
    a.H = p.H;
    a.Hkv = p.Hkv;
    a.r = p.r;
    a.windowed = p.mask == GDPA_MASK_CAUSAL_WINDOW;
    a.window = p.window;
    a.alpha = io.alpha;
    const unsigned grid = (unsigned)((int64_t)p.smalls.size() - p.n_small8);
    if (p.d == 128) {
        if (io.act == kSoftmax)
            own_bwd_kernel<128, kSoftmax><<<grid, kThreads, 0, st>>>(a);
        else
            GDPA_DISPATCH_ACT(io.act, A, own_bwd_kernel<128, A><<<grid, kThreads, 0, st>>>(a))
    } else {
        if (io.act == kSoftmax)
            own_bwd_kernel<64, kSoftmax><<<grid, kThreads, 0, st>>>(a);
        else
            GDPA_DISPATCH_ACT(io.act, A, own_bwd_kernel<64, A><<<grid, kThreads, 0, st>>>(a))
    }
    p.launches += 1;
    p.chain += 1;
    return cudaGetLastError() == cudaSuccess ? GDPA_OK : GDPA_ERR_CUDA;
}

}  // namespace gdpa
