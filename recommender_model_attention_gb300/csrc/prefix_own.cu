// The end of the tensor-core forward of shared-prefix attention: every row's
// small own keys, joined with its prefix parts, into O and lse.
//
// A block takes 32 packed rows of a tile.  First its 8 warps take the rows'
// samples in turn (at most 16 rows of one sample at a time, usually one or a
// few) and stream the sample's keys through registers: 16 keys a step, m16n8k16
// products, K and V straight from global memory in 16-byte loads.  The order
// of the contraction is free, so K's columns are dealt to the lanes as they
// are loaded (lane q of a quad takes columns 32 i + 8 q .. + 7, the queries
// alike), and V's 8-column loads make the lane of row group g own output
// columns 8 g + i of product i: nothing passes through shared memory or is
// transposed but by byte permutes.  Work is bounded by reading the keys once:
// a 128-row tile on the fifth-generation tensor core would cost each sample
// its whole chain of latencies (1.7 us a 128-key block) for a row or two.
// Then a thread per (row, 16 columns) joins the sums in shared memory with the
// row's parts.  (One user, 512 candidates with 8-64 own keys, 16384 shared:
// 280 us with the own keys as tensor-core tiles.)
#include <cuda_bf16.h>

#include "act.cuh"
#include "prefix_internal.h"
#include "prefix_mma.cuh"
#include "tc_common.cuh"

namespace gdpa {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 32;

struct OwnArgs {
    const PrefixTile* tiles;
    const PrefixOwn* own;
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16* o;
    float* lse;
    const float* parts;
    const float* ml;
    int H, Hkv, r;
    int windowed, window;
    float alpha;
};

// Attention of packed rows [0, nrows) (<= 16; row i at q + qoff(i)) over keys
// [0, nk): unnormalised sums into out[i][D + 4], (maximum, sum) into st[i].
template <int D, int ACT, typename QP>
__device__ void own_rows(const OwnArgs& a, QP qrow, int nrows, const __nv_bfloat16* k,
                         const __nv_bfloat16* v, int64_t ks, int nk, const int* ipos, float* out,
                         float2* st, int lane) {
    constexpr bool kSm = ACT == kSoftmax;
    constexpr int kC = D / 32;
    const int g = lane >> 2, q = lane & 3;
    uint4 qa[kC], qb[kC];
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < kC; ++i) {
        qa[i] = g < nrows ? ldg16(qrow(g) + 32 * i + 8 * q) : z;
        qb[i] = g + 8 < nrows ? ldg16(qrow(g + 8) + 32 * i + 8 * q) : z;
    }
    const ActScale sc = act_scale<ACT>(a.alpha);
    float acc[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    const int pos[2] = {ipos[0], ipos[1]};
    int key_lo = 0, key_hi = nk;
    if (a.windowed) {   // keys some row of the warp sees
        int lo = max(0, min(pos[0], pos[1]) - a.window + 1), hi = max(pos[0], pos[1]) + 1;
        for (int o = 4; o < 32; o <<= 1) {
            lo = min(lo, __shfl_xor_sync(~0u, lo, o));
            hi = max(hi, __shfl_xor_sync(~0u, hi, o));
        }
        key_lo = lo & ~15;
        key_hi = min(nk, hi);
    }
    for (int j0 = key_lo; j0 < key_hi; j0 += 16) {
        uint4 kk[2][kC], vv[4][D / 64];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int j = min(j0 + 8 * n + g, nk - 1);
#pragma unroll
            for (int i = 0; i < kC; ++i) kk[n][i] = ldg16(k + j * ks + 32 * i + 8 * q);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int j = j0 + 2 * q + (u & 1) + (u >> 1) * 8;
#pragma unroll
            for (int h = 0; h < D / 64; ++h) vv[u][h] = j < nk ? ldg16(v + j * ks + 64 * h + 8 * g) : z;
        }
        float s[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
            for (int i = 0; i < kC; ++i) {
                mma16816(s[n], qa[i].x, qb[i].x, qa[i].y, qb[i].y, kk[n][i].x, kk[n][i].y);
                mma16816(s[n], qa[i].z, qb[i].z, qa[i].w, qb[i].w, kk[n][i].z, kk[n][i].w);
            }
        }
        // row half x (rows g, g + 8): weights of keys j0 + 8 n + 2 q + u
        uint32_t p[2][2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            bool ok[4];
            float t[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = j0 + 8 * (e >> 1) + 2 * q + (e & 1);
                ok[e] = j < nk;
                if (a.windowed) ok[e] = ok[e] && j <= pos[x] && j > pos[x] - a.window;
                t[e] = s[e >> 1][2 * x + (e & 1)];
            }
            float w[4];
            if constexpr (kSm) {
                float top = -INFINITY;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    t[e] = ok[e] ? t[e] * sc.c0 : -INFINITY;
                    top = fmaxf(top, t[e]);
                }
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                const float mn = fmaxf(m[x], top);
                const float ref = mn == -INFINITY ? 0.0f : mn;
                const float f = ex2_approx(m[x] - ref);
                m[x] = mn;
                float sum = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e] = ex2_approx(t[e] - ref);
                    sum += w[e];
                }
                l[x] = fmaf(l[x], f, sum);
                if (f != 1.0f) {
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        acc[i][2 * x] *= f;
                        acc[i][2 * x + 1] *= f;
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = ok[e] ? act_s<ACT>(t[e], sc) : 0.0f;
            }
            p[x][0] = tc::pack_bf16x2(w[0], w[1]);
            p[x][1] = tc::pack_bf16x2(w[2], w[3]);
        }
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                mma16816(acc[8 * h + e], p[0][0], p[1][0], p[0][1], p[1][1],
                         pair_of(vv[0][h], vv[1][h], e), pair_of(vv[2][h], vv[3][h], e));
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int row = g + 8 * x;
        if (kSm) {
            l[x] += __shfl_xor_sync(~0u, l[x], 1);
            l[x] += __shfl_xor_sync(~0u, l[x], 2);
        }
        if (row >= nrows) continue;
        if (kSm && q == 0) st[row] = make_float2(m[x], l[x]);
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
#pragma unroll
            for (int u = 0; u < 2; ++u)   // product 8 h + e holds columns 64 h + 16 q + 8 u + e
#pragma unroll
                for (int e = 0; e < 8; e += 4)
                    *reinterpret_cast<float4*>(out + row * (D + 4) + 64 * h + 16 * q + 8 * u + e) =
                        make_float4(acc[8 * h + e][2 * x + u], acc[8 * h + e + 1][2 * x + u],
                                    acc[8 * h + e + 2][2 * x + u], acc[8 * h + e + 3][2 * x + u]);
    }
}

template <int D, int ACT>
__global__ void __launch_bounds__(kThreads) own_merge_kernel(const OwnArgs a) {
    constexpr bool kSm = ACT == kSoftmax;
    __shared__ __align__(16) float own_o[kRows * (D + 4)];
    __shared__ float2 own_st[kRows];
    const PrefixTile t = a.tiles[blockIdx.x];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nrows = t.n * a.r, row0 = blockIdx.y * kRows;
    if (row0 >= nrows) return;
    const int row = row0 + lane;
    const bool real = row < nrows;
    const int tl = real ? row / a.r : 0, j = row - tl * a.r, tok = t.tok + tl;
    PrefixOwn ow = {0, 0, 0, 0, 0, 0, 0, 0};
    if (real) ow = a.own[tok];
    const bool small = ow.small && ow.nk > 0;
    // runs of rows of one sample, cut at 16 rows: lane `lane` starts one?
    const int prev_k0 = __shfl_up_sync(~0u, ow.k0, 1);
    const bool prev_small = __shfl_up_sync(~0u, (int)small, 1);
    const bool fresh = lane == 0 || prev_k0 != ow.k0 || prev_small != small;
    const uint32_t starts = __ballot_sync(~0u, fresh);
    const int run0 = 31 - __clz(starts & (0xffffffffu >> (31 - lane)));
    const uint32_t cuts = __ballot_sync(~0u, fresh || (lane - run0) % 16 == 0);
    const uint32_t work = __ballot_sync(~0u, small) & cuts;
    int unit = 0;
    for (uint32_t w = work; w; w &= w - 1, ++unit) {
        if (unit % (kThreads / 32) != warp) continue;
        const int ra = __ffs(w) - 1;
        const uint32_t later = ra == 31 ? 0u : cuts >> (ra + 1);
        const int rb = min(later ? ra + __ffs(later) : 32, nrows - row0);
        const int k0 = __shfl_sync(~0u, ow.k0, ra), nk = __shfl_sync(~0u, ow.nk, ra);
        const int ip[2] = {__shfl_sync(~0u, ow.i, min(ra + (lane >> 2), rb - 1)),
                           __shfl_sync(~0u, ow.i, min(ra + (lane >> 2) + 8, rb - 1))};
        auto qrow = [&](int i) {
            const int x = row0 + ra + i, tt = x / a.r;
            return a.q + ((int64_t)(t.tok + tt) * a.H + t.hk * a.r + (x - tt * a.r)) * D;
        };
        const int64_t ks = (int64_t)a.Hkv * D, k_at = (int64_t)k0 * ks + t.hk * D;
        own_rows<D, ACT>(a, qrow, rb - ra, a.k + k_at, a.v + k_at, ks, nk, ip, own_o + ra * (D + 4),
                         own_st + ra, lane);
    }
    __syncthreads();
    if (!real) return;
    const int layers = small ? 0 : ow.layers;
    const int orow = ow.row0 + j;
    const int64_t own0 = (int64_t)ow.part + (int64_t)t.hk * ow.layers * ow.rows;
    const float2* st = reinterpret_cast<const float2*>(a.ml);
    float top = -INFINITY, sum = 0.0f, ref = 0.0f;
    if (kSm) {
        for (int i = 0; i < t.layers; ++i) top = fmaxf(top, st[(int64_t)t.part + (int64_t)i * nrows + row].x);
        for (int i = 0; i < layers; ++i) top = fmaxf(top, st[own0 + (int64_t)i * ow.rows + orow].x);
        if (small) top = fmaxf(top, own_st[lane].x);
        ref = top == -INFINITY ? 0.0f : top;
    }
    const int c = warp * (D / 32);   // this thread's float4 columns: D / 8 values of its row
    if constexpr (D == 128 || D == 64) {
        constexpr int kN = D / 32;
        float4 acc[kN];
#pragma unroll
        for (int x = 0; x < kN; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](float w, const float4& s, float4& y) {
            y.x = fmaf(w, s.x, y.x);
            y.y = fmaf(w, s.y, y.y);
            y.z = fmaf(w, s.z, y.z);
            y.w = fmaf(w, s.w, y.w);
        };
        if (small) {
            float w = 1.0f;
            if (kSm) {
                const float2 s = own_st[lane];
                w = ex2_approx(s.x - ref);   // 0 for a row that sees none of them
                sum = w * s.y;
            }
#pragma unroll
            for (int x = 0; x < kN; ++x)
                add(w, *reinterpret_cast<const float4*>(own_o + lane * (D + 4) + 4 * (c + x)), acc[x]);
        }
        for (int i = 0; i < t.layers + layers; ++i) {
            const bool pre = i < t.layers;
            const int n = pre ? nrows : ow.rows, prow = pre ? row : orow;
            const int64_t part = pre ? (int64_t)t.part + (int64_t)i * nrows : own0 + (int64_t)(i - t.layers) * n;
            float w = 1.0f;
            if (kSm) {
                const float2 s = st[part + prow];
                w = ex2_approx(s.x - ref);
                sum = fmaf(w, s.y, sum);
                if (s.x == -INFINITY) continue;
            }
            const float4* src = reinterpret_cast<const float4*>(a.parts) + part * (D / 4) + prow;
#pragma unroll
            for (int x = 0; x < kN; ++x) add(w, src[(int64_t)(c + x) * n], acc[x]);
        }
        const float inv = !kSm ? 1.0f : sum > 0.0f ? 1.0f / sum : 0.0f;
        const int64_t at = (int64_t)tok * a.H + t.hk * a.r + j;
        uint32_t out[2 * kN];
#pragma unroll
        for (int x = 0; x < kN; ++x) {
            out[2 * x] = tc::pack_bf16x2(acc[x].x * inv, acc[x].y * inv);
            out[2 * x + 1] = tc::pack_bf16x2(acc[x].z * inv, acc[x].w * inv);
        }
        uint4* dst = reinterpret_cast<uint4*>(a.o + at * D + 4 * c);
#pragma unroll
        for (int x = 0; x < kN / 2; ++x)
            dst[x] = make_uint4(out[4 * x], out[4 * x + 1], out[4 * x + 2], out[4 * x + 3]);
        if (kSm && a.lse && warp == 0)
            a.lse[at] = sum > 0.0f ? (top + log2f(sum)) * 0.69314718055994530942f : -INFINITY;
    }
}

}  // namespace

gdpa_status launch_prefix_own_merge(PrefixPlan& p, const PrefixIO& io, cudaStream_t st) {
    if (p.tiles.empty()) return GDPA_OK;
    OwnArgs a;
    a.tiles = p.dev_tiles();
    a.own = p.dev_own();
    a.q = (const __nv_bfloat16*)io.q;
    a.k = (const __nv_bfloat16*)io.k;
    a.v = (const __nv_bfloat16*)io.v;
    a.o = (__nv_bfloat16*)io.o;
    a.lse = io.act == kSoftmax ? io.lse : nullptr;
    a.parts = p.d_parts;
    a.ml = p.d_ml;
    a.H = p.H;
    a.Hkv = p.Hkv;
    a.r = p.r;
    a.windowed = p.mask == GDPA_MASK_CAUSAL_WINDOW;
    a.window = p.window;
    a.alpha = io.alpha;
    const dim3 grid((unsigned)p.tiles.size(), 4);
    if (p.d == 128) {
        if (io.act == kSoftmax)
            own_merge_kernel<128, kSoftmax><<<grid, kThreads, 0, st>>>(a);
        else
            GDPA_DISPATCH_ACT(io.act, A, own_merge_kernel<128, A><<<grid, kThreads, 0, st>>>(a))
    } else {
        if (io.act == kSoftmax)
            own_merge_kernel<64, kSoftmax><<<grid, kThreads, 0, st>>>(a);
        else
            GDPA_DISPATCH_ACT(io.act, A, own_merge_kernel<64, A><<<grid, kThreads, 0, st>>>(a))
    }
    p.launches += 1;
    return cudaGetLastError() == cudaSuccess ? GDPA_OK : GDPA_ERR_CUDA;
}

}  // namespace gdpa
