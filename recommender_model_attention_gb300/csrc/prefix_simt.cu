// Shared-prefix attention on the CUDA cores: float32 arithmetic for float32
// rows and for head dims that the tensor-core kernels do not take; and the
// merge of the parts, which both families share.
//
// Forward and dQ walk the plan's pieces: a block of 4 warps takes 32 rows of
// one slot of a piece, 8 rows a warp (or 8 rows, 2 a warp), and streams its
// keys through shared memory 32 at a time; a lane owns one key of the scores,
// and for the sums four columns of every key, or of every second, fourth, ...
// where a row has fewer than 128 columns.  Forward keeps a running maximum and
// sum per row.  dK and dV walk the backward units: 32 keys a block, 8 a warp,
// all of the unit's rows that see them streamed 32 at a time, so that each
// gradient row (or its part, where a unit's rows were split) is written once, by
// one warp, in an order that never changes.  They are bound by shared-memory
// reads (9 16-byte reads for 32 multiply-adds in the scores): 512 rows on 1000
// keys in 16 groups of 2 key heads, d = 128, 0.43 ms forward, 20 TFLOP/s; float32
// has no tensor-core path that keeps its products.
#include <cuda_bf16.h>

#include "act.cuh"
#include "prefix_internal.h"
#include "tc_common.cuh"

namespace gdpa {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 32;    // rows (or keys) of a block
constexpr int kPer = 8;      // of a warp

struct SimtArgs {
    const PrefixPiece* pieces;
    const RowBlock* blocks;
    const PrefixUnit* units;
    const void *q, *kp, *vp, *k, *v, *d_o;
    const float *lse, *delta;
    float* parts;
    float* ml;
    float* unit_parts;
    void *dkp, *dvp, *dk, *dv;
    int H, Hkv, r, d;
    int windowed, window;
    float alpha;
};

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ void st4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void st4(__nv_bfloat16* p, float4 v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(tc::pack_bf16x2(v.x, v.y), tc::pack_bf16x2(v.z, v.w));
}
__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}
__device__ __forceinline__ void axpy4(float4& y, float a, float4 x) {
    y.x = fmaf(a, x.x, y.x);
    y.y = fmaf(a, x.y, y.y);
    y.z = fmaf(a, x.z, y.z);
    y.w = fmaf(a, x.w, y.w);
}

// rows [0, n) of `ld_elems`-strided global rows into a [32][stride] float tile
template <typename E>
__device__ __forceinline__ void load_tile(float* dst, int stride, const E* src, int64_t row_stride,
                                          int n, int d) {
    const int c4 = d / 4;
    for (int i = threadIdx.x; i < kRows * c4; i += kThreads) {
        const int row = i / c4, c = i - row * c4;
        const float4 v = row < n ? ld4(src + row * row_stride + 4 * c) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(dst + row * stride + 4 * c) = v;
    }
}

// The same of float32 rows, copied while the threads go on (rows past n as
// zeros); tile_arrived waits for the thread's own copies.
__device__ __forceinline__ void copy_tile(float* dst, int stride, const float* src, int64_t row_stride, int n, int d) {
    const int c4 = d / 4;
    for (int i = threadIdx.x; i < kRows * c4; i += kThreads) {
        const int row = i / c4, c = i - row * c4;
        const float* from = src + (row < n ? row : 0) * row_stride + 4 * c;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst + row * stride + 4 * c)),
                     "l"(from), "r"(row < n ? 16 : 0)
                     : "memory");
    }
}
__device__ __forceinline__ void tile_arrived() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// packed rows [row0, row0 + ROWS) of tokens from `tok` (row = token * r + head
// within the group of query heads), rows >= nrows as zeros
template <int ROWS, typename E>
__device__ __forceinline__ void load_rows(float* dst, int stride, const E* src, const SimtArgs& a,
                                          int tok, int hk, int row0, int nrows) {
    const int c4 = a.d / 4;
    for (int i = threadIdx.x; i < ROWS * c4; i += kThreads) {
        const int rl = i / c4, c = i - rl * c4, row = row0 + rl;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row < nrows) {
            const int t = row / a.r;
            v = ld4(src + ((int64_t)(tok + t) * a.H + hk * a.r + (row - t * a.r)) * a.d + 4 * c);
        }
        *reinterpret_cast<float4*>(dst + rl * stride + 4 * c) = v;
    }
}

// p and ds of one pair, in the float32 path's precise forms.  t = the scaled
// score; lse, delta: the row's (softmax).
template <int ACT>
__device__ __forceinline__ void p_ds(float t, float dp, float lse, float delta, float& p, float& ds) {
    if constexpr (ACT == kSoftmax) {
        p = expf(t - lse);
        ds = p * (dp - delta);
    } else {
        float da;
        act_dact_f<ACT, false>(t, p, da);
        ds = dp * da;
    }
}

template <int R>
__device__ __forceinline__ void load_weights(float* p, const float* w) {
    if constexpr (R == 2) {
        *reinterpret_cast<float2*>(p) = *reinterpret_cast<const float2*>(w);
    } else {
#pragma unroll
        for (int i = 0; i < R; i += 4) *reinterpret_cast<float4*>(p + i) = *reinterpret_cast<const float4*>(w + i);
    }
}

// the sum over a warp's ng groups of c4 lanes, in its first group
__device__ __forceinline__ void join_lanes(float4& v, int lane, int g, int ng, int c4) {
    for (int s = 1; s < ng; s *= 2) {
        const int from = (lane + s * c4) & 31;
        const float x = __shfl_sync(~0u, v.x, from), y = __shfl_sync(~0u, v.y, from);
        const float z = __shfl_sync(~0u, v.z, from), w = __shfl_sync(~0u, v.w, from);
        if ((g & (2 * s - 1)) == 0 && g + s < ng) {
            v.x += x;
            v.y += y;
            v.z += z;
            v.w += w;
        }
    }
}

// Forward (BWD false) or dQ (BWD true) of 4 R rows of a slot of a piece, R a warp.
template <typename E, int ACT, bool BWD, int R>
__global__ void __launch_bounds__(kThreads, R == 2 ? 7 : BWD ? 3 : 4) simt_rows_kernel(const SimtArgs a) {
    extern __shared__ float sm[];
    constexpr int kBlock = 4 * R;
    const RowBlock rb = a.blocks[blockIdx.x];
    const PrefixPiece pc = a.pieces[rb.piece];
    const int slot = rb.sub & 1, row0 = (rb.sub >> 1) * kBlock;
    const int part = slot ? pc.part1 : pc.part0;
    const bool dual = pc.flags & kPieceDual, own = pc.flags & kPieceOwn;
    const int tok = pc.tok + (!dual && slot ? pc.nA : 0);
    const int nrows = (!dual && slot ? pc.nB : pc.nA) * a.r;
    const int i0 = pc.i0 + (tok - pc.tok);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int qs = a.d, ks = a.d + 4;
    float* Q = sm;                       // [4 R][d]
    float* DO = Q + kBlock * qs;          // [4 R][d] (BWD)
    // float32 keys, few rows: two tiles in turn, the next one copied meanwhile
    // (8 rows a warp hide the loads behind more blocks, for which two tiles
    // leave no shared memory)
    constexpr int kTiles = sizeof(E) == 4 && R == 2 ? 2 : 1;
    float* const KV = DO + (BWD ? kBlock * qs : 0);   // K, V: [32][d + 4] each
    float* W = KV + kTiles * 2 * kRows * ks + warp * kRows * R;   // weights [32 keys][R rows]
    const E* kb = (const E*)(own ? a.k : a.kp);
    const E* vb = (const E*)(own ? a.v : a.vp);
    load_rows<kBlock>(Q, qs, (const E*)a.q, a, tok, pc.hk, row0, nrows);
    if constexpr (BWD) load_rows<kBlock>(DO, qs, (const E*)a.d_o, a, tok, pc.hk, row0, nrows);
    // the sums: a lane has four columns of every ng-th key
    const int c4 = a.d / 4, ng = 32 / c4, g = lane / c4, gc = lane - g * c4;
    float4 acc[R];
    float m[R], l[R], lse[R], delta[R];
    int ipos[R];
#pragma unroll
    for (int w = 0; w < R; ++w) {
        acc[w] = make_float4(0.f, 0.f, 0.f, 0.f);
        m[w] = -INFINITY;
        l[w] = 0.f;
        const int row = row0 + warp * R + w, t = row / a.r;
        ipos[w] = i0 + t;
        lse[w] = INFINITY;
        delta[w] = 0.f;
        if (BWD && ACT == kSoftmax && row < nrows) {
            const int64_t at = (int64_t)(tok + t) * a.H + pc.hk * a.r + (row - t * a.r);
            const float x = a.lse[at];
            lse[w] = x == -INFINITY ? INFINITY : x;   // a row that sees no key: weights 0
            delta[w] = a.delta[at];
        }
    }
    auto after = [&](int key) { return key + ((dual && (key & 127) == 96) ? kRows + kBN : kRows); };
    auto fetch = [&](int key, float* K) {
        const int n = min(kRows, pc.nk - key);
        const int64_t src = ((int64_t)(pc.k0 + key) * a.Hkv + pc.hk) * a.d, stride = (int64_t)a.Hkv * a.d;
        if constexpr (kTiles == 2) {
            copy_tile(K, ks, kb + src, stride, n, a.d);
            copy_tile(K + kRows * ks, ks, vb + src, stride, n, a.d);
        } else {
            load_tile(K, ks, kb + src, stride, n, a.d);
            load_tile(K + kRows * ks, ks, vb + src, stride, n, a.d);
        }
    };
    int turn = 0;
    const int key_first = dual ? slot * kBN : 0;
    if (kTiles == 2 && key_first < pc.nk) fetch(key_first, KV);
    for (int key = key_first; key < pc.nk; key = after(key)) {
        const int n = min(kRows, pc.nk - key);
        float *K = KV + turn * 2 * kRows * ks, *V = K + kRows * ks;
        if constexpr (kTiles == 2) {
            tile_arrived();
            __syncthreads();   // and the tile before has been read
            turn ^= 1;
            if (after(key) < pc.nk) fetch(after(key), KV + turn * 2 * kRows * ks);
        } else {
            __syncthreads();
            fetch(key, K);
            __syncthreads();
        }
        float s[R], dp[R];
#pragma unroll
        for (int w = 0; w < R; ++w) s[w] = dp[w] = 0.f;
        if constexpr (BWD) {   // 16 columns at a time: dP less delta cancels, so shorter chains of roundings
            for (int c0 = 0; c0 < c4; c0 += 4) {
                float s16[R], dp16[R];
#pragma unroll
                for (int w = 0; w < R; ++w) s16[w] = dp16[w] = 0.f;
                for (int c = c0; c < min(c0 + 4, c4); ++c) {
                    const float4 kv = *reinterpret_cast<const float4*>(K + lane * ks + 4 * c);
                    const float4 vv = *reinterpret_cast<const float4*>(V + lane * ks + 4 * c);
#pragma unroll
                    for (int w = 0; w < R; ++w) {
                        const int at = (warp * R + w) * qs + 4 * c;
                        s16[w] = dot4(kv, *reinterpret_cast<const float4*>(Q + at), s16[w]);
                        dp16[w] = dot4(vv, *reinterpret_cast<const float4*>(DO + at), dp16[w]);
                    }
                }
#pragma unroll
                for (int w = 0; w < R; ++w) {
                    s[w] += s16[w];
                    dp[w] += dp16[w];
                }
            }
        } else {
            for (int c = 0; c < c4; ++c) {
                const float4 kv = *reinterpret_cast<const float4*>(K + lane * ks + 4 * c);
#pragma unroll
                for (int w = 0; w < R; ++w)
                    s[w] = dot4(kv, *reinterpret_cast<const float4*>(Q + (warp * R + w) * qs + 4 * c), s[w]);
            }
        }
        const int jpos = pc.j0 + key + lane;
        __syncwarp();
#pragma unroll
        for (int w = 0; w < R; ++w) {
            bool ok = lane < n;
            if (own && a.windowed) ok = ok && jpos <= ipos[w] && jpos > ipos[w] - a.window;
            const float t = s[w] * a.alpha;
            float out;
            if constexpr (BWD) {
                float p;
                p_ds<ACT>(t, dp[w], lse[w], delta[w], p, out);
                out = ok ? out * a.alpha : 0.f;
            } else if constexpr (ACT == kSoftmax) {
                float top = ok ? t : -INFINITY;
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
                const float mn = fmaxf(m[w], top);
                const float ref = mn == -INFINITY ? 0.f : mn;
                out = ok ? expf(t - ref) : 0.f;
                float sum = out;
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
                const float f = expf(m[w] - ref);   // 0 while m is still -inf
                l[w] = fmaf(l[w], f, sum);
                acc[w].x *= f; acc[w].y *= f; acc[w].z *= f; acc[w].w *= f;
                m[w] = mn;
            } else {
                out = ok ? act_f<ACT, false>(t) : 0.f;
            }
            W[lane * R + w] = out;
        }
        __syncwarp();
        if (g < ng) {
            const float* X = BWD ? K : V;
            for (int j = g; j < n; j += ng) {
                const float4 x = *reinterpret_cast<const float4*>(X + j * ks + 4 * gc);
                float p[R];
                load_weights<R>(p, W + j * R);
#pragma unroll
                for (int w = 0; w < R; ++w) axpy4(acc[w], p[w], x);
            }
        }
    }
#pragma unroll
    for (int w = 0; w < R; ++w) join_lanes(acc[w], lane, g, ng, c4);
    float4* out = reinterpret_cast<float4*>(a.parts) + (int64_t)part * c4;
#pragma unroll
    for (int w = 0; w < R; ++w) {
        const int row = row0 + warp * R + w;
        if (row >= nrows) break;
        if (lane < c4) out[lane * nrows + row] = acc[w];
        if (!BWD && ACT == kSoftmax && lane == 0)   // maximum in base 2, as the merge takes it
            reinterpret_cast<float2*>(a.ml)[(int64_t)part + row] = make_float2(counted(m[w] * kLog2e, l[w]), l[w]);
    }
}

// dK and dV of 32 keys of a unit: every row that sees them, in order.
template <typename E, int ACT>
__global__ void __launch_bounds__(kThreads) simt_keys_kernel(const SimtArgs a) {
    extern __shared__ float sm[];
    const PrefixUnit u = a.units[blockIdx.x];
    const int key0 = blockIdx.y * kRows;
    const int n = min(kRows, u.nk - key0);
    if (n <= 0) return;
    const bool own = u.flags & kPieceOwn;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ks = a.d, qs = a.d + 4;
    float* K = sm;                     // [32][d]
    float* V = K + kRows * ks;
    float* Q = V + kRows * ks;         // [32][d + 4]
    float* DO = Q + kRows * qs;
    float* W = DO + kRows * qs + warp * 2 * kRows * kPer;   // p, ds [32 rows][8 keys]
    float* X = W + kRows * kPer;
    const int64_t src = ((int64_t)(u.k0 + key0) * a.Hkv + u.hk) * a.d, stride = (int64_t)a.Hkv * a.d;
    load_tile(K, ks, (const E*)(own ? a.k : a.kp) + src, stride, n, a.d);
    load_tile(V, ks, (const E*)(own ? a.v : a.vp) + src, stride, n, a.d);
    const int c4 = a.d / 4, ng = 32 / c4, g = lane / c4, gc = lane - g * c4, nrows = u.ntok * a.r;
    float4 gk[kPer], gv[kPer];
#pragma unroll
    for (int w = 0; w < kPer; ++w) gk[w] = gv[w] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int row0 = 0; row0 < nrows; row0 += kRows) {
        __syncthreads();
        load_rows<kRows>(Q, qs, (const E*)a.q, a, u.tok, u.hk, row0, nrows);
        load_rows<kRows>(DO, qs, (const E*)a.d_o, a, u.tok, u.hk, row0, nrows);
        __syncthreads();
        const int row = row0 + lane, t = row / a.r, ipos = u.i0 + t;
        float lse = INFINITY, delta = 0.f;
        if (ACT == kSoftmax && row < nrows) {
            const int64_t at = (int64_t)(u.tok + t) * a.H + u.hk * a.r + (row - t * a.r);
            const float x = a.lse[at];
            lse = x == -INFINITY ? INFINITY : x;
            delta = a.delta[at];
        }
        float s[kPer], dp[kPer];
#pragma unroll
        for (int w = 0; w < kPer; ++w) s[w] = dp[w] = 0.f;
        for (int c0 = 0; c0 < c4; c0 += 4) {
            float s16[kPer], dp16[kPer];
#pragma unroll
            for (int w = 0; w < kPer; ++w) s16[w] = dp16[w] = 0.f;
            for (int c = c0; c < min(c0 + 4, c4); ++c) {
                const float4 qv = *reinterpret_cast<const float4*>(Q + lane * qs + 4 * c);
                const float4 dv = *reinterpret_cast<const float4*>(DO + lane * qs + 4 * c);
#pragma unroll
                for (int w = 0; w < kPer; ++w) {
                    s16[w] = dot4(qv, *reinterpret_cast<const float4*>(K + (warp * kPer + w) * ks + 4 * c), s16[w]);
                    dp16[w] = dot4(dv, *reinterpret_cast<const float4*>(V + (warp * kPer + w) * ks + 4 * c), dp16[w]);
                }
            }
#pragma unroll
            for (int w = 0; w < kPer; ++w) {
                s[w] += s16[w];
                dp[w] += dp16[w];
            }
        }
        __syncwarp();
#pragma unroll
        for (int w = 0; w < kPer; ++w) {
            const int jpos = u.j0 + key0 + warp * kPer + w;
            bool ok = row < nrows && warp * kPer + w < n;
            if (own && a.windowed) ok = ok && jpos <= ipos && jpos > ipos - a.window;
            float p, ds;
            p_ds<ACT>(s[w] * a.alpha, dp[w], lse, delta, p, ds);
            W[lane * kPer + w] = ok ? p : 0.f;
            X[lane * kPer + w] = ok ? ds * a.alpha : 0.f;
        }
        __syncwarp();
        if (g < ng) {
            const int m = min(kRows, nrows - row0);
            for (int i = g; i < m; i += ng) {
                const float4 qv = *reinterpret_cast<const float4*>(Q + i * qs + 4 * gc);
                const float4 dv = *reinterpret_cast<const float4*>(DO + i * qs + 4 * gc);
                float p[kPer], x[kPer];
                load_weights<kPer>(p, W + i * kPer);
                load_weights<kPer>(x, X + i * kPer);
#pragma unroll
                for (int w = 0; w < kPer; ++w) {
                    axpy4(gv[w], p[w], dv);
                    axpy4(gk[w], x[w], qv);
                }
            }
        }
    }
#pragma unroll
    for (int w = 0; w < kPer; ++w) {
        join_lanes(gv[w], lane, g, ng, c4);
        join_lanes(gk[w], lane, g, ng, c4);
    }
    if (lane < c4) {
        const int split = u.flags / kUnitPart;
        E* dk = (E*)(own ? a.dk : a.dkp) + src;
        E* dv = (E*)(own ? a.dv : a.dvp) + src;
#pragma unroll
        for (int w = 0; w < kPer; ++w) {
            const int j = warp * kPer + w;
            if (j >= n) break;
            if (split) {   // one of several ranges of the rows
                float* to = a.unit_parts + ((int64_t)(split - 1) * 2 * kBN + key0 + j) * a.d + 4 * lane;
                st4(to, gv[w]);
                st4(to + (int64_t)kBN * a.d, gk[w]);
                continue;
            }
            st4(dk + j * stride + 4 * lane, gk[w]);
            st4(dv + j * stride + 4 * lane, gv[w]);
        }
    }
}

// dK and dV of 8 keys of a unit whose rows were split, its parts in order.
template <typename E>
__global__ void __launch_bounds__(256) join_kernel(const PrefixUnit* joins, const float* parts, E* dkp, E* dvp,
                                                   E* dk, E* dv, int Hkv, int d) {
    const PrefixUnit u = joins[blockIdx.x];
    const int c4 = d / 4, key0 = blockIdx.y * 8, n = min(8, u.nk - key0);
    grid_wait_previous();
    const bool own = u.flags & kPieceOwn;
    for (int i = threadIdx.x; i < 2 * n * c4; i += blockDim.x) {
        const bool second = i >= n * c4;
        const int x = second ? i - n * c4 : i, key = key0 + x / c4, c = 4 * (x % c4);
        const float* src = parts + ((int64_t)u.tok * 2 * kBN + (second ? kBN : 0) + key) * d + c;
        float4 sum = ld4(src);
#pragma unroll 4
        for (int t = 1; t < u.ntok; ++t) axpy4(sum, 1.f, ld4(src + (int64_t)t * 2 * kBN * d));
        E* to = second ? (own ? dk : dkp) : (own ? dv : dvp);
        st4(to + ((int64_t)(u.k0 + key) * Hkv + u.hk) * d + c, sum);
    }
}

// Join the parts of 8 rows of a tile: a thread per (row, 4 columns).  The
// first kAtOnce layers, usually all, are loaded together before anything is
// known of them; further ones as many at a time, a warp's four threads of a row
// sharing a look at their maxima.  Few registers, so that many blocks hide the
// chain of loads (tile, token, layers) of each other.
template <typename E, int kAtOnce>
__global__ void __launch_bounds__(256, kAtOnce > 4 ? 2 : 4) merge_kernel(const PrefixTile* tiles, const PrefixOwn* owns,
                                                    const float* parts, const float* ml, E* out,
                                                    float* lse, int H, int r, int d, int softmax) {
    const PrefixTile t = tiles[blockIdx.x];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nrows = t.n * r, row = blockIdx.y * 8 + (lane & 7);
    if (blockIdx.y * 8 >= nrows) return;
    const bool real = row < nrows;
    const int tl = real ? row / r : 0, j = row - tl * r, tok = t.tok + tl;
    int4 own4 = make_int4(0, 0, 0, 0);
    if (real) own4 = __ldg(reinterpret_cast<const int4*>(owns + tok));
    const PrefixOwn ow = {own4.x, own4.y, own4.z, own4.w};
    const int orow = ow.row0 + j, total = real ? t.layers + ow.layers : 0;
    const int64_t own0 = (int64_t)ow.part + (int64_t)t.hk * ow.layers * ow.rows;
    const float2* st = reinterpret_cast<const float2*>(ml);
    const float4* src = reinterpret_cast<const float4*>(parts);
    const int c4 = d / 4, c = (lane >> 3) + 4 * warp;
    // layer x: its first row in the workspace, its rows, this row's place
    auto place = [&](int x, int& n, int& at) {
        const bool pre = x < t.layers;
        n = pre ? nrows : ow.rows;
        at = pre ? row : orow;
        return pre ? (int64_t)t.part + (int64_t)x * nrows : own0 + (int64_t)(x - t.layers) * ow.rows;
    };
    float2 s[kAtOnce];
    float4 v[kAtOnce];
    auto load = [&](int x0) {
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            s[u] = make_float2(-INFINITY, 0.f);
            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (x0 + u < total && c < c4) {
                int n, at;
                const int64_t p = place(x0 + u, n, at);
                if (softmax) s[u] = st[p + at];
                v[u] = src[p * c4 + (int64_t)c * n + at];
            }
        }
    };
    grid_wait_previous();
    load(0);
    float top = -INFINITY, ref = 0.f, sum = 0.f;
    if (softmax) {
#pragma unroll 4
        for (int x = kAtOnce + (lane >> 3); x < total; x += 4) {
            int n, at;
            const int64_t p = place(x, n, at);
            top = fmaxf(top, st[p + at].x);
        }
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) top = fmaxf(top, s[u].x);
        ref = top == -INFINITY ? 0.f : top;
    }
    if (!real || c >= c4) return;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x0 = 0; x0 < total; x0 += kAtOnce) {
        if (x0 > 0) load(x0);
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            float w = 1.f;
            if (softmax) {
                if (s[u].x == -INFINITY) continue;   // no such layer, or nothing visible in it
                w = exp2f(s[u].x - ref);
                sum = fmaf(w, s[u].y, sum);
            }
            axpy4(acc, w, v[u]);
        }
    }
    const float inv = !softmax ? 1.f : sum == 0.f ? 0.f : 1.f / sum;   // (a NaN stays one)
    const int64_t at = (int64_t)tok * H + t.hk * r + j;
    st4(out + at * d + 4 * c, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    if (softmax && lse && c == 0)
        lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994530942f;
}

// delta = dO . O of every row, a warp a row
template <typename E>
__global__ void __launch_bounds__(256) delta_kernel(const E* d_o, const E* o, float* delta,
                                                    int64_t rows, int d) {
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int lane = threadIdx.x & 31;
    float s = 0.f;
    if (4 * lane < d) s = dot4(ld4(d_o + row * d + 4 * lane), ld4(o + row * d + 4 * lane), 0.f);
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
    if (lane == 0) delta[row] = s;
}

SimtArgs args_of(const PrefixPlan& p, const PrefixIO& io, const float* delta) {
    SimtArgs a;
    a.pieces = p.dev_pieces();
    a.blocks = p.dev_blocks();
    a.units = p.dev_units();
    a.q = io.q; a.kp = io.kp; a.vp = io.vp; a.k = io.k; a.v = io.v;
    a.d_o = io.d_o;
    a.lse = io.lse;
    a.delta = delta;
    a.parts = p.d_parts;
    a.ml = p.d_ml;
    a.dkp = io.dkp; a.dvp = io.dvp; a.dk = io.dk; a.dv = io.dv;
    a.unit_parts = p.d_grad;
    a.H = p.H; a.Hkv = p.Hkv; a.r = p.r; a.d = p.d;
    a.windowed = p.mask == GDPA_MASK_CAUSAL_WINDOW;
    a.window = p.window;
    a.alpha = io.alpha;
    return a;
}

template <auto kKern>
gdpa_status go(dim3 grid, int smem, PrefixPlan& p, const SimtArgs& a, cudaStream_t st) {
    // the most any kernel takes, at d = 128: dK and dV, or dQ with 2 rows a warp
    constexpr int kKeysMost = (2 * kRows * 128 + 2 * kRows * 132 + 8 * kRows * kPer) * 4;
    constexpr int kRowsMost = (2 * 8 * 128 + 4 * kRows * 132 + 4 * kRows * 2) * 4;
    constexpr int kMost = kKeysMost > kRowsMost ? kKeysMost : kRowsMost;
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(kKern, kMost, p.device, done)) return GDPA_ERR_CUDA;
    kKern<<<grid, kThreads, smem, st>>>(a);
    p.launches += 1;
    return cudaGetLastError() == cudaSuccess ? GDPA_OK : GDPA_ERR_CUDA;
}

#define PREFIX_DISPATCH(act, ...)                                         \
    if ((act) == kSoftmax) { constexpr int A = kSoftmax; __VA_ARGS__; }   \
    else GDPA_DISPATCH_ACT(act, A, __VA_ARGS__)

template <typename E, bool BWD, int R>
gdpa_status rows_t(PrefixPlan& p, int act, const SimtArgs& a, cudaStream_t st) {
    gdpa_status s = GDPA_OK;
    const int tiles = sizeof(E) == 4 && R == 2 ? 2 : 1;
    const int smem = ((BWD ? 2 : 1) * 4 * R * p.d + tiles * 2 * kRows * (p.d + 4) + 4 * kRows * R) * 4;
    const dim3 grid((unsigned)p.blocks.size());
    PREFIX_DISPATCH(act, s = (go<simt_rows_kernel<E, A, BWD, R>>(grid, smem, p, a, st)))
    return s;
}

template <typename E, bool BWD>
gdpa_status rows_of(PrefixPlan& p, int act, const SimtArgs& a, cudaStream_t st) {
    if (p.blocks.empty()) return GDPA_OK;
    return p.warp_rows == 2 ? rows_t<E, BWD, 2>(p, act, a, st) : rows_t<E, BWD, kPer>(p, act, a, st);
}

template <typename E>
gdpa_status fwd_t(PrefixPlan& p, const PrefixIO& io, cudaStream_t st) {
    return rows_of<E, false>(p, io.act, args_of(p, io, nullptr), st);
}

template <typename E>
gdpa_status bwd_t(PrefixPlan& p, const PrefixIO& io, const float* delta, cudaStream_t st) {
    const SimtArgs a = args_of(p, io, delta);
    gdpa_status s = rows_of<E, true>(p, io.act, a, st);
    if (s == GDPA_OK && !p.units.empty()) {
        const int smem = (2 * kRows * p.d + 2 * kRows * (p.d + 4) + 8 * kRows * kPer) * 4;
        const dim3 grid((unsigned)p.units.size(), 4);
        PREFIX_DISPATCH(io.act, s = (go<simt_keys_kernel<E, A>>(grid, smem, p, a, st)))
    }
    return s;
}

}  // namespace

gdpa_status launch_prefix_simt_fwd(PrefixPlan& p, gdpa_dtype dt, const PrefixIO& io, cudaStream_t st) {
    return dt == GDPA_BF16 ? fwd_t<__nv_bfloat16>(p, io, st) : fwd_t<float>(p, io, st);
}

gdpa_status launch_prefix_simt_bwd(PrefixPlan& p, gdpa_dtype dt, const PrefixIO& io,
                                   const float* delta, cudaStream_t st) {
    return dt == GDPA_BF16 ? bwd_t<__nv_bfloat16>(p, io, delta, st) : bwd_t<float>(p, io, delta, st);
}

gdpa_status launch_prefix_join(PrefixPlan& p, gdpa_dtype dt, const PrefixIO& io, cudaStream_t st) {
    if (p.joins.empty()) return GDPA_OK;
    const dim3 grid((unsigned)p.joins.size(), kBN / 8);
    const bool early = p.chain > 0;
    const float* parts = p.d_grad;
    auto go = [&](auto* t) {
        using E = std::remove_pointer_t<decltype(t)>;
        return launch_kernel(join_kernel<E>, grid, 256, 0, st, early, p.dev_joins(), parts, (E*)io.dkp, (E*)io.dvp,
                             (E*)io.dk, (E*)io.dv, p.Hkv, p.d);
    };
    const bool ok = dt == GDPA_BF16 ? go((__nv_bfloat16*)nullptr) : go((float*)nullptr);
    p.launches += 1;
    p.chain += 1;
    return ok ? GDPA_OK : GDPA_ERR_CUDA;
}

gdpa_status launch_prefix_merge(PrefixPlan& p, gdpa_dtype dt, void* out, float* lse, bool softmax,
                                cudaStream_t st) {
    if (p.tiles.empty()) return GDPA_OK;
    const dim3 grid((unsigned)p.tiles.size(), kBM / 8);
    const int threads = p.d > 64 ? 256 : 128;   // a warp has 16 columns of 8 rows
    const float *parts = p.d_parts, *ml = p.d_ml;
    const bool early = p.chain > 0;
    const int sm = softmax;
    auto go = [&](auto* o, auto kern) {
        return launch_kernel(kern, grid, threads, 0, st, early, p.dev_tiles(), p.dev_own(), parts, ml, o, lse, p.H,
                             p.r, p.d, sm);
    };
    using B = __nv_bfloat16;
    // few row tiles of many layers (a decoding step): rounds of 12 loads, where
    // they leave room for all blocks at once (38 layers of 4 tiles: 9 us, 13 with
    // 4; up to 10 layers of 122 tiles 16 and 12)
    const bool deep = p.max_layers > 8 && (int64_t)grid.x * grid.y <= 2 * p.S;
    const bool ok = dt == GDPA_BF16 ? (deep ? go((B*)out, merge_kernel<B, 12>) : go((B*)out, merge_kernel<B, 4>))
                    : deep          ? go((float*)out, merge_kernel<float, 12>)
                                    : go((float*)out, merge_kernel<float, 4>);
    p.launches += 1;
    return ok ? GDPA_OK : GDPA_ERR_CUDA;
}

gdpa_status launch_prefix_delta(PrefixPlan& p, gdpa_dtype dt, const PrefixIO& io, float* delta,
                                cudaStream_t st) {
    const int64_t rows = p.Tq * p.H;
    if (rows == 0) return GDPA_OK;
    const int64_t blocks = (rows + 7) / 8;
    if (blocks > 0x7fffffff) return GDPA_ERR_UNSUPPORTED;
    if (dt == GDPA_BF16)
        delta_kernel<<<(unsigned)blocks, 256, 0, st>>>((const __nv_bfloat16*)io.d_o,
                                                       (const __nv_bfloat16*)io.o, delta, rows, p.d);
    else
        delta_kernel<<<(unsigned)blocks, 256, 0, st>>>((const float*)io.d_o, (const float*)io.o,
                                                       delta, rows, p.d);
    p.launches += 1;
    return cudaGetLastError() == cudaSuccess ? GDPA_OK : GDPA_ERR_CUDA;
}

}  // namespace gdpa
