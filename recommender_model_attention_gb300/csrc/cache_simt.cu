// Attention over the history cache on the CUDA cores: float32 rows, and head
// dims that the tensor-core kernel does not take.
//
// The same shares, segments and masks; a CTA's four warps take turns over the
// groups of 16 events.  A warp expands a group to float32 in shared memory, a
// lane makes the scores of one row with 8 of the events and then the row's sums
// of every second 4 columns: 4 products a value read from shared memory.  What
// bounds it is that traffic and the latency of a group; these are the small
// float32 configurations, not the serving path.
#include "cache_attn.cuh"

namespace gdpa {
namespace {

constexpr int kThreads = 128;

// 16 bytes of a cache row as float32 values
template <int STORE>
__device__ __forceinline__ void expand_to(float* dst, const uint4& q, float scale) {
    constexpr int N = cache_per_chunk(STORE);
    float x[N];
    expand<STORE>(q, x);
#pragma unroll
    for (int i = 0; i < N; ++i) dst[i] = STORE == GDPA_STORE_E4M3 ? x[i] * scale : x[i];
}

template <typename E, int STORE, bool SM>
__global__ void __launch_bounds__(kThreads)
cache_simt_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int kPer = cache_per_chunk(STORE);   // values a chunk
    extern __shared__ __align__(16) float fsm[];
    __shared__ int64_t scan_tmp[kThreads / 32 + 2];
    __shared__ float wsm[4][16][17];
    __shared__ float2 ml[4][16];
    const int d = a.c.d, d4 = d / 4, ld = d + 4;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane & 15, half = lane >> 4;
    float* Q = fsm;                                  // [16][ld]
    float* K = fsm + (1 + 2 * warp) * 16 * ld;       // this warp's keys, and its sums at the end
    float* V = K + 16 * ld;
    asm volatile("griddepcontrol.launch_dependents;");
    if (tid == 0) a.desc[blockIdx.x].parts = 0;
    Share sh = find_share<kThreads>(a, scan_tmp);
    while (sh.more()) {
        const Segment g = next_segment(a, sh);
        if (g.rows == 0) break;
        for (int i = tid; i < 16 * d; i += kThreads) {
            const int x = i / d, c = i - x * d, rho = g.rho0 + x, tok = rho / a.G;
            Q[x * ld + c] = x < g.rows ? to_f(((const E*)a.q)[(g.s.t0 + tok) * a.qt + (g.h * a.G + rho - tok * a.G) * a.qh + c]) : 0.0f;
        }
        const RowView rv = row_view(a, g, r);
        __syncthreads();
        float o[16][4];
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        float m = -INFINITY, l = 0.0f, lost = 0.0f;
        for (int i = warp; i < g.n; i += 4) {
            const int e0 = segment_group(g, i) * kCacheGroup;
            const int64_t blk = cache_block(a.c, a.w, g.b, e0, g.h);
            if (blk < 0) continue;                   // (the whole warp)
            const int in = e0 & ((1 << a.c.page_log) - 1), chunks = a.c.row / 16;
            for (int j = lane; j < 16 * chunks; j += 32) {
                const int e = j / chunks, c = j - e * chunks;
                const int at = cache_chunk(a.c.row, a.c.page_log, in + e, c);
                float sk = 1.0f, sv = 1.0f;
                if (STORE == GDPA_STORE_E4M3) {
                    sk = cache_scale(a.c.ks[(blk << a.c.page_log) + in + e]);
                    sv = cache_scale(a.c.vs[(blk << a.c.page_log) + in + e]);
                }
                expand_to<STORE>(K + e * ld + c * kPer, *reinterpret_cast<const uint4*>(a.c.k + blk * a.c.block + at), sk);
                expand_to<STORE>(V + e * ld + c * kPer, *reinterpret_cast<const uint4*>(a.c.v + blk * a.c.block + at), sv);
            }
            __syncwarp();
            float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            for (int c = 0; c < d4; ++c) {
                const float4 q = *reinterpret_cast<const float4*>(Q + r * ld + 4 * c);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 k = *reinterpret_cast<const float4*>(K + (8 * half + j) * ld + 4 * c);
                    s[j] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s[j]))));
                }
            }
            const uint32_t bits = row_bits(a, g, rv, e0);
            float f = 1.0f;
            if constexpr (SM) {
                float mt = m;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s[j] = (bits >> (8 * half + j) & 1u) ? s[j] * a.alpha : -INFINITY;
                    mt = fmaxf(mt, s[j]);
                }
                mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
                f = m == -INFINITY ? 0.0f : expf(m - mt);
                m = mt;
                const float ref = m == -INFINITY ? 0.0f : m;
                l *= f;
                lost *= f;
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s[j] = expf(s[j] - ref);
                    sum += s[j];
                }
                add_compensated(l, lost, sum);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float w = s[j] * a.alpha;
                    switch (a.act) {
                        case kGeluErf: w = act_f<kGeluErf, false>(w); break;
                        case kGeluTanh: w = act_f<kGeluTanh, false>(w); break;
                        case kSilu: w = act_f<kSilu, false>(w); break;
                        case kTaylor6: w = act_f<kTaylor6, false>(w); break;
                        default: break;
                    }
                    s[j] = w;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) wsm[warp][r][8 * half + j] = s[j];
            __syncwarp();
            if (f != 1.0f) {
#pragma unroll
                for (int x = 0; x < 16; ++x)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[x][j] *= f;
            }
            if (__all_sync(0xffffffffu, bits == 0xffffu || r >= g.rows)) {
                // the group's events among themselves first: O is rounded once for them
                float w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = wsm[warp][r][e];
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const int c = 2 * x + half;
                    if (c >= d4) break;
                    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float4 v = *reinterpret_cast<const float4*>(V + e * ld + 4 * c);
                        y[0] = fmaf(w[e], v.x, y[0]);
                        y[1] = fmaf(w[e], v.y, y[1]);
                        y[2] = fmaf(w[e], v.z, y[2]);
                        y[3] = fmaf(w[e], v.w, y[3]);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[x][j] += y[j];
                }
                __syncwarp();
                continue;
            }
            for (int e = 0; e < 16; ++e) {
                if (!(bits >> e & 1u)) continue;     // whatever a hidden event holds
                const float w = wsm[warp][r][e];
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const int c = 2 * x + half;
                    if (c < d4) {
                        const float4 v = *reinterpret_cast<const float4*>(V + e * ld + 4 * c);
                        o[x][0] = fmaf(w, v.x, o[x][0]);
                        o[x][1] = fmaf(w, v.y, o[x][1]);
                        o[x][2] = fmaf(w, v.z, o[x][2]);
                        o[x][3] = fmaf(w, v.w, o[x][3]);
                    }
                }
            }
            __syncwarp();
        }
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (half == 0) ml[warp][r] = make_float2(m * kLog2e, l);
#pragma unroll
        for (int x = 0; x < 16; ++x) {
            const int c = 2 * x + half;
            if (c < d4) put4(K + r * ld + 4 * c, o[x]);
        }
        __syncthreads();
        finish_segment<E, SM, kThreads>(
            a, g, 4,
            [&](int w, int x, int c) { return reinterpret_cast<const float4*>(fsm + ((1 + 2 * w) * 16 + x) * ld + c); },
            [&](int w, int x) { return ml[w][x]; });
        __syncthreads();
    }
}

template <typename E, int STORE, bool SM>
gdpa_status launch(const AttnArgs& a, int grid, cudaStream_t st) {
    const int bytes = 9 * 16 * (a.c.d + 4) * 4;
    static std::atomic<uint64_t> done{0};
    if (!cache_smem((const void*)cache_simt_kernel<E, STORE, SM>, 9 * 16 * 132 * 4, done)) return GDPA_ERR_CUDA;
    cache_simt_kernel<E, STORE, SM><<<grid, kThreads, bytes, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? GDPA_OK : GDPA_ERR_CUDA;
}

template <typename E, int STORE>
gdpa_status launch_act(const AttnArgs& a, int grid, cudaStream_t st) {
    return a.act == kSoftmax ? launch<E, STORE, true>(a, grid, st) : launch<E, STORE, false>(a, grid, st);
}

}  // namespace

gdpa_status launch_cache_simt(const AttnArgs& a, gdpa_dtype dt, int grid, cudaStream_t st) {
    if (dt == GDPA_F32)
        return a.c.store == GDPA_STORE_E4M3 ? launch_act<float, GDPA_STORE_E4M3>(a, grid, st)
                                            : launch_act<float, GDPA_STORE_F32>(a, grid, st);
    return a.c.store == GDPA_STORE_E4M3 ? launch_act<__nv_bfloat16, GDPA_STORE_E4M3>(a, grid, st)
                                        : launch_act<__nv_bfloat16, GDPA_STORE_BF16>(a, grid, st);
}

}  // namespace gdpa
