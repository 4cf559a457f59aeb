// Attention over the history cache on the CUDA cores for up to 4 query rows a key
// head: a new event of float32 rows, or of a head dim that the tensor-core kernels
// do not take.
//
// With so few rows a cached byte meets a handful of products, so what bounds the
// kernel is reading the cache once.  Neighbouring lanes hold the 16-byte chunks of
// one event's row (32 lanes, or 2, 4, .. events side by side), load straight from
// the pages, multiply with their columns of the queries in registers and add up
// over the event's lanes.  Each run of lanes keeps a softmax of its own over the
// events that it took; they are joined at the end of a segment.  Four events a
// lane are on their way at a time, and two to four CTAs an SM.  (512 users' newest events
// on 3 GB of float32 rows: 620 us, 4.8 TB/s; 3199 by the kernel for 16 rows a warp.)
#include "cache_attn.cuh"

namespace gdpa {
namespace {

constexpr int kThreads = 128, kAhead = 4;

template <typename E, int STORE, bool SM, int R>
__global__ void __launch_bounds__(kThreads, cache_few_per_sm(STORE, R))
cache_few_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int N = cache_per_chunk(STORE);
    __shared__ int64_t scan_tmp[kThreads / 32 + 2];
    __shared__ float2 ml[4][4];
    __shared__ __align__(16) float sums[4][R][132];
    const int chunks = a.c.row / 16;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int lanes = 1, shift = 0;                        // of an event: chunks, rounded up to a power of two
    while (lanes < chunks) lanes *= 2, ++shift;
    const int c = lane & (lanes - 1), ev = lane >> shift, events = 32 >> shift;
    asm volatile("griddepcontrol.launch_dependents;");
    if (tid == 0) a.desc[blockIdx.x].parts = 0;
    Share sh = find_share<kThreads>(a, scan_tmp);
    while (sh.more()) {
        const Segment g = next_segment(a, sh);
        if (g.rows == 0) break;
        float q[R][N], o[R][N], m[R], l[R], lost[R];
        RowView rv[R];
        int hi_min = 0x7fffffff, lo_max = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            rv[r] = row_view(a, g, r);
            m[r] = -INFINITY;
            l[r] = lost[r] = 0.0f;
            const int rho = g.rho0 + r, tok = max(rv[r].tok, 0);
            const E* src = (const E*)a.q + (g.s.t0 + tok) * a.qt + (g.h * a.G + rho - tok * a.G) * a.qh + c * N;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                q[r][i] = rv[r].tok >= 0 && c < chunks ? to_f(src[i]) : 0.0f;
                o[r][i] = 0.0f;
            }
            if (rv[r].tok >= 0) {
                hi_min = min(hi_min, rv[r].hi);
                lo_max = max(lo_max, rv[r].lo);
            }
        }
        for (int i = warp; i < g.n; i += 4) {
            const int e0 = segment_group(g, i) * kCacheGroup;
            const int64_t blk = cache_block(a.c, a.w, g.b, e0, g.h);
            if (blk < 0) continue;                   // (the whole warp)
            const int in = e0 & ((1 << a.c.page_log) - 1);
            const uint8_t *kp = a.c.k + blk * a.c.block, *vp = a.c.v + blk * a.c.block;
            uint32_t bits[R];
            const bool masked = !(e0 + 16 <= hi_min && (e0 >= lo_max || e0 + 16 <= a.sinks));
#pragma unroll
            for (int r = 0; r < R; ++r) bits[r] = masked ? row_bits(a, g, rv[r], e0) : 0xffffu;
            for (int b0 = 0; b0 < 16; b0 += kAhead * events) {
                uint4 kq[kAhead], vq[kAhead];
                float ks[kAhead], vs[kAhead];
#pragma unroll
                for (int p = 0; p < kAhead; ++p) {
                    const int e = b0 + p * events + ev;
                    kq[p] = vq[p] = make_uint4(0, 0, 0, 0);
                    ks[p] = vs[p] = 1.0f;
                    if (e < 16 && c < chunks) {
                        const int at = cache_chunk(a.c.row, a.c.page_log, in + e, c);
                        kq[p] = __ldg(reinterpret_cast<const uint4*>(kp + at));
                        vq[p] = __ldg(reinterpret_cast<const uint4*>(vp + at));
                        if constexpr (STORE == GDPA_STORE_E4M3) {
                            ks[p] = cache_scale(a.c.ks[(blk << a.c.page_log) + in + e]);
                            vs[p] = cache_scale(a.c.vs[(blk << a.c.page_log) + in + e]);
                        }
                    }
                }
                float s[R][kAhead];
#pragma unroll
                for (int p = 0; p < kAhead; ++p) {
                    float x[N];
                    expand<STORE>(kq[p], x);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        float y = 0.0f;
#pragma unroll
                        for (int j = 0; j < N; ++j) y = fmaf(q[r][j], x[j], y);
                        s[r][p] = y * ks[p];         // (lanes of an event have the same power of two, or zeros)
                    }
                }
                for (int k = 1; k < lanes; k <<= 1)
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int p = 0; p < kAhead; ++p) s[r][p] += __shfl_xor_sync(0xffffffffu, s[r][p], k);
                const auto sees = [&](int r, int p) {
                    const int e = b0 + p * events + ev;
                    return e < 16 && (bits[r] >> e & 1u);
                };
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if constexpr (SM) {
                        float top = m[r];
#pragma unroll
                        for (int p = 0; p < kAhead; ++p) {
                            s[r][p] = sees(r, p) ? s[r][p] * a.alpha : -INFINITY;
                            top = fmaxf(top, s[r][p]);
                        }
                        if (top > m[r]) {
                            const float f = m[r] == -INFINITY ? 0.0f : expf(m[r] - top);
                            m[r] = top;
                            l[r] *= f;
                            lost[r] *= f;
#pragma unroll
                            for (int j = 0; j < N; ++j) o[r][j] *= f;
                        }
                        const float ref = m[r] == -INFINITY ? 0.0f : m[r];
                        float sum = 0.0f;
#pragma unroll
                        for (int p = 0; p < kAhead; ++p) {
                            s[r][p] = expf(s[r][p] - ref);
                            sum += s[r][p];
                        }
                        add_compensated(l[r], lost[r], sum);
                    } else {
#pragma unroll
                        for (int p = 0; p < kAhead; ++p) {
                            float w = s[r][p] * a.alpha;
                            switch (a.act) {
                                case kGeluErf: w = act_f<kGeluErf, false>(w); break;
                                case kGeluTanh: w = act_f<kGeluTanh, false>(w); break;
                                case kSilu: w = act_f<kSilu, false>(w); break;
                                case kTaylor6: w = act_f<kTaylor6, false>(w); break;
                                default: break;
                            }
                            s[r][p] = w;
                        }
                    }
                }
                if constexpr (STORE == GDPA_STORE_E4M3) {
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int p = 0; p < kAhead; ++p) s[r][p] *= vs[p];
                }
                if (!masked) {
                    // the events of a step among themselves first: O is rounded once for them
                    // (events that there are not: weights and values of 0)
                    constexpr int V = N / 4;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float x[kAhead][V];
#pragma unroll
                        for (int p = 0; p < kAhead; ++p) expand_word<STORE>((&vq[p].x)[i], x[p]);
#pragma unroll
                        for (int r = 0; r < R; ++r)
#pragma unroll
                            for (int j = 0; j < V; ++j) {
                                float y = s[r][0] * x[0][j];
#pragma unroll
                                for (int p = 1; p < kAhead; ++p) y = fmaf(s[r][p], x[p][j], y);
                                o[r][V * i + j] += y;
                            }
                    }
                    continue;
                }
#pragma unroll
                for (int p = 0; p < kAhead; ++p) {
                    float x[N];
                    expand<STORE>(vq[p], x);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        if (!sees(r, p)) continue;   // whatever a hidden event holds
#pragma unroll
                        for (int j = 0; j < N; ++j) o[r][j] = fmaf(s[r][p], x[j], o[r][j]);
                    }
                }
            }
        }
        // the runs of lanes of this warp, then the warps
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float f = 1.0f;
            if constexpr (SM) {
                float top = m[r];
                for (int k = lanes; k < 32; k <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
                // (no events, or NaNs alone: its sum is 0 or NaN)
                f = m[r] == -INFINITY ? 1.0f : expf(m[r] - top);
                m[r] = top;
                l[r] *= f;
                for (int k = lanes; k < 32; k <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], k);
                if (lane == 0) ml[warp][r] = make_float2(m[r] * kLog2e, l[r]);
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                float y = o[r][j] * f;
                for (int k = lanes; k < 32; k <<= 1) y += __shfl_xor_sync(0xffffffffu, y, k);
                if (lane < chunks) sums[warp][r][c * N + j] = y;
            }
        }
        __syncthreads();
        finish_segment<E, SM, kThreads>(
            a, g, 4, [&](int w, int x, int k) { return reinterpret_cast<const float4*>(&sums[w][x][k]); },
            [&](int w, int x) { return ml[w][x]; });
        __syncthreads();
    }
}

template <typename E, int STORE, int R>
gdpa_status launch(const AttnArgs& a, int grid, cudaStream_t st) {
    if (a.act == kSoftmax) cache_few_kernel<E, STORE, true, R><<<grid, kThreads, 0, st>>>(a);
    else cache_few_kernel<E, STORE, false, R><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? GDPA_OK : GDPA_ERR_CUDA;
}

template <typename E, int STORE>
gdpa_status launch_rows(const AttnArgs& a, int grid, cudaStream_t st) {
    return a.TM == 1 ? launch<E, STORE, 1>(a, grid, st) : a.TM == 2 ? launch<E, STORE, 2>(a, grid, st) : launch<E, STORE, 4>(a, grid, st);
}

}  // namespace

gdpa_status launch_cache_few(const AttnArgs& a, gdpa_dtype dt, int grid, cudaStream_t st) {
    if (dt == GDPA_F32)
        return a.c.store == GDPA_STORE_E4M3 ? launch_rows<float, GDPA_STORE_E4M3>(a, grid, st)
                                            : launch_rows<float, GDPA_STORE_F32>(a, grid, st);
    return a.c.store == GDPA_STORE_E4M3 ? launch_rows<__nv_bfloat16, GDPA_STORE_E4M3>(a, grid, st)
                                        : launch_rows<__nv_bfloat16, GDPA_STORE_BF16>(a, grid, st);
}

}  // namespace gdpa
