// The warp-level products of the history cache's attention: a stage (one or two
// groups of 16 events) in shared memory against one warp's query rows, for up to
// 16 rows (Rows16) and up to 8 (Rows8).
//
// Rows16: rows are the m of m16n8k16, S = Q K^T and O += P V; the scores a thread
// gets are the A operand of the second product as they are.
// Rows8: events, then columns of d, are the m: S^T = K Q^T, O^T += V^T P^T.  Half
// the products and a quarter of the scores a thread for the same operands from
// shared memory; the weights are turned by movmatrix between the two.
// In both a thread's 16 bytes of a key row are operands of 2 (8-bit: 4) steps of
// the contraction, whose order over d is free as long as Q has the same, and two
// value rows' bytes interleaved are operands of the second product, each thread's
// part of O being runs of d.
#pragma once

#include "cache_attn.cuh"
#include "tc_common.cuh"

namespace gdpa {
namespace cache_mma {

using namespace tc;

constexpr int kThreads = 128;

template <int D, bool FP8, bool R8>
struct Cfg {
    static constexpr int kRow = FP8 ? D : 2 * D;            // bytes of a cache row
    static constexpr int kCols = kRow >= 128 ? kRow / 128 : 1;
    static constexpr int kKeys = 16 * kRow;                 // bytes of a group's K (or V)
    static constexpr int kScales = FP8 ? 32 : 0;            // ... of its scales
    // groups of a ring's stage, taken together: the more, the more independent
    // products and the fewer waits and votes a byte; bf16 rows of 128 leave no
    // room for two
    static constexpr int kTake = FP8 || D == 64 ? 2 : 1;
    static constexpr int kPerSm = R8 ? 3 : 2;
    static constexpr int kStage = kTake * 2 * kKeys;
    static constexpr int kRing = kStage == 4096 ? 16 : R8 ? 8 : 12;   // stages of all rings
    // sums of a row in shared memory: runs of d a thread holds, padded so that
    // neither rows nor runs meet a bank twice
    static constexpr int kOwn = R8 ? (FP8 && D == 128 ? 16 : 8) : (FP8 && D == 128 ? 32 : 16);
    static constexpr int kSkip = R8 ? 4 : 8;
    static constexpr int kRowLen = D + kSkip * (D / kOwn) + 4;
    static constexpr int kRows = R8 ? 8 : 16;
    static constexpr int kSums = 4 * kRows * kRowLen * 4;
    static constexpr int kMain = kRing * kStage > kSums ? kRing * kStage : kSums;
    static constexpr int kBytes = kMain + kRing * kTake * kScales;
    __device__ static __forceinline__ int sum_at(int r, int c) { return r * kRowLen + c + kSkip * (c / kOwn); }
};

// first of the 4 columns of step s of the contraction over d, of a thread with t = lane & 3
template <int D, bool FP8>
__device__ __forceinline__ int step_col(int t, int s) {
    if constexpr (FP8 && D == 128) return 32 * t + 4 * s;
    return 64 * (s >> 2) + 16 * t + 4 * (s & 3);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <bool FP8>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (FP8) mma_f16(c, a[0], a[1], a[2], a[3], b0, b1);
    else mma_bf16(c, a[0], a[1], a[2], a[3], b0, b1);
}

// two E4M3 codes (the low or the high half of w) as f16 values
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
    uint32_t h;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(w));
    return h;
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
    uint32_t h;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(h) : "r"(w));
    return h;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// all bits of those of the packed bf16 pair / 8-bit codes that are infinities or NaNs
template <bool FP8>
__device__ __forceinline__ uint32_t odd_bits(uint32_t w) {
    if constexpr (FP8) return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
    return __vcmpeq2(w & 0x7f807f80u, 0x7f807f80u);
}


// where the 16-byte piece c (of those that a thread with this t takes) of event e's keys lies in a group
template <int D, bool FP8>
__device__ __forceinline__ uint4 key_piece(const uint8_t* kp, int e, int t, int c) {
    if constexpr (FP8 && D == 64)
        return *reinterpret_cast<const uint4*>(kp + e * 64 + ((t ^ ((e >> 1) & 3)) << 4));
    else
        return *reinterpret_cast<const uint4*>(kp + (c >> 1) * 2048 + e * 128 + (((2 * t + (c & 1)) ^ (e & 7)) << 4));
}

// a thread's words of event e's values: 16 bytes (8-bit, 64 columns: 8) a column of the layout
template <int D, bool FP8, int VW>
__device__ __forceinline__ void value_words(const uint8_t* vp, int e, int gq, uint32_t (&v)[VW]) {
    if constexpr (FP8 && D == 128) {
        *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(vp + e * 128 + ((gq ^ (e & 7)) << 4));
    } else if constexpr (FP8) {
        *reinterpret_cast<uint2*>(v) = *reinterpret_cast<const uint2*>(
            vp + e * 64 + (((gq >> 1) ^ ((e >> 1) & 3)) << 4) + 8 * (gq & 1));
    } else {
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
            *reinterpret_cast<uint4*>(v + 4 * c) = *reinterpret_cast<const uint4*>(vp + c * 2048 + e * 128 + ((gq ^ (e & 7)) << 4));
    }
}

// a value of event e in a group (for what is left out of the products)
template <int D, bool FP8>
__device__ __forceinline__ float value_at(const uint8_t* vp, int e, int col) {
    if constexpr (FP8) {
        const uint32_t h = codes_lo(vp[cache_chunk(D, 4, e, col >> 4) + (col & 15)]);
        return __half2float(__ushort_as_half((uint16_t)h));
    } else {
        return __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(vp + cache_chunk(2 * D, 4, e, col >> 3) + 2 * (col & 7)));
    }
}

// Row r of a tile: the pieces of it that a thread with this t multiplies, two
// words a step.
template <int D, bool FP8>
__device__ __forceinline__ void load_query(const AttnArgs& a, const Segment& g, int r, int tok, int t, uint32_t (&w)[D / 16][2]) {
    const int rho = g.rho0 + r, at = max(tok, 0);
    const __nv_bfloat16* src = (const __nv_bfloat16*)a.q + (g.s.t0 + at) * a.qt + (g.h * a.G + rho - at * a.G) * a.qh;
#pragma unroll
    for (int s = 0; s < D / 16; s += 2) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (tok >= 0) {
            const __nv_bfloat16* p = src + step_col<D, FP8>(t, s);
            if (a.q_wide) {
                v = __ldg(reinterpret_cast<const uint4*>(p));
            } else {
                const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
                uint32_t* o = &v.x;
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = h[2 * j] | (uint32_t)h[2 * j + 1] << 16;
            }
        }
        w[s][0] = v.x;
        w[s][1] = v.y;
        w[s + 1][0] = v.z;
        w[s + 1][1] = v.w;
    }
}

// The same for 8-bit keys: f16 values of the row times a power of two that brings
// its largest to [1, 2).  Returns the factor that undoes it.
template <int STEPS>
__device__ __forceinline__ float scale_query(uint32_t (&w)[STEPS][2]) {
    float top = 0.0f;
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int j = 0; j < 2; ++j) top = fmaxf(top, fmaxf(fabsf(bf16_lo(w[s][j])), fabsf(bf16_hi(w[s][j]))));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float f = inverse_power(top);   // (infinities stay what they are)
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int j = 0; j < 2; ++j) w[s][j] = pack_f16(bf16_lo(w[s][j]) * f, bf16_hi(w[s][j]) * f);
    return 1.0f / f;
}

// The running state of a thread's two rows, and what is the same for both forms.
template <int D, bool FP8, bool SM, int GN>
struct RowState {
    RowView rv[2];
    int hi_min, lo_max, hi_max;   // of all rows of the warp
    float qs[2];                  // scale of the scores
    float m[2], l[2];             // softmax: reference, sum
    float top[2], F[2];           // 8-bit: largest w 2^e_v in O; O is in units of 1 / F
    uint32_t bits[2][GN];         // events of the stage that the rows see
    bool masked;

    __device__ __forceinline__ void start() {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            m[x] = -INFINITY;
            l[x] = top[x] = 0.0f;
            F[x] = 1.0f;
        }
    }
    __device__ __forceinline__ void views(const AttnArgs& a, const Segment& g, int r0, int r1) {
        hi_min = 0x7fffffff;
        lo_max = hi_max = 0;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            rv[x] = row_view(a, g, x ? r1 : r0);
            if (rv[x].tok >= 0) {
                hi_min = min(hi_min, rv[x].hi);
                hi_max = max(hi_max, a.mask == GDPA_CACHE_TREE ? g.s.start + rv[x].tok + 1 : rv[x].hi);
                lo_max = max(lo_max, rv[x].lo);
            }
        }
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            hi_min = min(hi_min, __shfl_xor_sync(0xffffffffu, hi_min, k));
            hi_max = max(hi_max, __shfl_xor_sync(0xffffffffu, hi_max, k));
            lo_max = max(lo_max, __shfl_xor_sync(0xffffffffu, lo_max, k));
        }
    }
    __device__ __forceinline__ void mask(const AttnArgs& a, const Segment& g, const int (&e0)[GN], uint32_t missing) {
        masked = missing != 0;
#pragma unroll
        for (int u = 0; u < GN; ++u) masked = masked || !(e0[u] + 16 <= hi_min && (e0[u] >= lo_max || e0[u] + 16 <= a.sinks));
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int u = 0; u < GN; ++u) {
                bits[x][u] = 0xffffu;
                if (masked) bits[x][u] = missing >> u & 1u ? 0u : row_bits(a, g, rv[x], e0[u]);
            }
    }
    // Scores of NE events a row to weights (8-bit: times the values' powers of two
    // vs, still to be multiplied by F).  event(k): place of the thread's k-th event
    // in the stage; over(v): the largest of v over the lanes that share the rows;
    // scale(f): the rows' O times f.
    template <int NE, typename Event, typename Over, typename Scale>
    __device__ __forceinline__ void weigh(const AttnArgs& a, float (&s)[2][NE], const float (&vs)[NE], Event event, Over over, Scale scale) {
        // of what no row hides nothing is looked at
        const auto where_hidden = [&](float v) {
            if (!masked) return;
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int k = 0; k < NE; ++k)
                    if (!(bits[x][event(k) >> 4] >> (event(k) & 15) & 1u)) s[x][k] = v;
        };
        float f[2];
        if constexpr (SM) {
            where_hidden(-INFINITY);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float mt = s[x][0];
#pragma unroll
                for (int k = 1; k < NE; ++k) mt = fmaxf(mt, s[x][k]);
                mt = over(mt);
                // the reference moves when it would be passed by more than 8 (weights below 2^8)
                f[x] = 1.0f;
                if (mt > m[x] + 8.0f || m[x] == -INFINITY) {
                    f[x] = m[x] == -INFINITY ? 0.0f : ex2_approx(m[x] - mt);
                    m[x] = fmaxf(mt, -INFINITY);   // (of NaNs alone: none)
                }
            }
            if (__any_sync(0xffffffffu, f[0] != 1.0f || f[1] != 1.0f)) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    l[x] *= f[x];
                    top[x] *= f[x];
                }
                scale(f);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float ref = m[x] == -INFINITY ? 0.0f : m[x];
                float sum = 0.0f;   // (apart: one rounding to the size of l for all of them)
#pragma unroll
                for (int k = 0; k < NE; ++k) {
                    s[x][k] = ex2_approx(s[x][k] - ref);
                    sum += s[x][k];
                }
                l[x] += sum;
            }
        } else {
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int k = 0; k < NE; ++k) {
                    float& w = s[x][k];
                    switch (a.act) {
                        case kGeluErf: w = act_f<kGeluErf, true>(w); break;
                        case kGeluTanh: w = act_f<kGeluTanh, true>(w); break;
                        case kSilu: w = act_f<kSilu, true>(w); break;
                        case kTaylor6: w = act_f<kTaylor6, true>(w); break;
                        default: break;
                    }
                }
            if constexpr (!FP8) where_hidden(0.0f);
        }
        if constexpr (FP8) {
            // weights times the values' powers of two, in units of 1 / F
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int k = 0; k < NE; ++k) s[x][k] *= vs[k];
            where_hidden(0.0f);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float big = fabsf(s[x][0]);
#pragma unroll
                for (int k = 1; k < NE; ++k) big = fmaxf(big, fabsf(s[x][k]));
                big = over(big);
                const bool none = top[x] == 0.0f;   // O holds nothing yet
                top[x] = fmaxf(top[x], big);
                const float now = big * F[x];
                f[x] = 1.0f;
                if (big > 0.0f && !(now >= 0x1p7f && now <= 0x1p15f)) {
                    // (what O holds stays below 2^80 times the codes and their number, and the step is a float)
                    float next = fminf(inverse_power(big, 14), inverse_power(top[x], 80));
                    if (!none) next = fminf(next, F[x] * 0x1p126f);
                    f[x] = fminf(next / F[x], 0x1p126f);
                    F[x] = next;
                }
            }
            if (__any_sync(0xffffffffu, f[0] != 1.0f || f[1] != 1.0f)) scale(f);
        }
    }
    // two of a row's weights as operands
    __device__ __forceinline__ uint32_t pack(int x, float w0, float w1) const {
        return FP8 ? pack_f16(w0 * F[x], w1 * F[x]) : pack_bf16x2(w0, w1);
    }
};

// Clears the infinities and NaNs among value words; whether there were any.
template <bool FP8, int VW>
__device__ __forceinline__ bool clear_odd(uint32_t (&v)[4][VW]) {
    uint32_t odd = 0;
#pragma unroll
    for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int c = 0; c < VW; ++c) {
            const uint32_t x = odd_bits<FP8>(v[y][c]);
            odd |= x;
            v[y][c] &= ~x;
        }
    return odd != 0;
}

template <int D, bool FP8, bool SM>
struct Rows16 : RowState<D, FP8, SM, Cfg<D, FP8, false>::kTake> {
    using C = Cfg<D, FP8, false>;
    static constexpr int GN = C::kTake, STEPS = D / 16, NT = D / 8, VW = FP8 ? (D == 128 ? 4 : 2) : D / 16;
    using S = RowState<D, FP8, SM, GN>;
    uint32_t qf[STEPS][4];
    float o[NT][4];

    // rows gq and gq + 8 of the 16 from r0
    __device__ __forceinline__ void start(const AttnArgs& a, const Segment& g, int r0, int gq, int t) {
        S::start();
        S::views(a, g, r0 + gq, r0 + gq + 8);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            uint32_t w[STEPS][2];
            load_query<D, FP8>(a, g, r0 + gq + 8 * x, this->rv[x].tok, t, w);
            this->qs[x] = a.alpha;
            if constexpr (FP8) this->qs[x] *= scale_query<STEPS>(w);
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                qf[s][x] = w[s][0];
                qf[s][2 + x] = w[s][1];
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
    }

    // column of O in tile n
    __device__ static __forceinline__ int col(int t, int n, int c) {
        if constexpr (FP8 && D == 128) return 32 * t + 16 * c + n;
        return 64 * (n >> 3) + 16 * t + 8 * c + (n & 7);
    }

    __device__ __forceinline__ void stage(const AttnArgs& a, const Segment& g, const int (&e0)[GN], uint32_t missing,
                                          const uint8_t* kv, const uint8_t* scales, int lane) {
        const int gq = lane >> 2, t = lane & 3;
        // S: events 8 n + gq are B columns; the thread's scores are events 8 n + 2 t + j
        constexpr int SPLIT = GN == 1 ? 2 : 1;   // independent sums of a tile: every second step apart
        float acc[2 * GN][SPLIT][4];
#pragma unroll
        for (int n = 0; n < 2 * GN; ++n)
#pragma unroll
            for (int y = 0; y < SPLIT; ++y) acc[n][y][0] = acc[n][y][1] = acc[n][y][2] = acc[n][y][3] = 0.0f;
#pragma unroll
        for (int c = 0; c < (FP8 ? D / 64 : D / 32); ++c) {
            uint4 w[2 * GN];
#pragma unroll
            for (int n = 0; n < 2 * GN; ++n) w[n] = key_piece<D, FP8>(kv + (n >> 1) * 2 * C::kKeys, 8 * (n & 1) + gq, t, c);
            if constexpr (FP8) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int n = 0; n < 2 * GN; ++n) {
                        const uint32_t x = (&w[n].x)[j];
                        mma16<true>(acc[n][j % SPLIT], qf[4 * c + j], codes_lo(x), codes_hi(x));
                    }
            } else {
#pragma unroll
                for (int n = 0; n < 2 * GN; ++n) mma16<false>(acc[n][0], qf[2 * c], w[n].x, w[n].y);
#pragma unroll
                for (int n = 0; n < 2 * GN; ++n) mma16<false>(acc[n][SPLIT - 1], qf[2 * c + 1], w[n].z, w[n].w);
            }
        }
        float s[2][4 * GN], vs[4 * GN];
#pragma unroll
        for (int n = 0; n < 2 * GN; ++n) {
            float ks[2] = {1.0f, 1.0f};
            vs[2 * n] = vs[2 * n + 1] = 1.0f;
            if constexpr (FP8) {
                const uint8_t* sc = scales + (n >> 1) * C::kScales + 8 * (n & 1) + 2 * t;
                const uint32_t kb = *reinterpret_cast<const uint16_t*>(sc), vb = *reinterpret_cast<const uint16_t*>(sc + 16);
                ks[0] = cache_scale(kb & 255);
                ks[1] = cache_scale(kb >> 8);
                vs[2 * n] = cache_scale(vb & 255);
                vs[2 * n + 1] = cache_scale(vb >> 8);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int i = 2 * x + j;
                    const float y = SPLIT == 1 ? acc[n][0][i] : acc[n][0][i] + acc[n][SPLIT - 1][i];
                    s[x][2 * n + j] = y * ks[j] * this->qs[x];
                }
        }
        S::mask(a, g, e0, missing);
        S::weigh(
            a, s, vs, [&](int k) { return 8 * (k >> 1) + 2 * t + (k & 1); },
            [&](float v) {
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
            },
            [&](const float (&f)[2]) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[n][i] *= f[i >> 1];
            });
#pragma unroll
        for (int u = 0; u < GN; ++u) {
            const uint8_t* vp = kv + u * 2 * C::kKeys + C::kKeys;
            uint32_t pf[4];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x) pf[2 * n + x] = S::pack(x, s[x][4 * u + 2 * n], s[x][4 * u + 2 * n + 1]);
            // events 2 t, 2 t + 1, 2 t + 8, 2 t + 9 are this thread's part of B
            uint32_t v[4][VW];
#pragma unroll
            for (int y = 0; y < 4; ++y) value_words<D, FP8, VW>(vp, 2 * t + (y & 1) + 8 * (y >> 1), gq, v[y]);
            const bool odd = this->masked && clear_odd<FP8, VW>(v);
            if constexpr (FP8) {
#pragma unroll
                for (int c = 0; c < VW; ++c) {
                    const uint32_t a0 = __byte_perm(v[0][c], v[1][c], 0x5140), a1 = __byte_perm(v[0][c], v[1][c], 0x7362);
                    const uint32_t b0 = __byte_perm(v[2][c], v[3][c], 0x5140), b1 = __byte_perm(v[2][c], v[3][c], 0x7362);
                    mma16<true>(o[4 * c], pf, codes_lo(a0), codes_lo(b0));
                    mma16<true>(o[4 * c + 1], pf, codes_hi(a0), codes_hi(b0));
                    mma16<true>(o[4 * c + 2], pf, codes_lo(a1), codes_lo(b1));
                    mma16<true>(o[4 * c + 3], pf, codes_hi(a1), codes_hi(b1));
                }
            } else {
#pragma unroll
                for (int c = 0; c < VW; ++c) {
                    mma16<false>(o[2 * c], pf, __byte_perm(v[0][c], v[1][c], 0x5410), __byte_perm(v[2][c], v[3][c], 0x5410));
                    mma16<false>(o[2 * c + 1], pf, __byte_perm(v[0][c], v[1][c], 0x7632), __byte_perm(v[2][c], v[3][c], 0x7632));
                }
            }
            if (this->masked && __any_sync(0xffffffffu, odd)) {
                // what was left out, one event at a time, for the rows that see it
#pragma unroll 1
                for (int e = 0; e < 16; ++e) {
                    const int src = (lane & ~3) | ((e & 7) >> 1);
                    float wt[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float w0 = e < 8 ? s[x][4 * u] : s[x][4 * u + 2], w1 = e < 8 ? s[x][4 * u + 1] : s[x][4 * u + 3];
                        wt[x] = __shfl_sync(0xffffffffu, (e & 1) ? w1 : w0, src) * this->F[x];
                    }
                    if (!((this->bits[0][u] | this->bits[1][u]) >> e & 1u)) continue;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float y = value_at<D, FP8>(vp, e, col(t, n, c));
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                if ((this->bits[x][u] >> e & 1u) && !isfinite(y)) o[n][2 * x + c] = fmaf(wt[x], y, o[n][2 * x + c]);
                        }
                }
            }
        }
    }

    // sums (of this warp), maxima and sums of the weights (rows of a warp's 16)
    __device__ __forceinline__ void finish(const Segment& g, int r0, int gq, int t, float* sums, float2* ml) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float l = this->l[x];
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            const int r = gq + 8 * x;
            if (t == 0) ml[r] = make_float2(this->m[x], l);
            if (r0 + r >= g.rows) continue;
            const float f = FP8 ? 1.0f / this->F[x] : 1.0f;
#pragma unroll
            for (int n = 0; n < NT; n += 4)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    *reinterpret_cast<float4*>(sums + C::sum_at(r, col(t, n, c))) =
                        make_float4(o[n][2 * x + c] * f, o[n + 1][2 * x + c] * f, o[n + 2][2 * x + c] * f, o[n + 3][2 * x + c] * f);
        }
    }
};

// an 8 x 8 matrix of 16-bit values, a row in four lanes, turned
__device__ __forceinline__ uint32_t turn(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int D, bool FP8, bool SM>
struct Rows8 : RowState<D, FP8, SM, Cfg<D, FP8, true>::kTake> {
    using C = Cfg<D, FP8, true>;
    static constexpr int GN = C::kTake, STEPS = D / 16, MT = D / 16, VW = FP8 ? (D == 128 ? 4 : 2) : D / 16;
    using S = RowState<D, FP8, SM, GN>;
    uint32_t qf[STEPS][2];   // of row gq
    float o[MT][4];          // columns col(i), col(i) + 1 (c >> 1) of rows 2 t, 2 t + 1 (c & 1)

    __device__ __forceinline__ void start(const AttnArgs& a, const Segment& g, int r0, int gq, int t) {
        S::start();
        S::views(a, g, r0 + 2 * t, r0 + 2 * t + 1);
        uint32_t w[STEPS][2];
        load_query<D, FP8>(a, g, r0 + gq, row_view(a, g, r0 + gq).tok, t, w);
        this->qs[0] = this->qs[1] = a.alpha;
        if constexpr (FP8) {
            const float f = scale_query<STEPS>(w);
#pragma unroll
            for (int x = 0; x < 2; ++x) this->qs[x] *= __shfl_sync(0xffffffffu, f, 4 * (2 * t + x));
        }
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            qf[s][0] = w[s][0];
            qf[s][1] = w[s][1];
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    }

    // first of the two columns of O in tile i
    __device__ static __forceinline__ int col(int gq, int i) {
        if constexpr (FP8) return (D / 8) * gq + 2 * i;
        return 64 * (i >> 2) + 8 * gq + 2 * (i & 3);
    }

    __device__ __forceinline__ void stage(const AttnArgs& a, const Segment& g, const int (&e0)[GN], uint32_t missing,
                                          const uint8_t* kv, const uint8_t* scales, int lane) {
        const int gq = lane >> 2, t = lane & 3;
        // S^T: events gq and gq + 8 of a group are A rows, and the thread's scores with rows 2 t, 2 t + 1
        constexpr int SPLIT = 2;   // independent sums of a group: every second step apart
        float acc[GN][SPLIT][4];
#pragma unroll
        for (int u = 0; u < GN; ++u)
#pragma unroll
            for (int y = 0; y < SPLIT; ++y) acc[u][y][0] = acc[u][y][1] = acc[u][y][2] = acc[u][y][3] = 0.0f;
#pragma unroll
        for (int c = 0; c < (FP8 ? D / 64 : D / 32); ++c) {
            uint4 w[GN][2];
#pragma unroll
            for (int u = 0; u < GN; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) w[u][h] = key_piece<D, FP8>(kv + u * 2 * C::kKeys, 8 * h + gq, t, c);
            if constexpr (FP8) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int u = 0; u < GN; ++u) {
                        const uint32_t x = (&w[u][0].x)[j], y = (&w[u][1].x)[j];
                        const uint32_t k[4] = {codes_lo(x), codes_lo(y), codes_hi(x), codes_hi(y)};
                        mma16<true>(acc[u][j & 1], k, qf[4 * c + j][0], qf[4 * c + j][1]);
                    }
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int u = 0; u < GN; ++u) {
                        const uint32_t k[4] = {j ? w[u][0].z : w[u][0].x, j ? w[u][1].z : w[u][1].x, j ? w[u][0].w : w[u][0].y,
                                               j ? w[u][1].w : w[u][1].y};
                        mma16<false>(acc[u][j], k, qf[2 * c + j][0], qf[2 * c + j][1]);
                    }
            }
        }
        float s[2][2 * GN], vs[2 * GN];
#pragma unroll
        for (int u = 0; u < GN; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float ks = 1.0f;
                vs[2 * u + h] = 1.0f;
                if constexpr (FP8) {
                    const uint8_t* sc = scales + u * C::kScales + 8 * h + gq;
                    ks = cache_scale(sc[0]);
                    vs[2 * u + h] = cache_scale(sc[16]);
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int i = 2 * h + x;
                    const float y = acc[u][0][i] + acc[u][1][i];
                    s[x][2 * u + h] = y * ks * this->qs[x];
                }
            }
        S::mask(a, g, e0, missing);
        S::weigh(
            a, s, vs, [&](int k) { return 8 * k + gq; },
            [&](float v) {
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            },
            [&](const float (&f)[2]) {
#pragma unroll
                for (int n = 0; n < MT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[n][i] *= f[i & 1];
            });
#pragma unroll
        for (int u = 0; u < GN; ++u) {
            const uint8_t* vp = kv + u * 2 * C::kKeys + C::kKeys;
            // weights of an event with rows 2 t, 2 t + 1 -> of row gq with events 2 t, 2 t + 1
            uint32_t p[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float w0 = s[0][2 * u + h], w1 = s[1][2 * u + h];
                p[h] = turn(FP8 ? pack_f16(w0 * this->F[0], w1 * this->F[1]) : pack_bf16x2(w0, w1));
            }
            uint32_t v[4][VW];
#pragma unroll
            for (int y = 0; y < 4; ++y) value_words<D, FP8, VW>(vp, 2 * t + (y & 1) + 8 * (y >> 1), gq, v[y]);
            const bool odd = this->masked && clear_odd<FP8, VW>(v);
#pragma unroll
            for (int c = 0; c < VW; ++c) {
                if constexpr (FP8) {
                    const uint32_t a0 = __byte_perm(v[0][c], v[1][c], 0x5140), a1 = __byte_perm(v[0][c], v[1][c], 0x7362);
                    const uint32_t b0 = __byte_perm(v[2][c], v[3][c], 0x5140), b1 = __byte_perm(v[2][c], v[3][c], 0x7362);
                    const uint32_t x[4] = {codes_lo(a0), codes_hi(a0), codes_lo(b0), codes_hi(b0)};
                    const uint32_t y[4] = {codes_lo(a1), codes_hi(a1), codes_lo(b1), codes_hi(b1)};
                    mma16<true>(o[2 * c], x, p[0], p[1]);
                    mma16<true>(o[2 * c + 1], y, p[0], p[1]);
                } else {
                    const uint32_t x[4] = {__byte_perm(v[0][c], v[1][c], 0x5410), __byte_perm(v[0][c], v[1][c], 0x7632),
                                           __byte_perm(v[2][c], v[3][c], 0x5410), __byte_perm(v[2][c], v[3][c], 0x7632)};
                    mma16<false>(o[c], x, p[0], p[1]);
                }
            }
            if (this->masked && __any_sync(0xffffffffu, odd)) {
                // what was left out, one event at a time, for the rows that see it
#pragma unroll 1
                for (int e = 0; e < 16; ++e) {
                    const int src = 4 * (e & 7) + t;
                    float wt[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        wt[x] = __shfl_sync(0xffffffffu, e < 8 ? s[x][2 * u] : s[x][2 * u + 1], src) * this->F[x];
                    if (!((this->bits[0][u] | this->bits[1][u]) >> e & 1u)) continue;
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float y = value_at<D, FP8>(vp, e, col(gq, i) + c);
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                if ((this->bits[x][u] >> e & 1u) && !isfinite(y)) o[i][2 * c + x] = fmaf(wt[x], y, o[i][2 * c + x]);
                        }
                }
            }
        }
    }

    __device__ __forceinline__ void finish(const Segment& g, int r0, int gq, int t, float* sums, float2* ml) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float l = this->l[x];
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
            const int r = 2 * t + x;
            if (gq == 0) ml[r] = make_float2(this->m[x], l);
            if (r0 + r >= g.rows) continue;
            const float f = FP8 ? 1.0f / this->F[x] : 1.0f;
#pragma unroll
            for (int i = 0; i < MT; i += 2)
                *reinterpret_cast<float4*>(sums + C::sum_at(r, col(gq, i))) =
                    make_float4(o[i][x] * f, o[i][2 + x] * f, o[i + 1][x] * f, o[i + 1][2 + x] * f);
        }
    }
};

}  // namespace cache_mma
}  // namespace gdpa
