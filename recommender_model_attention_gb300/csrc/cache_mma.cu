// Attention over the history cache for bf16 rows with d = 64 or 128, on
// warp-level tensor-core products (m16n8k16).
//
// With a handful of query rows a key head (one new event, or a small tree, times
// the heads that share it) every cached byte is used for a few products only, so
// what bounds the kernel is reading the cache once.  Each warp therefore streams
// its own events: groups of 16 come in by bulk copies through a ring in shared
// memory, several groups ahead, and are used from there as operands without any
// rearrangement (the cache lies in the order that needs none): a thread's 16
// bytes of a key row are the B operand of S = Q K^T for 4 (8-bit: 8) steps of
// the contraction, whose order over d is free as long as Q has the same; two
// value rows' bytes interleaved are the B operand of O += P V, each thread's
// columns of O being a run of d.  A CTA's four warps take turns over the groups
// (KS = 4 / RT of them, the others hold further 16-row tiles of the same events)
// and join their sums in shared memory.
//
// 8-bit keys are multiplied as they are (m16n8k32): S = 2^(e_k + e_q) (q' + 2^-5
// q'') . c, where q' are the codes of the row scaled by a power of two to below
// 256 and q'' those of 2^5 times the rest, two E4M3 numbers of 4 bits for bf16's 8
// (elements below 2^-15 of the largest lose bits, at most 2^-22 of it).  Such a
// product takes half of an f16 one's time for twice the depth, and saves the
// conversions.  8-bit values become f16 (exactly).  Their rows' powers of two go
// into the weights, w 2^e_v F, rounded to f16; F is a power of two that keeps the
// largest w 2^e_v that O holds within [2^-6, 2^8], moved (and O with it) when
// it leaves that range, so that rows of any size keep f16's 11 bits.  bf16
// caches use bf16 products, weights rounded to bf16 (2^-9 of each).
// Scores, maxima, sums and O are float32.
//
// A group that some row does not see is masked bit by bit.  A hidden event's
// weight is 0, and 0 times an infinity or a NaN would be NaN: a masked group's
// values enter the product without those, which are then added one by one to the
// rows that see them.
#include "cache_attn.cuh"
#include "tc_common.cuh"

namespace gdpa {
namespace {

using namespace tc;

constexpr int kThreads = 128;

template <int D, bool FP8>
struct Cfg {
    static constexpr int kRow = FP8 ? D : 2 * D;            // bytes of a cache row
    static constexpr int kCols = kRow >= 128 ? kRow / 128 : 1;
    static constexpr int kKeys = 16 * kRow;                 // bytes of a group's K (or V)
    static constexpr int kScales = FP8 ? 32 : 0;            // ... of its scales
    // groups of a ring's stage, taken together: the more, the more independent
    // products and the fewer waits and votes a byte; bf16 rows of 128 leave no
    // room for two
    static constexpr int kTake = FP8 || D == 64 ? 2 : 1;
    static constexpr int kRing = FP8 && D == 64 ? 16 : 12;   // stages of all rings
    static constexpr int kOwn = FP8 && D == 128 ? 32 : 16;  // run of columns of a thread's part of O
    static constexpr int kColSkip = D + 8 * (D / kOwn);     // padded columns of a row of sums
    static constexpr int kRowLen = kColSkip + 4;
    static constexpr int kSums = 4 * 16 * kRowLen * 4;
    static constexpr int kStage = kTake * 2 * kKeys;
    static constexpr int kRingBytes = kRing * kStage;
    static constexpr int kMain = kRingBytes > kSums ? kRingBytes : kSums;
    static constexpr int kBytes = kMain + kRing * kTake * kScales;
};

// columns of O (and of Q, in groups of 4: see below) that a thread holds
template <int D, bool FP8>
__device__ __forceinline__ int own_col(int t, int n, int c) {   // n: 8-column tile of O, c: 0 or 1
    if constexpr (FP8 && D == 128) return 32 * t + 16 * c + n;
    return 64 * (n >> 3) + 16 * t + 8 * c + (n & 7);
}
// first of the 4 columns of step s of the contraction over d
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
__device__ __forceinline__ void mma_e4m3(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// two values of a query row (at most 256) as E4M3 codes, and 2^5 times what these leave of them
__device__ __forceinline__ void split_q(float x, float y, uint32_t& hi, uint32_t& lo) {
    uint16_t h, l;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(y), "f"(x));
    uint32_t f;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"(h));
    const float2 v = __half22float2(*reinterpret_cast<__half2*>(&f));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(l) : "f"((y - v.y) * 32.0f), "f"((x - v.x) * 32.0f));
    hi = h;
    lo = l;
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

__device__ __forceinline__ void bulk_load(uint64_t* bar, void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// all bits of those of the packed bf16 pair / 8-bit codes that are infinities or NaNs
template <bool FP8>
__device__ __forceinline__ uint32_t odd_bits(uint32_t w) {
    if constexpr (FP8) return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
    return __vcmpeq2(w & 0x7f807f80u, 0x7f807f80u);
}

// the power of two 2^-floor(log2 x), x > 0 finite and normal; kept within f32
__device__ __forceinline__ float inverse_power(float x) {
    const uint32_t e = __float_as_uint(x) >> 23;
    return __uint_as_float((uint32_t)(min(max(254 - (int)e, 1), 254)) << 23);
}

template <int D, bool FP8, bool SM>
__global__ void __launch_bounds__(kThreads, kCacheMmaPerSm)
cache_mma_kernel(const __grid_constant__ AttnArgs a) {
    using C = Cfg<D, FP8>;
    constexpr int KSTEPS = D / 16, NT = D / 8;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint64_t full[C::kRing], empty[C::kRing];
    __shared__ int64_t scan_tmp[kThreads / 32 + 2];
    __shared__ uint8_t gone[C::kRing];              // groups of a stage whose page lies outside the cache
    __shared__ float2 ml[4][16];
    __shared__ int abort_flag;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gq = lane >> 2, t = lane & 3;
    const int RT = a.RT, KS = 4 / RT;
    const int rt = warp % RT, ks = warp / RT;
    const int NS = C::kRing / 4 * RT, ring0 = ks * NS;   // this warp's ring: stages ring0 .. ring0 + NS
    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < C::kRing; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], RT);
        }
        fence_mbar_init();
    }
    const Abort ab{&abort_flag, a.c.err, kWaitLimitNs};
    asm volatile("griddepcontrol.launch_dependents;");
    if (tid == 0) a.desc[blockIdx.x].parts = 0;
    Share sh = find_share<kThreads>(a, scan_tmp);   // (synchronises the CTA)
    // places in this warp's ring, and the parity of their use: of the next group
    // to load (the wait for it to be empty) and to use; groups on their way
    int st_in = ring0, st_out = ring0, on_way = 0;
    uint32_t ph_in = 1, ph_out = 0;
    const auto next_place = [&](int& st, uint32_t& ph) {
        if (++st == ring0 + NS) {
            st = ring0;
            ph ^= 1;
        }
    };
    while (sh.u < sh.u_end) {
        const Segment g = next_segment(a, sh);
        if (g.rows == 0) break;
        constexpr int GN = C::kTake;
        const int stages = (g.n + GN - 1) / GN;
        const int mine = stages > ks ? (stages - ks + KS - 1) / KS : 0;   // this ring's: ks, ks + KS, ...
        // ---- loads: the ring's first warp; pages looked up 32 groups at a time, a
        // lane a copy: K and V of each group by columns of the layout, and the scales
        constexpr uint32_t kPiece = C::kKeys / C::kCols;
        constexpr int kCopies = 2 * C::kCols + (FP8 ? 2 : 0);   // of a group
        const int cu = lane / kCopies, cc = lane % kCopies;     // group of the stage, copy
        const bool is_v = cc & 1, is_scale = cc >= 2 * C::kCols;
        int64_t my_block = -1;
        const auto issue = [&](int i) {             // whole warp, stage i of this ring's
            if ((i & (32 / GN - 1)) == 0) {
                const int j = (ks + KS * (i + lane / GN)) * GN + lane % GN;
                my_block = j < g.n ? cache_block(a.c, a.w, g.b, (int64_t)segment_group(g, j) * kCacheGroup, g.h) : -1;
            }
            const int at0 = (i & (32 / GN - 1)) * GN;
            const int64_t blk = __shfl_sync(0xffffffffu, my_block, at0 + min(cu, GN - 1));
            const uint32_t there = __ballot_sync(0xffffffffu, my_block >= 0) >> at0 & ((1u << GN) - 1);
            if (!__all_sync(0xffffffffu, mbar_wait(&empty[st_in], ph_in, ab, 1))) return false;
            if (lane == 0) {
                gone[st_in] = (uint8_t)~there;
                mbar_arrive_expect_tx(&full[st_in], __popc(there) * (2 * C::kKeys + C::kScales));
            }
            __syncwarp();
            if (cu < GN && blk >= 0) {
                const int e0 = (segment_group(g, (ks + KS * i) * GN + cu) * kCacheGroup) & ((1 << a.c.page_log) - 1);
                if (is_scale) {
                    bulk_load(&full[st_in], smem + C::kMain + (st_in * GN + cu) * C::kScales + 16 * is_v,
                              (is_v ? a.c.vs : a.c.ks) + (blk << a.c.page_log) + e0, 16);
                } else {
                    const int col = cc >> 1;
                    const int at = C::kRow >= 128 ? ((col << a.c.page_log) + e0) * 128 : e0 * C::kRow;
                    bulk_load(&full[st_in], smem + st_in * C::kStage + cu * 2 * C::kKeys + is_v * C::kKeys + col * kPiece,
                              (is_v ? a.c.v : a.c.k) + blk * a.c.block + at, kPiece);
                }
            }
            ++on_way;
            next_place(st_in, ph_in);
            return true;
        };
        int ahead = 0;
        bool ok = true;
        if (rt == 0)
            for (; ahead < mine && ahead < NS && ok; ++ahead) ok = issue(ahead);

        // ---- this thread's rows gq and gq + 8 of the warp's tile
        const bool active = 16 * rt < g.rows;
        RowView rv[2];
        uint32_t qf[KSTEPS][4];
        float qs[2];
        int hi_min = 0x7fffffff, lo_max = 0, hi_max = 0;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int r = 16 * rt + gq + 8 * x;
            rv[x] = row_view(a, g, r);
            if (rv[x].tok >= 0) {
                hi_min = min(hi_min, rv[x].hi);
                hi_max = max(hi_max, a.mask == GDPA_CACHE_TREE ? g.s.start + rv[x].tok + 1 : rv[x].hi);
                lo_max = max(lo_max, rv[x].lo);
            }
            const int rho = g.rho0 + r, tok = max(rv[x].tok, 0);
            const __nv_bfloat16* src = (const __nv_bfloat16*)a.q + (g.s.t0 + tok) * a.qt + (g.h * a.G + rho - tok * a.G) * a.qh;
            uint32_t w[KSTEPS][2];
#pragma unroll
            for (int s = 0; s < KSTEPS; s += 2) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (rv[x].tok >= 0) {
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
            qs[x] = a.alpha;
            if constexpr (FP8) {
                float top = 0.0f;
#pragma unroll
                for (int s = 0; s < KSTEPS; ++s)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        top = fmaxf(top, fmaxf(fabsf(bf16_lo(w[s][j])), fabsf(bf16_hi(w[s][j]))));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const float f = inverse_power(top);   // of infinities: whatever, their products are
                // steps of 32: words 2 j and 2 j + 1 of a piece, codes of 4 values each
#pragma unroll
                for (int s = 0; s < KSTEPS; ++s) {
                    uint32_t hi[2], lo[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) split_q(bf16_lo(w[s][j]) * f * 128.0f, bf16_hi(w[s][j]) * f * 128.0f, hi[j], lo[j]);
                    qf[s >> 1][2 * (s & 1) + x] = hi[0] | hi[1] << 16;
                    qf[KSTEPS / 2 + (s >> 1)][2 * (s & 1) + x] = lo[0] | lo[1] << 16;
                }
                qs[x] *= 0x1p-7f / f;
            } else {
#pragma unroll
                for (int s = 0; s < KSTEPS; ++s) {
                    qf[s][x] = w[s][0];
                    qf[s][2 + x] = w[s][1];
                }
            }
        }
#pragma unroll
        for (int m = 4; m < 32; m <<= 1) {
            hi_min = min(hi_min, __shfl_xor_sync(0xffffffffu, hi_min, m));
            hi_max = max(hi_max, __shfl_xor_sync(0xffffffffu, hi_max, m));
            lo_max = max(lo_max, __shfl_xor_sync(0xffffffffu, lo_max, m));
        }
        float o[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
        float top[2] = {0.0f, 0.0f}, F[2] = {1.0f, 1.0f};   // 8-bit: largest w 2^e_v in O; O's unit

        // ---- the ring's stages
        for (int i = 0; i < mine && ok; ++i) {
            const int st = st_out;
            if (!__all_sync(0xffffffffu, mbar_wait(&full[st], ph_out, ab, 2))) {
                ok = false;
                break;
            }
            next_place(st_out, ph_out);
            const uint8_t* stage = smem + st * C::kStage;
            const uint32_t missing = gone[st] & ((1u << GN) - 1);   // (also groups behind the last)
            int e0[GN];
#pragma unroll
            for (int u = 0; u < GN; ++u) e0[u] = segment_group(g, (ks + KS * i) * GN + u) * kCacheGroup;
            if (active && e0[0] < hi_max) {
                // S = Q K^T: events 8 n + gq are B columns (n: 2 tiles a group)
                float s[2 * GN][4];
                {
                    // independent sums of a tile: what is left of Q apart (8-bit), or every second step
                    constexpr int SPLIT = FP8 || GN == 1 ? 2 : 1;
                    float acc[2 * GN][SPLIT][4];
#pragma unroll
                    for (int n = 0; n < 2 * GN; ++n)
#pragma unroll
                        for (int y = 0; y < SPLIT; ++y) acc[n][y][0] = acc[n][y][1] = acc[n][y][2] = acc[n][y][3] = 0.0f;
                    constexpr int CH = FP8 ? (D == 128 ? 2 : 1) : D / 32;   // 16-byte pieces of a key row a thread takes
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        uint4 w[2 * GN];
#pragma unroll
                        for (int n = 0; n < 2 * GN; ++n) {
                            const uint8_t* kp = stage + (n >> 1) * 2 * C::kKeys;
                            const int e = 8 * (n & 1) + gq;
                            if constexpr (FP8 && D == 64)
                                w[n] = *reinterpret_cast<const uint4*>(kp + (e >> 1) * 128 + (((4 * (e & 1) + t) ^ (2 * ((e >> 1) & 3))) << 4));
                            else
                                w[n] = *reinterpret_cast<const uint4*>(kp + (c >> 1) * 2048 + e * 128 + (((2 * t + (c & 1)) ^ (e & 7)) << 4));
                        }
                        if constexpr (FP8) {
#pragma unroll
                            for (int y = 0; y < 2; ++y)
#pragma unroll
                                for (int n = 0; n < 2 * GN; ++n) mma_e4m3(acc[n][y], qf[y * (KSTEPS / 2) + 2 * c], w[n].x, w[n].y);
#pragma unroll
                            for (int y = 0; y < 2; ++y)
#pragma unroll
                                for (int n = 0; n < 2 * GN; ++n) mma_e4m3(acc[n][y], qf[y * (KSTEPS / 2) + 2 * c + 1], w[n].z, w[n].w);
                        } else {
#pragma unroll
                            for (int n = 0; n < 2 * GN; ++n) mma16<false>(acc[n][0], qf[2 * c], w[n].x, w[n].y);
#pragma unroll
                            for (int n = 0; n < 2 * GN; ++n) mma16<false>(acc[n][SPLIT - 1], qf[2 * c + 1], w[n].z, w[n].w);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < 2 * GN; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            s[n][j] = SPLIT == 1 ? acc[n][0][j] : FP8 ? fmaf(acc[n][SPLIT - 1][j], 0x1p-5f, acc[n][0][j]) : acc[n][0][j] + acc[n][SPLIT - 1][j];
                }
                // scores: rows gq, gq + 8 (x), events 8 n + 2 t + j
                float vs[2 * GN][2];
#pragma unroll
                for (int n = 0; n < 2 * GN; ++n) {
                    float ksc[2] = {1.0f, 1.0f};
                    vs[n][0] = vs[n][1] = 1.0f;
                    if constexpr (FP8) {
                        const uint8_t* sc = smem + C::kMain + (st * GN + (n >> 1)) * C::kScales + 8 * (n & 1) + 2 * t;
                        const uint32_t kb = *reinterpret_cast<const uint16_t*>(sc);
                        const uint32_t vb = *reinterpret_cast<const uint16_t*>(sc + 16);
                        ksc[0] = cache_scale(kb & 255);
                        ksc[1] = cache_scale(kb >> 8);
                        vs[n][0] = cache_scale(vb & 255);
                        vs[n][1] = cache_scale(vb >> 8);
                    }
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int j = 0; j < 2; ++j) s[n][2 * x + j] = s[n][2 * x + j] * ksc[j] * qs[x];
                }
                bool masked = missing != 0;
#pragma unroll
                for (int u = 0; u < GN; ++u)
                    masked = masked || !(e0[u] + 16 <= hi_min && (e0[u] >= lo_max || e0[u] + 16 <= a.sinks));
                uint32_t bits[2][GN];
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int u = 0; u < GN; ++u) bits[x][u] = 0xffffu;
                if (masked) {
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int u = 0; u < GN; ++u) bits[x][u] = missing >> u & 1u ? 0u : row_bits(a, g, rv[x], e0[u]);
                }
                const auto seen = [&](int x, int n, int j) { return (bits[x][n >> 1] >> (8 * (n & 1) + 2 * t + j)) & 1u; };
                if constexpr (SM) {
                    float f[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float mt = -INFINITY;
#pragma unroll
                        for (int n = 0; n < 2 * GN; ++n)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                if (masked && !seen(x, n, j)) s[n][2 * x + j] = -INFINITY;
                                mt = fmaxf(mt, s[n][2 * x + j]);
                            }
                        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
                        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
                        // the reference moves when it would be passed by more than 8 (weights below 2^8)
                        f[x] = 1.0f;
                        if (mt > m[x] + 8.0f || m[x] == -INFINITY) {
                            f[x] = m[x] == -INFINITY ? 0.0f : ex2_approx(m[x] - mt);
                            m[x] = mt;
                        }
                    }
                    if (__any_sync(0xffffffffu, f[0] != 1.0f || f[1] != 1.0f)) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            l[x] *= f[x];
                            top[x] *= f[x];
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                o[n][2 * x] *= f[x];
                                o[n][2 * x + 1] *= f[x];
                            }
                        }
                    }
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float ref = m[x] == -INFINITY ? 0.0f : m[x];
#pragma unroll
                        for (int n = 0; n < 2 * GN; ++n)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                s[n][2 * x + j] = ex2_approx(s[n][2 * x + j] - ref);
                                l[x] += s[n][2 * x + j];
                            }
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < 2 * GN; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float& w = s[n][j];
                            switch (a.act) {
                                case kGeluErf: w = act_f<kGeluErf, true>(w); break;
                                case kGeluTanh: w = act_f<kGeluTanh, true>(w); break;
                                case kSilu: w = act_f<kSilu, true>(w); break;
                                case kTaylor6: w = act_f<kTaylor6, true>(w); break;
                                default: break;
                            }
                            if (masked && !seen(j >> 1, n, j & 1)) w = 0.0f;
                        }
                }
                if constexpr (FP8) {
                    // weights times the values' powers of two, in units of 1 / F
                    float f[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float big = 0.0f;
#pragma unroll
                        for (int n = 0; n < 2 * GN; ++n)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                s[n][2 * x + j] = masked && !seen(x, n, j) ? 0.0f : s[n][2 * x + j] * vs[n][j];
                                big = fmaxf(big, fabsf(s[n][2 * x + j]));
                            }
                        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                        top[x] = fmaxf(top[x], big);
                        const float now = top[x] * F[x];
                        f[x] = 1.0f;
                        if (top[x] > 0.0f && !(now >= 0x1p-6f && now <= 0x1p8f)) {
                            const float next = inverse_power(top[x]);
                            f[x] = fminf(next / F[x], 0x1p100f);   // (what O held is nothing by then)
                            F[x] = next;
                        }
                    }
                    if (__any_sync(0xffffffffu, f[0] != 1.0f || f[1] != 1.0f)) {
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                o[n][2 * x] *= f[x];
                                o[n][2 * x + 1] *= f[x];
                            }
                    }
                }
#pragma unroll
                for (int u = 0; u < GN; ++u) {
                    const uint8_t* vp = stage + u * 2 * C::kKeys + C::kKeys;
                    uint32_t pf[4];
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const float w0 = s[2 * u + n][2 * x], w1 = s[2 * u + n][2 * x + 1];
                            pf[2 * n + x] = FP8 ? pack_f16(w0 * F[x], w1 * F[x]) : pack_bf16x2(w0, w1);
                        }
                    // O += P V: events 2 t, 2 t + 1, 2 t + 8, 2 t + 9 are this thread's part of B
                    const int ev[4] = {2 * t, 2 * t + 1, 2 * t + 8, 2 * t + 9};
                    constexpr int VW = FP8 ? (D == 128 ? 4 : 2) : D / 16;   // words a row
                    uint32_t v[4][VW];
                    uint32_t odd = 0;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int e = ev[y];
                        if constexpr (FP8 && D == 128) {
                            *reinterpret_cast<uint4*>(v[y]) = *reinterpret_cast<const uint4*>(vp + e * 128 + ((gq ^ (e & 7)) << 4));
                        } else if constexpr (FP8) {
                            *reinterpret_cast<uint2*>(v[y]) = *reinterpret_cast<const uint2*>(
                                vp + (e >> 1) * 128 + (((4 * (e & 1) + (gq >> 1)) ^ (2 * ((e >> 1) & 3))) << 4) + 8 * (gq & 1));
                        } else {
#pragma unroll
                            for (int c = 0; c < D / 64; ++c)
                                *reinterpret_cast<uint4*>(v[y] + 4 * c) = *reinterpret_cast<const uint4*>(vp + c * 2048 + e * 128 + ((gq ^ (e & 7)) << 4));
                        }
                    }
                    if (masked) {
#pragma unroll
                        for (int y = 0; y < 4; ++y)
#pragma unroll
                            for (int c = 0; c < VW; ++c) {
                                const uint32_t x = odd_bits<FP8>(v[y][c]);
                                odd |= x;
                                v[y][c] &= ~x;
                            }
                    }
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
                    if (masked && __any_sync(0xffffffffu, odd != 0)) {
                        // what was left out, one event at a time, for the rows that see it
#pragma unroll 1
                        for (int e = 0; e < 16; ++e) {
                            const int src = (lane & ~3) | ((e & 7) >> 1);
                            float wt[2];
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const float w0 = e < 8 ? s[2 * u][2 * x] : s[2 * u + 1][2 * x], w1 = e < 8 ? s[2 * u][2 * x + 1] : s[2 * u + 1][2 * x + 1];
                                wt[x] = __shfl_sync(0xffffffffu, (e & 1) ? w1 : w0, src) * F[x];
                            }
                            if (!((bits[0][u] | bits[1][u]) >> e & 1u)) continue;
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int c = 0; c < 2; ++c) {
                                    const int col = own_col<D, FP8>(t, n, c);
                                    float y;
                                    if constexpr (FP8) {
                                        const int at = cache_chunk(C::kRow, 4, e, col >> 4) + (col & 15);
                                        const uint32_t h = codes_lo(vp[at]);
                                        y = __half2float(__ushort_as_half((uint16_t)h));
                                    } else {
                                        y = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(vp + cache_chunk(C::kRow, 4, e, col >> 3) + 2 * (col & 7)));
                                    }
#pragma unroll
                                    for (int x = 0; x < 2; ++x)
                                        if ((bits[x][u] >> e & 1u) && !isfinite(y)) o[n][2 * x + c] = fmaf(wt[x], y, o[n][2 * x + c]);
                                }
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
            --on_way;
            if (rt == 0 && ahead < mine) {
                ok = issue(ahead);
                ++ahead;
            }
        }
        // ---- the warps' sums, through the rings' memory
        if (!ok) {
            // gave up: copies still on their way land before the memory is given back
            if (rt == 0)
                for (; on_way > 0; --on_way) {
                    mbar_wait_teardown(&full[st_out], ph_out);
                    next_place(st_out, ph_out);
                }
        }
        __syncthreads();
        if (abort_flag) return;
        float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
            l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
            const int r = gq + 8 * x;
            if (t == 0) ml[warp][r] = make_float2(m[x], l[x]);
            if (16 * rt + r >= g.rows) continue;
            const float f = FP8 ? 1.0f / F[x] : 1.0f;
            float* row = sums + (warp * 16 + r) * C::kRowLen;
#pragma unroll
            for (int n = 0; n < NT; n += 4)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int col = own_col<D, FP8>(t, n, c);
                    *reinterpret_cast<float4*>(row + col + 8 * (col / C::kOwn)) =
                        make_float4(o[n][2 * x + c] * f, o[n + 1][2 * x + c] * f, o[n + 2][2 * x + c] * f, o[n + 3][2 * x + c] * f);
                }
        }
        __syncthreads();
        finish_segment<__nv_bfloat16, SM, kThreads>(
            a, g, KS,
            [&](int w, int r, int c) { return reinterpret_cast<const float4*>(sums + (w * 16 + r) * C::kRowLen + c + 8 * (c / C::kOwn)); },
            [&](int w, int r) { return ml[w][r]; });
        fence_proxy_async_smem();   // the next segment's copies write where these sums were
        __syncthreads();
    }
}

template <int D, bool FP8, bool SM>
gdpa_status launch(const AttnArgs& a, int grid, cudaStream_t st) {
    constexpr int bytes = Cfg<D, FP8>::kBytes;
    if (cudaFuncSetAttribute(cache_mma_kernel<D, FP8, SM>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return GDPA_ERR_CUDA;
    cache_mma_kernel<D, FP8, SM><<<grid, kThreads, bytes, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? GDPA_OK : GDPA_ERR_CUDA;
}

}  // namespace

gdpa_status launch_cache_mma(const AttnArgs& a, int grid, cudaStream_t st) {
    const bool fp8 = a.c.store == GDPA_STORE_E4M3, sm = a.act == kSoftmax;
    if (a.c.d == 128)
        return fp8 ? sm ? launch<128, true, true>(a, grid, st) : launch<128, true, false>(a, grid, st)
                   : sm ? launch<128, false, true>(a, grid, st) : launch<128, false, false>(a, grid, st);
    return fp8 ? sm ? launch<64, true, true>(a, grid, st) : launch<64, true, false>(a, grid, st)
               : sm ? launch<64, false, true>(a, grid, st) : launch<64, false, false>(a, grid, st);
}

}  // namespace gdpa
