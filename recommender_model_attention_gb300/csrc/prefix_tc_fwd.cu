// Shared-prefix attention forward on the tensor cores (bf16 rows, d = 64 or
// 128): the parts of every row tile, for the merge to join.
//
// One CTA per planned share walks its pieces.  A piece is one or two row
// tiles (packed token by token, query heads of one key head side by side; a
// 3-D TMA box does the packing) against a run of keys.  Two slots, each with
// its own score and sum columns in TMEM (128 + d) and one warpgroup, a thread
// a row:
//   two tiles: slot s holds tile s, both read the same key blocks;
//   one tile:  slot s takes the key blocks s, s + 2, ... of the same rows and
//              gives a part of its own.
// Warp 0 loads (TMA): the piece's query tiles, then K and V blocks through
// one ring, in the order in which the tensor core takes them.  Warp 1 issues
// S = Q K^T and O += P V: one slot's P V and next S run while the other's
// weights are computed.  What bounds it is a slot's chain of scores, weights
// and sums, so the chain is kept short: a row's 128 scores are read once into
// its thread's registers (the first warpgroup hands its registers over), the
// P V of a block's first 64 keys starts when their weights are written, and a
// third of the exponentials are taken by the multiply-add pipe (exp2_poly)
// beside the one unit a warp scheduler has for them.
// A warpgroup keeps its rows' maximum as a reference that only moves when it
// would be passed by more than 8 (in base 2: weights stay below 2^8), so O is
// rescaled in TMEM a few times a piece rather than at every block; that S is
// complete says that the P V before it is (they are issued in that order and
// commits follow all work issued before), so the rescale needs no wait.
//
// Rows of keys behind the piece's last one share its 16-row step: their
// scores are masked by selection and the rows of V are cleared in shared
// memory, so that what they hold (another sample's rows, infinities) does not
// reach P V as 0 * inf.
//
// Every wait is bounded (csrc/tc_common.cuh); P is rounded to bf16 for the
// product, the weights' sum is taken in float32 before that rounding.
#include <cuda_bf16.h>

#include "act.cuh"
#include "prefix_tc.cuh"

namespace gdpa {
namespace {

using namespace tc;

constexpr int kThreads = 384;   // producer and issuer (and two idle warps), a warpgroup per slot
constexpr int kHalfBytes = 128 * 128;
constexpr uint32_t kTmemCols = 512;
constexpr float kRise = 8.0f;   // the reference follows a maximum this far above it

template <int D>
struct PfCfg {
    static constexpr int kHalves = D / 64;
    static constexpr int kTile = 128 * D * 2;
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int kOffQ = 0;
    static constexpr int kOffKV = 2 * kTile;
    static constexpr int kOffBar = kOffKV + kStages * kTile;
    enum {
        kQFull = 0, kQEmpty, kFull, kEmpty = kFull + kStages, kSFull = kEmpty + kStages,
        kPFull = kSFull + 2,    // per slot and half of the block's keys
        kOFull = kPFull + 4, kOFree = kOFull + 2, kMmaDone = kOFree + 2, kNumBars
    };
    static constexpr int kSmem = kOffBar + kNumBars * 8 + 16 + 1024;
};

struct PfParams {
    const PrefixPiece* pieces;
    const int32_t* seg;
    float* parts;
    float* ml;
    int r, windowed, window;
    int q_bytes;      // bytes of one query tile's load
    float alpha;
    int32_t* err;
    uint64_t wait_ns;
    int stall;        // test hook: CTA 0 never loads its first queries
};

// Blocks of a piece, of each slot, and where they lie in the ring (counted
// from the piece's first load).
struct Walk {
    int nb, n0, n1;
    bool dual;
    __device__ __forceinline__ Walk(const PrefixPiece& p) {
        nb = (p.nk + kBN - 1) / kBN;
        dual = p.flags & kPieceDual;
        n0 = dual ? (nb + 1) >> 1 : nb;
        n1 = dual ? nb >> 1 : nb;
    }
    __device__ __forceinline__ int blocks(int s) const { return s ? n1 : n0; }
    __device__ __forceinline__ int block(int s, int j) const { return dual ? 2 * j + s : j; }
    // two tiles: K0 V0 K1 V1 ...; one tile: K0 K1 V0 K2 V1 K3 ...
    __device__ __forceinline__ int v_at(int b) const { return dual ? min(b + 2, nb) + b : 2 * b + 1; }
};

template <int D>
__device__ __forceinline__ void pf_producer(const CUtensorMap* tmQ, const CUtensorMap* tmKp, const CUtensorMap* tmVp,
                            const CUtensorMap* tmK, const CUtensorMap* tmV, const PfParams& prm,
                            uint8_t* smem, uint64_t* bars, int seg0, int seg1, const Abort& ab) {
    using C = PfCfg<D>;
    const uint64_t keep = policy_evict_last(), once = policy_evict_first();
    int32_t q_armed = -1, armed[C::kStages];
    for (int s = 0; s < C::kStages; ++s) armed[s] = -1;
    uint32_t c = 0;
    for (int t = seg0; t < seg1; ++t) {
        const PrefixPiece p = load_piece(prm.pieces + t);
        const Walk w(p);
        const uint32_t n = (uint32_t)(t - seg0);
        if (!mbar_wait<true>(&bars[C::kQEmpty], (n & 1) ^ 1, ab, 61)) goto unwind;
        if (!(prm.stall && blockIdx.x == 0 && n == 0)) {
            mbar_arrive_expect_tx(&bars[C::kQFull], (uint32_t)(prm.q_bytes * (p.nB > 0 ? 2 : 1)));
            q_armed = (int32_t)(n & 1);
            for (int half = 0; half < (p.nB > 0 ? 2 : 1); ++half)
#pragma unroll
                for (int hf = 0; hf < C::kHalves; ++hf)
                    tma_load_3d(tmQ, &bars[C::kQFull], smem + C::kOffQ + half * C::kTile + hf * kHalfBytes,
                                hf * 64, p.hk * prm.r, p.tok + half * p.nA, once);
        }
        const bool own = p.flags & kPieceOwn;
        const CUtensorMap* mk = own ? tmK : tmKp;
        const CUtensorMap* mv = own ? tmV : tmVp;
        auto load = [&](const CUtensorMap* map, int b) -> bool {
            const uint32_t st = c % C::kStages, ph = (c / C::kStages) & 1;
            if (!mbar_wait<true>(&bars[C::kEmpty + st], ph ^ 1, ab, 62)) return false;
            mbar_arrive_expect_tx(&bars[C::kFull + st], C::kTile);
            armed[st] = (int32_t)ph;
#pragma unroll
            for (int hf = 0; hf < C::kHalves; ++hf)
                tma_load_2d(map, &bars[C::kFull + st], smem + C::kOffKV + st * C::kTile + hf * kHalfBytes,
                            p.hk * D + hf * 64, p.k0 + b * kBN, keep);
            ++c;
            return true;
        };
        if (w.dual) {
            for (int b = 0; b < w.nb + 2; ++b) {
                if (b >= 2 && !load(mv, b - 2)) goto unwind;
                if (b < w.nb && !load(mk, b)) goto unwind;
            }
        } else {
            for (int b = 0; b < w.nb; ++b)
                if (!load(mk, b) || !load(mv, b)) goto unwind;
        }
    }
unwind:
    // never leave the CTA with a TMA write still in flight
    if (q_armed >= 0) mbar_wait_teardown(&bars[C::kQFull], (uint32_t)q_armed);
    for (int s = 0; s < C::kStages; ++s)
        if (armed[s] >= 0) mbar_wait_teardown(&bars[C::kFull + s], (uint32_t)armed[s]);
}

// The issuer (one lane).
template <int D>
__device__ __forceinline__ void pf_mma(const PfParams& prm, uint8_t* smem, uint64_t* bars, uint32_t tmem, int seg0,
                                       int seg1, const Abort& ab) {
    using C = PfCfg<D>;
    constexpr uint32_t idesc_pv = idesc_bf16(128, D, false, true);
    constexpr uint64_t kStageDesc = C::kTile >> 4;
    const uint64_t q_desc = smem_desc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
    const uint64_t k_desc = smem_desc_sw128(smem_u32(smem + C::kOffKV), 16, 1024);
    const uint64_t v_desc = smem_desc_sw128(smem_u32(smem + C::kOffKV), kHalfBytes, 1024);
    RingAt<C::kStages> ring;
    uint32_t p_ph[2] = {0, 0}, o_ph[2] = {1, 1}, q_ph = 0;   // parities of each slot's weights, sums; queries
    for (int t = seg0; t < seg1; ++t, q_ph ^= 1) {
        const PrefixPiece p = load_piece(prm.pieces + t);
        const Walk w(p);
        const int nb = w.nb;
        const uint32_t last_keys = (uint32_t)(p.nk - (nb - 1) * kBN);
        const uint32_t idesc_full = idesc_bf16(128, 128, false, false);
        const uint32_t idesc_last = idesc_bf16(128, (last_keys + 15) & ~15u, false, false);
        const uint64_t q2 = q_desc + (w.dual ? 0 : kStageDesc);
        auto full = [&]() -> bool {
            if (!mbar_wait<true>(&bars[C::kFull + ring.st], ring.ph, ab, 64)) return false;
            tc_fence_after();
            return true;
        };
        // S of block b (in ring place ring) for slot s
        auto scores = [&](int s, int b) {
            one_scores<D>(tmem + s * 128, s ? q2 : q_desc, k_desc + ring.st * kStageDesc,
                          b == nb - 1 ? idesc_last : idesc_full);
            one_commit(&bars[C::kSFull + s]);
        };
        // O += P V of block b for slot s (V in ring place ring, landed)
        auto sums = [&](int s, int b, bool first) -> bool {
            const uint32_t sc = tmem + s * 128, oc = tmem + 256 + s * 128;
            const uint64_t vd = v_desc + ring.st * kStageDesc;
            if (first) {   // the slot's sums of its previous piece have been read
                if (!mbar_wait<true>(&bars[C::kOFree + s], o_ph[s], ab, 65)) return false;
                o_ph[s] ^= 1;
            }
            if (!mbar_wait<true>(&bars[C::kPFull + 2 * s], p_ph[s], ab, 66)) return false;
            tc_fence_after();
            const uint32_t keys = b == nb - 1 ? last_keys : 128u;
            one_sums(oc, sc, sc + 16, vd, idesc_pv, (keys + 15) >> 4, first ? 0 : 1);
            if (!mbar_wait<true>(&bars[C::kPFull + 2 * s + 1], p_ph[s], ab, 68)) return false;
            p_ph[s] ^= 1;
            if (keys > 64) {
                tc_fence_after();
                one_sums(oc, sc + 32, sc + 48, vd + mnmajor_step(4), idesc_pv, (keys - 49) >> 4, 1);
            }
            return true;
        };
        if (!mbar_wait<true>(&bars[C::kQFull], q_ph, ab, 63)) return;
        if (!w.dual) {
            for (int b = -1; b < nb; ++b) {
                const RingAt<C::kStages> v = ring;   // V of block b, then K of block b + 1
                if (b >= 0) {
                    if (!full() || !sums(0, b, b == 0)) return;
                    ring.next();
                }
                if (b + 1 < nb) {
                    if (!full()) return;
                    scores(0, b + 1);
                } else {
                    one_commit(&bars[C::kOFull]);
                }
                const RingAt<C::kStages> k = ring;
                if (b >= 0) {
                    ring = v;
                    if (!sums(1, b, b == 0)) return;
                    one_commit(&bars[C::kEmpty + v.st]);
                    ring = k;
                }
                if (b + 1 < nb) {
                    scores(1, b + 1);
                    one_commit(&bars[C::kEmpty + ring.st]);
                    if (b + 2 == nb) one_commit(&bars[C::kQEmpty]);   // the queries may be replaced
                    ring.next();
                } else {
                    one_commit(&bars[C::kOFull + 1]);
                }
            }
        } else {
            for (int b = -2; b < nb; ++b) {
                const int s = b & 1;
                if (b >= 0) {
                    if (!full() || !sums(s, b, b < 2)) return;
                    one_commit(&bars[C::kEmpty + ring.st]);
                    ring.next();
                    if (b + 2 >= nb) one_commit(&bars[C::kOFull + s]);
                }
                if (b + 2 < nb) {
                    if (!full()) return;
                    scores(s, b + 2);
                    one_commit(&bars[C::kEmpty + ring.st]);
                    ring.next();
                    if (b + 3 == nb) one_commit(&bars[C::kQEmpty]);
                }
            }
        }
    }
}

// 2^t of two values t <= 126 in multiply-adds: t = n + f with |f| <= 1/2
// (adding 1.5 * 2^23 leaves n in the low bits), a minimax polynomial of degree
// 4 for 2^f (of the relative error, by exchange, then rounded to float32 with the
// mean near 0: at most 2.7e-6, mean 4e-8, against the weights' rounding
// to bf16 of 2^-8), n added to the exponent; below -126, 0.
__device__ __forceinline__ float2 exp2_poly(float2 t) {
    constexpr float kMagic = 12582912.0f;
    const uint64_t x = f2_make(t.x, t.y), one = f2_make(1.0f, 1.0f);
    const uint64_t r = f2_fma(x, one, f2_make(kMagic, kMagic));
    const uint64_t n = f2_fma(r, one, f2_make(-kMagic, -kMagic));
    const uint64_t f = f2_fma(n, f2_make(-1.0f, -1.0f), x);
    uint64_t p = f2_fma(f, f2_make(0.009570101276f, 0.009570101276f), f2_make(0.05591785908f, 0.05591785908f));
    p = f2_fma(p, f, f2_make(0.2402474433f, 0.2402474433f));
    p = f2_fma(p, f, f2_make(0.6931217909f, 0.6931217909f));
    p = f2_fma(p, f, f2_make(0.9999992847f, 0.9999992847f));
    const float2 pf = f2_split(p), rf = f2_split(r);
    const float a = __uint_as_float(__float_as_uint(pf.x) + (__float_as_uint(rf.x) << 23));
    const float b = __uint_as_float(__float_as_uint(pf.y) + (__float_as_uint(rf.y) << 23));
    return make_float2(t.x < -126.0f ? 0.0f : a, t.y < -126.0f ? 0.0f : b);
}

template <int D, int ACT>
__device__ __forceinline__ void pf_rows(const PfParams& prm, uint8_t* smem, uint64_t* bars, uint32_t tmem,
                                        int seg0, int seg1, const Abort& ab) {
    using C = PfCfg<D>;
    constexpr bool kSm = ACT == kSoftmax;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t sc = trow + s * 128, oc = trow + 256 + s * 128;
    const bool flip = kSm && prm.alpha < 0.0f;
    ActScale ks = act_scale<ACT>(prm.alpha);
    if (kSm) {   // (a zero scale would make NaN of masked scores)
        ks.c0 = fabsf(ks.c0);
        if (ks.c0 < 1e-30f) ks.c0 = 1e-30f;
    }
    uint32_t base = 0, items = 0, used = 0;
    for (int t = seg0; t < seg1; ++t) {
        const PrefixPiece p = load_piece(prm.pieces + t);
        const Walk w(p);
        const int n = w.blocks(s);
        const int part = s ? p.part1 : p.part0;
        const int shift = s && !w.dual ? p.nA : 0;              // tokens before this slot's
        const int nrows = (s && !w.dual ? p.nB : p.nA) * prm.r;
        const bool real = row < nrows;
        const bool banded = (p.flags & kPieceOwn) && prm.windowed;
        const int ipos = p.i0 + shift + row / prm.r;
        float ref = -INFINITY, sum = 0.0f;
        for (int j = 0; j < n; ++j) {
            const int b = w.block(s, j);
            const int nv = min(kBN, p.nk - b * kBN);
            const bool cut = nv < kBN || banded;
            if (!wg_wait<true>(&bars[C::kSFull + s], (items + j) & 1, ab, 71)) return;
            tc_fence_after();
            uint32_t x[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(sc + c * 32, *reinterpret_cast<uint32_t(*)[32]>(x + c * 32));
            tmem_ld_wait();
            if (flip) {
#pragma unroll
                for (int e = 0; e < 128; ++e) x[e] ^= 0x80000000u;
            }
            if (cut) {
                int lo = 0, hi = nv;   // columns this row sees
                if (banded) {
                    const int at = ipos - (p.j0 + b * kBN);
                    hi = min(hi, at + 1);
                    lo = at >= prm.window ? at - prm.window + 1 : 0;
                }
#pragma unroll
                for (int e = 0; e < 128; ++e)
                    if (e < lo || e >= hi) x[e] = 0xff800000u;   // -inf
            }
            if constexpr (kSm) {
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 128; e += 8)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        m4[u] = max3_nan(m4[u], __uint_as_float(x[e + u]), __uint_as_float(x[e + 4 + u]));
                const float top = max3_nan(max3_nan(m4[0], m4[1], m4[2]), m4[3], m4[3]) * ks.c0;
                if (top != top) {   // (exp2_poly would take a NaN for a number)
                    sum = top;
                    if (ref == -INFINITY) ref = 0.0f;   // the part counts
                }
                const bool up = real && top > ref + kRise;   // also from -inf
                if (__any_sync(0xffffffffu, up)) {
                    const float nref = up ? top : ref;
                    const float f = up ? ex2_approx(ref - nref) : 1.0f;   // 0 from -inf
                    ref = nref;
                    sum *= f;
                    if (j > 0) {
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(oc + c, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st16(oc + c, o);
                        }
                        tmem_st_wait();
                    }
                }
            }
            const float nref = kSm ? (ref == -INFINITY ? 0.0f : -ref) : 0.0f;
            uint64_t sum2 = f2_make(0.0f, 0.0f);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int c = 2 * h; c < 2 * h + 2; ++c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float p0, p1;
                        const float s0 = __uint_as_float(x[c * 32 + e]), s1 = __uint_as_float(x[c * 32 + e + 1]);
                        if constexpr (kSm) {
                            const float2 tt = f2_split(
                                f2_fma(f2_make(s0, s1), f2_make(ks.c0, ks.c0), f2_make(nref, nref)));
                            if (e % 6 == 4) {   // one pair of three

                                const float2 y = exp2_poly(tt);
                                p0 = y.x;
                                p1 = y.y;
                            } else {
                                p0 = ex2_approx(tt.x);
                                p1 = ex2_approx(tt.y);
                            }
                            sum2 = f2_fma(f2_make(p0, p1), f2_make(1.0f, 1.0f), sum2);
                        } else {
                            act_s2<ACT>(s0, s1, ks, p0, p1);
                            if (cut) {
                                if (s0 == -INFINITY) p0 = 0.0f;
                                if (s1 == -INFINITY) p1 = 0.0f;
                            }
                        }
                        pk[e >> 1] = pack_bf16x2(p0, p1);
                    }
                    tmem_st16(sc + c * 16, pk);
                }
                tmem_st_wait();
                const int nh = nv - 64 * h;
                if (nh > 0 && nh < 64 && (nh & 15)) {
                    // V rows behind the last key, inside its 16-row step
                    const int at = w.v_at(b);
                    const uint32_t st = (base + (uint32_t)at) % C::kStages, ph = ((base + (uint32_t)at) / C::kStages) & 1;
                    if (!wg_wait<true>(&bars[C::kFull + st], ph, ab, 72)) return;
                    uint8_t* v = smem + C::kOffKV + st * C::kTile;
                    const int cnt = ((nv + 15) & ~15) - nv;
                    for (int i = row; i < cnt * (D / 8); i += 128) {
                        const int rr = nv + i / (D / 8), ch = i % (D / 8);
                        *reinterpret_cast<uint4*>(v + (ch >> 3) * kHalfBytes + rr * 128 + ((ch & 7) << 4)) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                mbar_arrive(&bars[C::kPFull + 2 * s + h]);
            }
            if constexpr (kSm) {
                const float2 a = f2_split(sum2);
                sum += a.x + a.y;
            }
        }
        if (n > 0) {
            if (!wg_wait<true>(&bars[C::kOFull + s], used & 1, ab, 73)) return;
            tc_fence_after();
            float4* out = reinterpret_cast<float4*>(prm.parts) + (int64_t)part * (D / 4) + row;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(oc + c * 32, o);
                tmem_ld_wait();
                if (real) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        out[(c * 8 + e) * nrows] =
                            make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                        __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
                }
            }
            tc_fence_before();
            mbar_arrive(&bars[C::kOFree + s]);
            if (kSm && real) reinterpret_cast<float2*>(prm.ml)[(int64_t)part + row] = make_float2(ref, sum);
            items += n;
            used += 1;
        }
        base += 2 * (uint32_t)w.nb;
    }
}

template <int D, int ACT>
__global__ void __launch_bounds__(kThreads, 1)
prefix_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmKp,
                  const __grid_constant__ CUtensorMap tmVp, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const PfParams prm) {
    using C = PfCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_let_next();
    const int seg0 = prm.seg[blockIdx.x], seg1 = prm.seg[blockIdx.x + 1];
    if (seg0 == seg1) {   // the whole CTA
        grid_wait_previous();
        return;
    }
    if (threadIdx.x == 0) {
        for (int b = 0; b < C::kNumBars; ++b) {
            const bool rows = (b >= C::kPFull && b < C::kPFull + 4) || (b >= C::kOFree && b < C::kOFree + 2);
            mbar_init(&bars[b], rows ? 128u : 1u);
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmKp);
        tma_prefetch_desc(&tmVp);
    }
    if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Abort ab{abort_flag, prm.err, prm.wait_ns};
    // 384 threads start with 168 registers: 88 + 2 * 208 a triple
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 0) {
            if (lane == 0) pf_producer<D>(&tmQ, &tmKp, &tmVp, &tmK, &tmV, prm, smem, bars, seg0, seg1, ab);
            __syncwarp();
        } else if (warp == 1) {
            if (elect_one()) {
                pf_mma<D>(prm, smem, bars, tmem, seg0, seg1, ab);
                // all of its products complete before TMEM is released
                one_commit(&bars[C::kMmaDone]);
                mbar_wait_teardown(&bars[C::kMmaDone], 0);
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        pf_rows<D, ACT>(prm, smem, bars, tmem, seg0, seg1, ab);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    grid_wait_previous();   // (the own keys' kernel, which nothing here reads)
}

template <int D, int ACT>
gdpa_status launch(PrefixPlan& p, const CUtensorMap* m, const PfParams& prm, cudaStream_t st) {
    auto kern = prefix_fwd_kernel<D, ACT>;
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(kern, PfCfg<D>::kSmem, p.device, done)) return GDPA_ERR_CUDA;
    const bool ok = launch_kernel(kern, dim3((unsigned)p.S), kThreads, PfCfg<D>::kSmem, st, p.chain > 0, m[0], m[1],
                                  m[2], m[3], m[4], prm);
    p.launches += 1;
    p.chain += 1;
    return ok ? GDPA_OK : GDPA_ERR_CUDA;
}

}  // namespace

gdpa_status launch_prefix_tc_fwd(PrefixPlan& p, const PrefixIO& io, cudaStream_t st) {
    if (p.seg[p.S] == 0) return GDPA_OK;
    CUtensorMap m[5];
    const uint64_t krow = (uint64_t)p.Hkv * p.d;
    // tensors without rows are never loaded from: any map will do
    const void* kp = p.Tp ? io.kp : io.k;
    const void* vp = p.Tp ? io.vp : io.v;
    const void* k = p.Tkv ? io.k : io.kp;
    const void* v = p.Tkv ? io.v : io.vp;
    const uint64_t np = p.Tp ? p.Tp : p.Tkv, nk = p.Tkv ? p.Tkv : p.Tp;
    if (!tc::make_tmap_rows(&m[0], io.q, p.Tq, p.H, p.d, p.r, p.tpt) ||
        !tc::make_tmap_bf16(&m[1], kp, np, krow, 128) || !tc::make_tmap_bf16(&m[2], vp, np, krow, 128) ||
        !tc::make_tmap_bf16(&m[3], k, nk, krow, 128) || !tc::make_tmap_bf16(&m[4], v, nk, krow, 128))
        return GDPA_ERR_CUDA;
    PfParams prm;
    prm.pieces = p.dev_pieces();
    prm.seg = p.dev_seg();
    prm.parts = p.d_parts;
    prm.ml = p.d_ml;
    prm.r = p.r;
    prm.windowed = p.mask == GDPA_MASK_CAUSAL_WINDOW;
    prm.window = p.window;
    prm.q_bytes = p.tpt * p.r * p.d * 2;
    prm.alpha = io.alpha;
    prm.err = p.dev_err();
    prm.wait_ns = tc::wait_limit_ns(p.wait_limit_us);
    prm.stall = p.stall == 1;
    gdpa_status s = GDPA_OK;
    if (p.d == 128) {
        if (io.act == kSoftmax)
            s = launch<128, kSoftmax>(p, m, prm, st);
        else
            GDPA_DISPATCH_ACT(io.act, A, s = launch<128, A>(p, m, prm, st))
    } else {
        if (io.act == kSoftmax)
            s = launch<64, kSoftmax>(p, m, prm, st);
        else
            GDPA_DISPATCH_ACT(io.act, A, s = launch<64, A>(p, m, prm, st))
    }
    return s;
}

}  // namespace gdpa
