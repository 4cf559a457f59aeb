// Shared-prefix attention forward on the tensor cores (bf16 rows, d = 64 or
// 128): the parts of every row tile, for the merge to join.
//
// One CTA per planned share walks its pieces.  A piece is one or two row
// tiles (packed token by token, query heads of one key head side by side; a
// 3-D TMA box does the packing) against a run of keys.  Two slots, each with
// its own score and sum columns in TMEM (128 + d) and two warpgroups, which
// take 64 keys of a block each, a thread a row:
//   two tiles: slot s holds tile s, both read the same key blocks;
//   one tile:  slot s takes the key blocks s, s + 2, ... of the same rows and
//              gives a part of its own.
// Warp 0 loads (TMA): the piece's query tiles, then K and V blocks through
// one ring, in the order in which the tensor core takes them.  Warp 1 issues
// S = Q K^T and O += P V: one slot's P V and next S run while the other's
// weights are computed; the P V of a block's first 64 keys starts when their
// warpgroup is done.  (An issuer per slot was no faster: a slot's chain of
// scores, weights and sums is what takes the time.)  The warpgroups (a row's two threads
// exchange their maxima through shared memory) keep the row maximum as a
// reference that only moves when it would be passed by more than 8 (in
// base 2: weights stay below 2^8), so O is rescaled in TMEM a few times a
// piece rather than at every block; that S is complete says that the P V
// before it is (they are issued in that order and commits follow all work
// issued before), so the rescale needs no wait of its own.
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

constexpr int kThreads = 64 + 512;
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
        kOFull = kPFull + 4, kOFree = kOFull + 2, kMeet = kOFree + 2, kMmaDone = kMeet + 2, kNumBars
    };
    static constexpr int kOffXchg = kOffBar + kNumBars * 8 + 16;   // [slot][half][128] maxima
    static constexpr int kSmem = kOffXchg + 2 * 2 * 128 * 4;       // no room for an alignment gap
    static_assert(kSmem <= 232448, "shared memory of a block");
};

struct PfParams {
    const PrefixPiece* pieces;
    const int32_t* seg;
    float* parts;
    float* ml;
    int r, tpt, windowed, window;
    int q_bytes;      // bytes of one query tile's load
    float alpha;
    int32_t* err;
    uint64_t wait_ns;
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
    __device__ __forceinline__ int k_at(int b) const { return dual ? (b < 2 ? b : 2 * b - 1) : 2 * b; }
    __device__ __forceinline__ int v_at(int b) const { return dual ? min(b + 2, nb) + b : 2 * b + 1; }
};

template <int D>
__device__ void pf_producer(const CUtensorMap* tmQ, const CUtensorMap* tmKp, const CUtensorMap* tmVp,
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
        if (!mbar_wait(&bars[C::kQEmpty], (n & 1) ^ 1, ab, 61)) goto unwind;
        mbar_arrive_expect_tx(&bars[C::kQFull], (uint32_t)(prm.q_bytes * (p.nB > 0 ? 2 : 1)));
        q_armed = (int32_t)(n & 1);
        for (int half = 0; half < (p.nB > 0 ? 2 : 1); ++half)
#pragma unroll
            for (int hf = 0; hf < C::kHalves; ++hf)
                tma_load_3d(tmQ, &bars[C::kQFull], smem + C::kOffQ + half * C::kTile + hf * kHalfBytes,
                            hf * 64, p.hk * prm.r, p.tok + half * p.nA, once);
        const bool own = p.flags & kPieceOwn;
        const CUtensorMap* mk = own ? tmK : tmKp;
        const CUtensorMap* mv = own ? tmV : tmVp;
        auto load = [&](const CUtensorMap* map, int b) -> bool {
            const uint32_t st = c % C::kStages, ph = (c / C::kStages) & 1;
            if (!mbar_wait(&bars[C::kEmpty + st], ph ^ 1, ab, 62)) return false;
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

template <int D>
__device__ void pf_mma(const PfParams& prm, uint8_t* smem, uint64_t* bars, uint32_t tmem, int seg0, int seg1,
                       const Abort& ab) {
    using C = PfCfg<D>;
    constexpr uint32_t idesc_pv = idesc_bf16(128, D, false, true);
    uint32_t base = 0, items0 = 0, items1 = 0, used0 = 0, used1 = 0;   // ring places; blocks, pieces of a slot
    tmem = (uint32_t)uniform((int)tmem);
    const uint32_t kv = smem_u32(smem + C::kOffKV);
    for (int t = seg0; t < seg1; ++t) {
        PrefixPiece p = load_piece(prm.pieces + t);
        p.nk = uniform(p.nk);
        p.flags = uniform(p.flags);
        const Walk w(p);
        if (!wg_wait(&bars[C::kQFull], (uint32_t)(t - seg0) & 1, ab, 63)) goto drain;
        // step j: each slot's P V of its block j - 1 (behind the first), then
        // its S of block j (before the last)
#pragma unroll 1
        for (int x = 0; x < 2 * (w.n0 + 1); ++x) {
            const int s = x & 1, j = (x >> 1) - 1, n = w.blocks(s);
            const uint32_t scol = tmem + s * 128, ocol = tmem + 256 + s * 128;
            const bool frees = w.dual || s == 1;   // the last slot to read a block
            if (j >= 0 && j < n) {
                const int b = w.block(s, j);
                const uint32_t at = base + (uint32_t)w.v_at(b), st = at % C::kStages;
                const uint32_t keys = (uint32_t)min(kBN, p.nk - b * kBN);
                const uint64_t vd = smem_desc_sw128(kv + st * C::kTile, kHalfBytes, 1024);
                const uint32_t ph = ((s ? items1 : items0) + j) & 1;
                // the slot's sums of its previous piece have been read
                if (j == 0 && !wg_wait(&bars[C::kOFree + s], ((s ? used1 : used0) & 1) ^ 1, ab, 65)) goto drain;
                if (!wg_wait(&bars[C::kFull + st], (at / C::kStages) & 1, ab, 67) ||
                    !wg_wait(&bars[C::kPFull + 2 * s], ph, ab, 66))
                    goto drain;
                tc_fence_after();
                mma_sums(ocol, scol, scol + 16, vd, idesc_pv, min(4u, (keys + 15) >> 4), j > 0);
                if (!wg_wait(&bars[C::kPFull + 2 * s + 1], ph, ab, 68)) goto drain;
                if (keys > 64) {
                    tc_fence_after();
                    mma_sums(ocol, scol + 64, scol + 80, vd + mnmajor_step(4), idesc_pv, (keys - 49) >> 4, 1);
                }
                if (frees) mma_commit(&bars[C::kEmpty + st]);
                if (j == n - 1) mma_commit(&bars[C::kOFull + s]);
            }
            if (j + 1 < n) {
                const int b = w.block(s, j + 1);
                const uint32_t at = base + (uint32_t)w.k_at(b), st = at % C::kStages;
                const uint32_t keys16 = (uint32_t)(min(kBN, p.nk - b * kBN) + 15) & ~15u;
                if (!wg_wait(&bars[C::kFull + st], (at / C::kStages) & 1, ab, 64)) goto drain;
                tc_fence_after();
                mma_scores<D>(scol, smem_desc_sw128(smem_u32(smem + C::kOffQ + (s && !w.dual ? C::kTile : 0)), 16, 1024),
                              smem_desc_sw128(kv + st * C::kTile, 16, 1024), idesc_bf16(128, keys16, false, false));
                mma_commit(&bars[C::kSFull + s]);
                if (frees) mma_commit(&bars[C::kEmpty + st]);
                // the piece's last S: its queries may be replaced
                if (b == w.nb - 1 && frees) mma_commit(&bars[C::kQEmpty]);
            }
        }
        items0 += w.n0;
        items1 += w.n1;
        used0 += w.n0 > 0;
        used1 += w.n1 > 0;
        base += 2 * (uint32_t)w.nb;
    }
drain:
    mma_commit(&bars[C::kMmaDone]);
    mbar_wait_teardown(&bars[C::kMmaDone], 0);
}

template <int D, int ACT>
__device__ void pf_rows(const PfParams& prm, uint8_t* smem, uint64_t* bars, uint32_t tmem, int seg0,
                        int seg1, const Abort& ab) {
    using C = PfCfg<D>;
    constexpr bool kSm = ACT == kSoftmax;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = (warp - 2) >> 3, h = ((warp - 2) >> 2) & 1;   // slot, half of the keys
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const int tid = (int)(threadIdx.x - 64) & 127;
    const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t sc = trow + s * 128, oc = trow + 256 + s * 128;
    float* xchg = reinterpret_cast<float*>(smem + C::kOffXchg) + s * 256;
    const bool flip = kSm && prm.alpha < 0.0f;
    ActScale ks = act_scale<ACT>(prm.alpha);
    if (kSm) {   // (a zero scale would make NaN of masked scores)
        ks.c0 = fabsf(ks.c0);
        if (ks.c0 < 1e-30f) ks.c0 = 1e-30f;
    }
    uint32_t base = 0, items = 0, used = 0, met = 0;
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
            const int nv = min(kBN, p.nk - b * kBN) - 64 * h;   // this half's keys, may be <= 0
            const bool cut = nv < 64 || banded;
            int lo = 0, hi = nv;   // columns this row sees
            if (banded) {
                const int at = ipos - (p.j0 + b * kBN + 64 * h);
                hi = min(hi, at + 1);
                lo = at >= prm.window ? at - prm.window + 1 : 0;
            }
            if (!wg_wait(&bars[C::kSFull + s], (items + j) & 1, ab, 71)) return;
            tc_fence_after();
            // 32 scores from column c on, those the row does not see as -inf
            auto scores = [&](int c, uint32_t (&x)[32]) {
                tmem_ld32(sc + 64 * h + c, x);
                tmem_ld_wait();
                if (flip) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] ^= 0x80000000u;
                }
                if (cut) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (c + e < lo || c + e >= hi) x[e] = 0xff800000u;
                }
            };
            if constexpr (kSm) {
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                for (int c = 0; c < 64; c += 32) {
                    if (c >= nv) break;
                    uint32_t x[32];
                    scores(c, x);
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
#pragma unroll
                        for (int u = 0; u < 4; ++u) m4[u] = fmaxf(m4[u], __uint_as_float(x[e + u]));
                }
                float top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                // the row's other 64 keys: both threads go on with the same
                // maximum (S of the next block comes only after both have
                // read, so one buffer is enough)
                xchg[h * 128 + row] = top;
                mbar_arrive(&bars[C::kMeet + s]);
                if (!wg_wait(&bars[C::kMeet + s], met++ & 1, ab, 74)) return;
                top = fmaxf(top, xchg[(h ^ 1) * 128 + row]) * ks.c0;
                const bool up = real && top > ref + kRise;   // also from -inf
                if (__any_sync(0xffffffffu, up)) {
                    const float nref = up ? top : ref;
                    const float f = up ? ex2_approx(ref - nref) : 1.0f;   // 0 from -inf
                    ref = nref;
                    sum *= f;
                    if (j > 0) {   // each thread rescales its half of the row's sums
#pragma unroll 1
                        for (int c = h * (D / 2); c < (h + 1) * (D / 2); c += 16) {
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
                tc_fence_before();
            }
            // this half's sums are ready for the other half's product
            mbar_arrive(&bars[C::kPFull + 2 * s + (h ^ 1)]);
            const float nref = kSm ? (ref == -INFINITY ? 0.0f : -ref) : 0.0f;
            uint64_t sum2 = f2_make(0.0f, 0.0f);
#pragma unroll 1
            for (int c = 0; c < 64; c += 32) {
                if (c >= nv) break;
                uint32_t x[32], pk[16];
                scores(c, x);
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    float p0, p1;
                    const float s0 = __uint_as_float(x[e]), s1 = __uint_as_float(x[e + 1]);
                    if constexpr (kSm) {
                        const float2 tt = f2_split(f2_fma(f2_make(s0, s1), f2_make(ks.c0, ks.c0), f2_make(nref, nref)));
                        p0 = ex2_approx(tt.x);
                        p1 = ex2_approx(tt.y);
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
                tmem_st16(sc + 64 * h + c / 2, pk);   // over this thread's own scores, already read
            }
            if constexpr (kSm) {
                const float2 a = f2_split(sum2);
                sum += a.x + a.y;
            }
            tmem_st_wait();
            if (nv > 0 && nv < 64 && (nv & 15)) {
                // V rows behind the last key, inside its 16-row step
                const int at = w.v_at(b);
                const uint32_t st = (base + (uint32_t)at) % C::kStages, ph = ((base + (uint32_t)at) / C::kStages) & 1;
                if (!wg_wait(&bars[C::kFull + st], ph, ab, 72)) return;
                uint8_t* v = smem + C::kOffKV + st * C::kTile;
                const int n0 = 64 * h + nv, cnt = ((nv + 15) & ~15) - nv;
                for (int i = tid; i < cnt * (D / 8); i += 128) {
                    const int rr = n0 + i / (D / 8), ch = i % (D / 8);
                    *reinterpret_cast<uint4*>(v + (ch >> 3) * kHalfBytes + rr * 128 + ((ch & 7) << 4)) =
                        make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
            }
            tc_fence_before();
            mbar_arrive(&bars[C::kPFull + 2 * s + h]);
        }
        if (n > 0) {
            if (!wg_wait(&bars[C::kOFull + s], used & 1, ab, 73)) return;
            tc_fence_after();
            float4* out = reinterpret_cast<float4*>(prm.parts) + (int64_t)part * (D / 4) + row;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const int c0 = h * (D / 2) + c * 32;
                uint32_t o[32];
                tmem_ld32(oc + c0, o);
                tmem_ld_wait();
                if (real) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        out[(c0 / 4 + e) * nrows] =
                            make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                        __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
                }
            }
            if constexpr (kSm) {
                // the row's sum over both halves of the keys, through a column
                // of O that has been read
                if (h == 1) {
                    tmem_st1(oc + D - 1, __float_as_uint(sum));
                    tmem_st_wait();
                }
                tc_fence_before();
                mbar_arrive(&bars[C::kMeet + s]);
                if (!wg_wait(&bars[C::kMeet + s], met++ & 1, ab, 75)) return;
                tc_fence_after();
                if (h == 0) {
                    const float other = __uint_as_float(tmem_ld1(oc + D - 1));
                    tmem_ld_wait();
                    if (real) reinterpret_cast<float2*>(prm.ml)[(int64_t)part + row] = make_float2(ref, sum + other);
                }
            }
            tc_fence_before();
            mbar_arrive(&bars[C::kOFree + s]);
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
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int seg0 = prm.seg[blockIdx.x], seg1 = prm.seg[blockIdx.x + 1];
    if (seg0 == seg1) return;   // the whole CTA
    if (smem_u32(smem) & 1023u) {   // the swizzled tiles need the alignment declared above
        if (threadIdx.x == 0) atomicCAS(prm.err, 0, kDevBad);
        return;
    }
    if (threadIdx.x == 0) {
        for (int b = 0; b < C::kNumBars; ++b) {
            const bool rows = (b >= C::kPFull && b < C::kPFull + 4) || (b >= C::kOFree && b < C::kMeet + 2);
            mbar_init(&bars[b], rows ? 256u : 1u);
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
    if (warp == 0) {
        if (lane == 0) pf_producer<D>(&tmQ, &tmKp, &tmVp, &tmK, &tmV, prm, smem, bars, seg0, seg1, ab);
        __syncwarp();
    } else if (warp == 1) {
        pf_mma<D>(prm, smem, bars, tmem, seg0, seg1, ab);
        __syncwarp();
    } else {
        pf_rows<D, ACT>(prm, smem, bars, tmem, seg0, seg1, ab);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D, int ACT>
gdpa_status launch(PrefixPlan& p, const CUtensorMap* m, const PfParams& prm, cudaStream_t st) {
    auto kern = prefix_fwd_kernel<D, ACT>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, PfCfg<D>::kSmem) !=
        cudaSuccess)
        return GDPA_ERR_CUDA;
    kern<<<p.S, kThreads, PfCfg<D>::kSmem, st>>>(m[0], m[1], m[2], m[3], m[4], prm);
    p.launches += 1;
    return cudaGetLastError() == cudaSuccess ? GDPA_OK : GDPA_ERR_CUDA;
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
    prm.tpt = p.tpt;
    prm.windowed = p.mask == GDPA_MASK_CAUSAL_WINDOW;
    prm.window = p.window;
    prm.q_bytes = p.tpt * p.r * p.d * 2;
    prm.alpha = io.alpha;
    prm.err = p.dev_err();
    prm.wait_ns = tc::wait_limit_ns(0);
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
