// Attention over the history cache for many query rows a key head (bf16, d = 64
// or 128), on tcgen05: whole chunks of new events, wide trees, many heads a key
// head.
//
// With more than a few rows a cached byte meets so many of them that products,
// not bytes, bound the work.  A tile is up to 256 rows against a segment's
// events in blocks of 128, in two slots of TMEM (128 columns of scores and d of
// sums each), a warpgroup each, a thread a row:
//   more than 128 rows: slot s holds rows 128 s .. of the tile, both read the
//                       same blocks;
//   else:               slot s takes the blocks s, s + 2, ... of the same rows,
//                       and slot 0's threads join the two at the end.
// One warp loads: each group of 16 events is a plain bulk copy (the cache holds
// rows in the operands' swizzle), its page looked up 32 groups ahead.  One lane
// issues S = Q K^T and O += P V; the order of loads and products and the lazily
// moved reference are shared-prefix attention's (prefix_tc_fwd.cu says why).
//
// 8-bit caches.  Keys are multiplied as they are (kind::f8f6f4): a query row,
// scaled by a power of two to below 256, is split into E4M3 codes and E5M2 codes
// of what they leave, at most 8 units of bf16's last place, which 3 bits hold
// (elements below 2^-13 of the largest lose bits, at most 2^-21 of it): two
// products of double rate; the keys' powers of two are applied to the scores.
// Values are expanded to bf16 by the worker warps, exactly (a code has 4 bits): its 7 bits behind the sign moved to bf16's place are the
// value times 2^-120, subnormal codes included, and one bf16 product by 2^(e +
// 120) (two where that leaves bf16's range) gives it.  (Keys expanded as well:
// the workers bound the kernel, 480 us for 8 x 512 rows on 16384 events.)
//
// Those 8 x 512 rows (4 heads a key head): bf16 220 us with the joining, 1.27
// PFLOP/s, bound by a slot's chain of scores, weights and sums (tensor pipe 60%
// busy); 8-bit 317 us: the row threads' instructions beside the workers'.
//
// A block that some row does not see is masked by selection, event by event, and
// workers clear the infinities and NaNs in its values (0 times them would be
// NaN); that this happened is noted, and at the end the rows that do see such
// events have them added.
#pragma once

#include "cache_attn.cuh"
#include "prefix_tc.cuh"

namespace gdpa {
namespace cache_tc {

using namespace tc;

constexpr int kHalfBytes = 128 * 128;
constexpr uint32_t kTmemCols = 512;
constexpr float kRise = 8.0f;   // the reference follows a maximum this far above it

struct Misc {
    uint32_t tmem;
    int abort_flag;
    uint8_t odd[8];      // by segment with blocks: its tag, if workers cleared something
    uint8_t gone[16];    // by block: groups without a page
};
// Workers are at most as many segments ahead of the row threads as there are stages
// of values (4): a place is not another's while it is needed.  (A tag that was left
// 1024 segments ago only costs time.)
__device__ __forceinline__ uint8_t odd_tag(uint32_t segment) { return (uint8_t)((segment >> 3 & 127u) + 1u); }

// Blocks of a segment, as both slots take them, and which are masked.
struct Walk {
    int nb, n1, n;
    int open0, open1;   // blocks of which every row sees everything
    bool dual;
    __device__ __forceinline__ void set(const AttnArgs& a, const Segment& g) {
        n = g.n;
        nb = (n + 7) >> 3;
        dual = g.rows <= 128;
        n1 = dual ? nb >> 1 : nb;
        const int i0 = g.rho0 / a.G, i1 = (g.rho0 + g.rows - 1) / a.G;
        // events below hi that are at or above lo are seen by all rows
        const int hi = min(g.s.end, g.s.start + (a.mask == GDPA_CACHE_CAUSAL ? i0 + 1 : 0));
        const int lo = a.window > 0 ? max(0, g.s.start + (a.mask == GDPA_CACHE_HISTORY ? 0 : i1) - a.window + 1) : 0;
        // in groups of the segment, behind the sinks
        const int from = max(g.na, (lo + 15) / 16 - g.b0), to = min(n, hi / 16 - g.b0);
        open0 = (from + 7) >> 3;
        open1 = to >> 3;
    }
    __device__ __forceinline__ int blocks(int s) const { return s ? n1 : dual ? nb - n1 : nb; }
    __device__ __forceinline__ int groups(int b) const { return min(8, n - 8 * b); }
    __device__ __forceinline__ bool masked(int b) const { return b < open0 || b >= open1; }
    // the tiles in the order of the ring: f(block, is V) until it returns false.
    // more than 128 rows: K0 V0 K1 V1 ...; else: K0 K1 V0 K2 V1 K3 ...
    template <typename F>
    __device__ __forceinline__ bool tiles(F f) const {
        const int lag = dual ? 2 : 1;
        for (int b = 0; b < nb + lag; ++b) {
            if (dual) {
                if (b >= 2 && !f(b - 2, true)) return false;
                if (b < nb && !f(b, false)) return false;
            } else if (b < nb) {
                if (!f(b, false) || !f(b, true)) return false;
            }
        }
        return true;
    }
};

// A warp's place in the work, in shared memory: in registers it would be spilled,
// and with this much shared memory taken local memory is as far as L2 (the row
// threads' 250 instructions a block took 6000 cycles).
struct Place {
    Share sh;
    Segment g;
    Walk w;
};

// The next segment; false: no more.  (Whole warps.)
__device__ __forceinline__ bool advance(const AttnArgs& a, Place& p) {
    Share sh = p.sh;
    Segment g;
    g.rows = 0;
    if (sh.more()) g = next_segment(a, sh);
    Walk w;
    if (g.rows > 0) w.set(a, g);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        p.sh = sh;
        p.g = g;
        p.w = w;
    }
    __syncwarp();
    return g.rows > 0;
}

template <int D, bool FP8>
struct Cfg {
    static constexpr int kHalves = D / 64;
    static constexpr int kTile = 128 * D * 2;                // 128 rows in bf16
    static constexpr int kCodes = 128 * D;                   // ... in 8 bits
    static constexpr int kKTile = FP8 ? kCodes : kTile;
    static constexpr int kK = D == 128 ? 3 : 4;                                // stages: keys
    static constexpr int kV = D == 128 ? 2 : 4;                                // values in bf16
    static constexpr int kR = FP8 ? (D == 128 ? 2 : 3) : 0;                    // values in 8 bits
    static constexpr int kWorkers = FP8 ? 6 : 2;             // warps
    static constexpr int kRows0 = 2 + kWorkers;              // first row warp
    static constexpr int kThreads = 32 * (kRows0 + 8);
    static constexpr int kOffK = 2 * kTile;                  // behind two tiles of queries (8-bit: each as two)
    static constexpr int kOffV = kOffK + kK * kKTile;
    static constexpr int kOffR = kOffV + kV * kTile;
    static constexpr int kOffKScale = kOffR + kR * kCodes;   // bytes of the K stages, of the 8-bit V stages
    static constexpr int kOffVScale = kOffKScale + (FP8 ? kK * 128 : 0);
    static constexpr int kOffScale = kOffVScale + kR * 128;  // powers of two of the last 8 blocks' keys
    static constexpr int kOffUnit = kOffScale + (FP8 ? 8 * 512 : 0);   // 8-bit: units of the tile's rows
    static constexpr int kOffFin = kOffUnit + (FP8 ? 256 * 4 : 0);
    static constexpr bool kStageApart = FP8 && D == 64;
    static constexpr int kOffStage = kOffFin + 128 * 8;
    static constexpr int kOffPlace = kOffStage + (kStageApart ? 8 * 4096 : 0);
    static constexpr int kOffScan = kOffPlace;               // (used before the places are)
    static constexpr int kOffBar = (kOffPlace + (int)sizeof(Place) * (kThreads / 32) + 15) & ~15;
    enum {
        kQFull = 0, kQEmpty, kFin, kMmaDone, kSFull, kPFull = kSFull + 2, kOFull = kPFull + 2, kOFree = kOFull + 2,
        kKFull = kOFree + 2,             // keys have landed
        kKReady = kKFull + kK,           // 8-bit: their powers of two are in place
        kKEmpty = kKReady + kK,
        kVFull = kKEmpty + kK,           // bf16: values have landed
        kVReady = kVFull + kV,           // workers have cleaned or expanded them
        kVEmpty = kVReady + kV,
        kRFull = kVEmpty + kV, kREmpty = kRFull + kR, kNumBars = kREmpty + kR
    };
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;  // Misc
    static constexpr int kSmem = kOffMisc + 32;
    static_assert(kSmem <= 232448, "shared memory");
};

// The loader (a whole warp).
template <int D, bool FP8>
__device__ __forceinline__ void load_tiles(const AttnArgs& a, uint8_t* smem, uint64_t* bars, Misc& misc, Place& at,
                                           const Abort& ab) {
    using C = Cfg<D, FP8>;
    constexpr uint32_t kGroupBytes = FP8 ? 16 * D + 16 : 16 * D * 2;
    constexpr int NV = FP8 ? C::kR : C::kV, kVFullBar = FP8 ? C::kRFull : C::kVFull, kVEmptyBar = FP8 ? C::kREmpty : C::kVEmpty;
    const int lane = threadIdx.x & 31;
    uint32_t block0 = 0;
    RingAt<C::kK> rk;
    RingAt<NV> rv;
    uint32_t nk = 0, nv = 0;
    const Segment& g = at.g;
    const Walk& w = at.w;
    while (advance(a, at)) {
        // page of group 32 i + lane of the segment
        const auto pages = [&](int i) {
            const int j = 32 * i + lane;
            if (j >= g.n) return -1;
            const int i_page = segment_group(g, j) >> (a.c.page_log - 4);
            if (i_page >= a.w.width) return -1;   // (events behind the table are none of the segment's)
            const int p = __ldg(a.w.table + g.b * a.w.stride + i_page);
            if ((unsigned)p >= (unsigned)a.c.pages) {
                cache_bad(a.c.err, kCacheBadPage, g.b, p);
                return -1;
            }
            return p;
        };
        int prev = -1, cur = pages(0), next = pages(1), set = 0;
        const bool ok = w.tiles([&](int b, bool is_v) {
            if (!is_v && (b >> 2) > set) {
                ++set;
                prev = cur;
                cur = next;
                next = pages(set + 1);
            }
            const int ng = w.groups(b);
            const int p = __shfl_sync(0xffffffffu, (b >> 2) == set ? cur : prev, 8 * (b & 3) + (lane & 7));
            const uint32_t there = __ballot_sync(0xffffffffu, lane < ng && p >= 0);
            const uint32_t st = is_v ? rv.st : rk.st;
            uint64_t* full = &bars[(is_v ? kVFullBar : C::kKFull) + st];
            if (!__all_sync(0xffffffffu, mbar_wait<true>(&bars[(is_v ? kVEmptyBar : C::kKEmpty) + st], (is_v ? rv.ph : rk.ph) ^ 1, ab, 62))) return false;
            uint8_t* dst = smem + (!is_v ? C::kOffK + st * C::kKTile : FP8 ? C::kOffR + st * C::kCodes : C::kOffV + st * C::kTile);
            uint8_t* sc = smem + (is_v ? C::kOffVScale : C::kOffKScale) + st * 128;
            if (!is_v && lane == 0) misc.gone[(block0 + b) & 15] = (uint8_t)(~there & ((1u << ng) - 1));
            if (there != (1u << ng) - 1) {   // groups without a page hold zeros
                for (int i = 0; i < ng; ++i) {
                    if (there >> i & 1) continue;
                    if constexpr (FP8) {
                        for (int x = lane; x < D; x += 32) *reinterpret_cast<uint4*>(dst + i * 16 * D + 16 * x) = make_uint4(0, 0, 0, 0);
                        if (lane == 0) *reinterpret_cast<uint4*>(sc + 16 * i) = make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
                    } else {
                        for (int x = lane; x < 2 * D; x += 32)
                            *reinterpret_cast<uint4*>(dst + (x >> 7) * kHalfBytes + i * 2048 + (x & 127) * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (lane == 0) mbar_arrive_expect_tx(full, kGroupBytes * __popc(there));
            __syncwarp();
            // groups that lie behind each other on a page come in one copy: a copy takes
            // the warp some 80 cycles, whatever its size
            const int i = lane & 7, hf = lane >> 3, at_g = segment_group(g, 8 * b + i);
            const int e0 = (at_g * kCacheGroup) & ((1 << a.c.page_log) - 1);
            const uint32_t starts = __ballot_sync(0xffffffffu, i == 0 || i >= ng || e0 == 0 || at_g != segment_group(g, 8 * b + i - 1) + 1) & 0xff;
            if ((there & starts) >> i & 1 && hf < (FP8 ? 1 : C::kHalves)) {
                const uint32_t n = __ffs((starts | 0x100) >> (i + 1));
                const int64_t blk = (int64_t)p * a.c.heads + g.h;
                const uint8_t* src = (is_v ? a.c.v : a.c.k) + blk * a.c.block;
                if constexpr (FP8) {
                    bulk_load(full, dst + i * 16 * D, src + e0 * D, n * 16 * D);
                    bulk_load(full, sc + 16 * i, (is_v ? a.c.vs : a.c.ks) + (blk << a.c.page_log) + e0, n * 16);
                } else {
                    bulk_load(full, dst + hf * kHalfBytes + i * 2048, src + (((int64_t)hf << a.c.page_log) + e0) * 128, n * 2048);
                }
            }
            if (is_v) {
                rv.next();
                ++nv;
            } else {
                rk.next();
                ++nk;
            }
            return true;
        });
        block0 += (uint32_t)w.nb;
        if (!ok) break;
    }
    // never leave the CTA with a copy still in flight
    for (uint32_t i = nk > (uint32_t)C::kK ? nk - C::kK : 0; i < nk; ++i) mbar_wait_teardown(&bars[C::kKFull + i % C::kK], (i / C::kK) & 1);
    for (uint32_t i = nv > (uint32_t)NV ? nv - NV : 0; i < nv; ++i) mbar_wait_teardown(&bars[kVFullBar + i % NV], (i / NV) & 1);
}

// 16 codes to 16 bf16 values: m is 2^(e + 120), m2 a second factor (0: none).
__device__ __forceinline__ void expand16(const uint4& q, uint32_t m, uint32_t m2, uint4& a, uint4& b) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint32_t o[8];
    const auto times = [](uint32_t x, uint32_t y) {
        const __nv_bfloat162 z = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&x), *reinterpret_cast<__nv_bfloat162*>(&y));
        return *reinterpret_cast<const uint32_t*>(&z);
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t p = __byte_perm(w[i >> 1], 0, (i & 1) ? 0x3424 : 0x1404);   // codes in the upper bytes
        o[i] = times(((p >> 4) & 0x07f007f0u) | (p & 0x80008000u), m);
    }
    if (m2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = times(o[i], m2);
    }
    a = make_uint4(o[0], o[1], o[2], o[3]);
    b = make_uint4(o[4], o[5], o[6], o[7]);
}

// Clears the infinities and NaNs among 8 bf16 values; whether there were any.
__device__ __forceinline__ bool clear_odd(uint4& v) {
    uint32_t any = 0;
    uint32_t* p = &v.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t z = __vcmpeq2(p[i] & 0x7f807f80u, 0x7f807f80u);
        any |= z;
        p[i] &= ~z;
    }
    return any != 0;
}
// Scale bytes from which on values may be infinite: 256 * 2^120 is.
constexpr uint32_t kOddScale = 247;

// The factors of a row's codes: 2^(e + 120) in both halves of m, and a second factor
// where that leaves bf16's range (else 0).
__device__ __forceinline__ void value_factors(uint32_t s, uint32_t& m, uint32_t& m2) {
    m = (s + 120u) << 7;
    m2 = 0;
    if (s > 134u) {
        m = 254u << 7;
        m2 = (s - 7u) << 7;
        m2 |= m2 << 16;
    }
}

// A masked block's values: what is infinite or a NaN, and events behind the last one
// (whatever their memory holds), are zeros; the former are noted.  (Out of line: the
// blocks that every row sees are the loop that is to go on.)
template <int D, int NT>
__device__ __noinline__ void expand_masked(const Segment& g, int i0, const uint8_t* codes, const uint8_t* sc, uint8_t* dst, int who, int events,
                                            uint8_t* mark, uint32_t segment) {
    constexpr int kChunks = D / 16;
    const int ch = who % kChunks;
    bool odd = false;
#pragma unroll 1
    for (int e = who / kChunks; e < events; e += NT / kChunks) {
        uint4* lo = reinterpret_cast<uint4*>(dst + (ch >> 2) * kHalfBytes + e * 128 + (((2 * ch) & 7) ^ (e & 7)) * 16);
        uint4* hi = reinterpret_cast<uint4*>(dst + (ch >> 2) * kHalfBytes + e * 128 + (((2 * ch + 1) & 7) ^ (e & 7)) * 16);
        const uint4 q = *reinterpret_cast<const uint4*>(codes + cache_chunk(D, 7, e, ch));
        const uint32_t s = sc[e];
        const bool there = segment_group(g, i0 + (e >> 4)) * kCacheGroup + (e & 15) < g.s.end;
        uint32_t m, m2;
        value_factors(s, m, m2);
        if (s == 255u) odd |= there;      // a row of NaNs
        if (s == 255u || !there) m = m2 = 0;
        m |= m << 16;
        uint4 x, y;
        expand16(q, m, m2, x, y);
        if (s >= kOddScale) {
            odd |= clear_odd(x);
            odd |= clear_odd(y);
        }
        *lo = x;
        *hi = y;
    }
    if (odd) mark[segment & 7] = odd_tag(segment);
}

// The workers (warps; whole).
template <int D, bool FP8>
__device__ __forceinline__ void work_tiles(const AttnArgs& a, uint8_t* smem, uint64_t* bars, Misc& misc, Place& at,
                                           const Abort& ab) {
    using C = Cfg<D, FP8>;
    const int lane = threadIdx.x & 31, who = threadIdx.x - 64;
    RingAt<C::kK> rk;
    RingAt<C::kV> rv;
    RingAt<FP8 ? C::kR : 1> rr;
    uint32_t block0 = 0, segment = 0;   // segments: those with blocks
    const Segment& g = at.g;
    const Walk& w = at.w;
    while (advance(a, at)) {
        const bool ok = w.tiles([&](int b, bool is_v) {
            const int ng = w.groups(b);
            if (!is_v) {
                if constexpr (FP8) {
                    if (!__all_sync(0xffffffffu, mbar_wait<true>(&bars[C::kKFull + rk.st], rk.ph, ab, 76))) return false;
                    for (int i = who; i < 128; i += 32 * C::kWorkers)
                        reinterpret_cast<float*>(smem + C::kOffScale)[((block0 + b) & 7) * 128 + i] = cache_scale(smem[C::kOffKScale + rk.st * 128 + i]);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[C::kKReady + rk.st]);
                    rk.next();
                }
                return true;
            }
            if (!__all_sync(0xffffffffu, mbar_wait<true>(&bars[C::kVEmpty + rv.st], rv.ph ^ 1, ab, 67))) return false;
            uint8_t* dst = smem + C::kOffV + rv.st * C::kTile;
            const bool clean = w.masked(b);
            if constexpr (FP8) {
                if (!__all_sync(0xffffffffu, mbar_wait<true>(&bars[C::kRFull + rr.st], rr.ph, ab, 69))) return false;
                const uint8_t* src = smem + C::kOffR + rr.st * C::kCodes;
                const uint8_t* sc = smem + C::kOffVScale + rr.st * 128;
                // a thread takes the same piece of every kRows-th row, where the
                // swizzle is the same: one address that moves.  (Unrolled twice: 8 x
                // 512 rows on 16384 events 373 us, not 331; four times 471: the roles'
                // loops together are more than the instruction cache holds.)
                constexpr int kChunks = D / 16, kRows = 32 * C::kWorkers / kChunks;
                static_assert(kRows % 8 == 0, "rows of the same swizzle");
                const int ch = who % kChunks, e1 = 16 * ng;
                if (clean) {
                    expand_masked<D, 32 * C::kWorkers>(g, 8 * b, src, sc, dst, who, e1, misc.odd, segment);
                } else {
                    int e = who / kChunks;
                    src += cache_chunk(D, 7, e, ch);
                    uint8_t* lo = dst + (ch >> 2) * kHalfBytes + e * 128 + (((2 * ch) & 7) ^ (e & 7)) * 16;
                    uint8_t* hi = dst + (ch >> 2) * kHalfBytes + e * 128 + (((2 * ch + 1) & 7) ^ (e & 7)) * 16;
#pragma unroll 1
                    for (; e < e1; e += kRows, src += kRows * D, lo += kRows * 128, hi += kRows * 128) {
                        const uint4 q = *reinterpret_cast<const uint4*>(src);
                        const uint32_t s = sc[e];
                        uint32_t m, m2;
                        value_factors(s, m, m2);
                        if (s == 255u) {     // a row of NaNs
                            m = 0x7fc0u;
                            m2 = 0;
                        }
                        m |= m << 16;
                        expand16(q, m, m2, *reinterpret_cast<uint4*>(lo), *reinterpret_cast<uint4*>(hi));
                    }
                }
                fence_proxy_async_smem();
            } else if (clean) {
                if (!__all_sync(0xffffffffu, mbar_wait<true>(&bars[C::kVFull + rv.st], rv.ph, ab, 69))) return false;
                bool odd = false;
                for (int x = who; x < 16 * ng * (D / 8); x += 32 * C::kWorkers) {
                    uint4* piece = reinterpret_cast<uint4*>(dst + (x & 7) * 16 + ((x >> 3) % (16 * ng)) * 128 + ((x >> 3) / (16 * ng)) * kHalfBytes);
                    uint4 v = *piece;
                    if (clear_odd(v)) {   // (what lies behind the last event is nobody's)
                        const int e = (x >> 3) % (16 * ng);
                        *piece = v;
                        odd |= segment_group(g, 8 * b + (e >> 4)) * kCacheGroup + (e & 15) < g.s.end;
                    }
                }
                if (odd) misc.odd[segment & 7] = odd_tag(segment);
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bars[C::kVReady + rv.st]);
                if constexpr (FP8) mbar_arrive(&bars[C::kREmpty + rr.st]);
            }
            rv.next();
            rr.next();
            return true;
        });
        block0 += (uint32_t)w.nb;
        if (!ok) return;
        segment += w.nb > 0;
    }
}

__device__ __forceinline__ void one_mma_ss_8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// K-major tiles of 8-bit rows: D bytes a row (128: 128-byte swizzle, 64: 64-byte).
template <int D>
__device__ __forceinline__ uint64_t codes_desc(uint32_t saddr) {
    uint64_t d = smem_desc_sw128(saddr, 16, 8 * D);
    if constexpr (D == 64) d ^= (uint64_t)(2 ^ 4) << 61;   // swizzle mode 4
    return d;
}
// Instruction descriptor of kind::f8f6f4 with A of E4M3 (format 0) or E5M2 (1), B
// of E4M3, fp32 D; the rest as idesc_bf16.
constexpr uint32_t kRestE5m2 = 1u << 7;
__host__ __device__ constexpr uint32_t idesc_e4m3(uint32_t M, uint32_t N) {
    return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// The issuer (one lane).  State that goes on between segments.
template <int D, bool FP8>
struct Issuer {
    RingAt<Cfg<D, FP8>::kK> rk;
    RingAt<Cfg<D, FP8>::kV> rv;
    uint32_t p_ph[2] = {0, 0}, o_ph[2] = {1, 1}, q_ph = 0;
};

template <int D, bool FP8>
__device__ __forceinline__ bool issue_segment(Issuer<D, FP8>& z, const Walk& w, uint8_t* smem, uint64_t* bars,
                                              uint32_t tmem, const Abort& ab) {
    using C = Cfg<D, FP8>;
    constexpr uint32_t idesc_pv = idesc_bf16(128, D, false, true);
    constexpr uint64_t kKDesc = C::kKTile >> 4, kVDesc = C::kTile >> 4;
    const uint64_t q_desc = FP8 ? codes_desc<D>(smem_u32(smem)) : smem_desc_sw128(smem_u32(smem), 16, 1024);
    const uint64_t k_desc = FP8 ? codes_desc<D>(smem_u32(smem + C::kOffK)) : smem_desc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
    const uint64_t v_desc = smem_desc_sw128(smem_u32(smem + C::kOffV), kHalfBytes, 1024);
    const int nb = w.nb;
    const uint32_t last_keys = (uint32_t)(16 * w.groups(nb - 1));
    const uint32_t idesc_full = FP8 ? idesc_e4m3(128, 128) : idesc_bf16(128, 128, false, false);
    const uint32_t idesc_last = FP8 ? idesc_e4m3(128, last_keys) : idesc_bf16(128, last_keys, false, false);
    const uint64_t q2 = q_desc + (w.dual ? 0 : (uint64_t)(C::kTile >> 4));
    auto keys = [&]() -> bool {
        if (!mbar_wait<true>(&bars[C::kKFull + z.rk.st], z.rk.ph, ab, 64)) return false;
        if (FP8 && !mbar_wait<true>(&bars[C::kKReady + z.rk.st], z.rk.ph, ab, 70)) return false;
        tc_fence_after();
        return true;
    };
    auto values = [&]() -> bool {
        if (!FP8 && !mbar_wait<true>(&bars[C::kVFull + z.rv.st], z.rv.ph, ab, 64)) return false;
        if (!mbar_wait<true>(&bars[C::kVReady + z.rv.st], z.rv.ph, ab, 70)) return false;
        tc_fence_after();
        return true;
    };
    auto scores = [&](int s, int b) {
        const uint64_t q = s ? q2 : q_desc, k = k_desc + z.rk.st * kKDesc;
        const uint32_t id = b == nb - 1 ? idesc_last : idesc_full;
        if constexpr (FP8) {   // both parts of the queries, 32 columns a step
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
                    one_mma_ss_8(tmem + s * 128, q + part * (C::kCodes >> 4) + 2 * i, k + 2 * i,
                                 id | (part ? kRestE5m2 : 0), part + i > 0);
        } else {
            one_scores<D>(tmem + s * 128, q, k, id);
        }
        one_commit(&bars[C::kSFull + s]);
    };
    auto sums = [&](int s, int b, bool first) -> bool {
        const uint32_t sc = tmem + s * 128, oc = tmem + 256 + s * 128;
        const uint64_t vd = v_desc + z.rv.st * kVDesc;
        if (first) {   // the slot's sums of its last segment have been read
            if (!mbar_wait<true>(&bars[C::kOFree + s], z.o_ph[s], ab, 65)) return false;
            z.o_ph[s] ^= 1;
        }
        if (!mbar_wait<true>(&bars[C::kPFull + s], z.p_ph[s], ab, 66)) return false;
        z.p_ph[s] ^= 1;
        tc_fence_after();
        const uint32_t keys = b == nb - 1 ? last_keys : 128u;
        one_sums(oc, sc, sc + 16, vd, idesc_pv, keys >> 4, first ? 0 : 1);
        if (keys > 64) one_sums(oc, sc + 32, sc + 48, vd + mnmajor_step(4), idesc_pv, (keys - 64) >> 4, 1);
        return true;
    };
    if (!mbar_wait<true>(&bars[C::kQFull], z.q_ph, ab, 63)) return false;
    tc_fence_after();
    z.q_ph ^= 1;
    if (!w.dual) {
        // both slots: S(b + 1) follows each slot's P V(b)
        for (int b = -1; b < nb; ++b) {
            if (b >= 0 && (!values() || !sums(0, b, b == 0))) return false;
            if (b + 1 < nb) {
                if (!keys()) return false;
                scores(0, b + 1);
            } else {
                one_commit(&bars[C::kOFull]);
            }
            if (b >= 0) {
                if (!sums(1, b, b == 0)) return false;
                one_commit(&bars[C::kVEmpty + z.rv.st]);
                z.rv.next();
            }
            if (b + 1 < nb) {
                scores(1, b + 1);
                one_commit(&bars[C::kKEmpty + z.rk.st]);
                z.rk.next();
                if (b + 2 == nb) one_commit(&bars[C::kQEmpty]);   // the queries may be replaced
            } else {
                one_commit(&bars[C::kOFull + 1]);
            }
        }
    } else {
        for (int b = -2; b < nb; ++b) {
            const int s = b & 1;
            if (b >= 0) {
                if (!values() || !sums(s, b, b < 2)) return false;
                one_commit(&bars[C::kVEmpty + z.rv.st]);
                z.rv.next();
                if (b + 2 >= nb) one_commit(&bars[C::kOFull + s]);
            }
            if (b + 2 < nb) {
                if (!keys()) return false;
                scores(s, b + 2);
                one_commit(&bars[C::kKEmpty + z.rk.st]);
                z.rk.next();
                if (b + 3 == nb) one_commit(&bars[C::kQEmpty]);
            }
        }
    }
    return true;
}

// Infinities and NaNs of the masked blocks' values (left out of the products)
// added to columns c0 .. c0 + 31 of a row that sees their events; element-wise
// activations give NaN there.
template <int D, bool FP8, bool SM>
__device__ __noinline__ void add_odd(const AttnArgs& a, const Segment& g, const Walk& w, int row, int c0, float* o) {
    const RowView rv = row_view(a, g, row);
    for (int b = 0; b < w.nb; ++b) {
        if (!w.masked(b)) continue;
        for (int i = 8 * b; i < 8 * b + w.groups(b); ++i) {
            const int e0 = segment_group(g, i) * kCacheGroup;
            const uint32_t bits = row_bits(a, g, rv, e0);
            const int64_t blk = bits ? cache_block(a.c, a.w, g.b, e0, g.h) : -1;
            if (blk < 0) continue;
            for (int j = 0; j < 16; ++j) {
                if (!(bits >> j & 1u)) continue;
                const int e = (e0 + j) & ((1 << a.c.page_log) - 1);
                const uint8_t* v = a.c.v + blk * a.c.block;
                const uint32_t scale = FP8 ? a.c.vs[(blk << a.c.page_log) + e] : 0u;
                if (FP8 && scale < kOddScale) continue;
                const auto add = [&](int c, float y) {
                    if (!isfinite(y)) o[c] += SM ? y : y - y;
                };
                if constexpr (FP8) {
                    for (int c = 0; c < 32; ++c) {
                        uint32_t h;
                        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)v[cache_chunk(D, a.c.page_log, e, (c0 + c) >> 4) + (c & 15)]));
                        add(c, scale == 255u ? __uint_as_float(0x7fc00000u) : __half22float2(*reinterpret_cast<__half2*>(&h)).x * cache_scale(scale));
                    }
                } else {
                    uint4 q[4], z;   // (whole pieces, few of which hold any)
#pragma unroll
                    for (int k = 0; k < 4; ++k) q[k] = *reinterpret_cast<const uint4*>(v + cache_chunk(2 * D, a.c.page_log, e, (c0 >> 3) + k));
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (!clear_odd(z = q[k])) continue;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            add(8 * k + 2 * c, bf16_lo((&q[k].x)[c]));
                            add(8 * k + 2 * c + 1, bf16_hi((&q[k].x)[c]));
                        }
                    }
                }
            }
        }
    }
}

// row_bits of the 8 groups of a block.  (Out of line: the instruction cache holds
// little more than the loop that is to go on.)
static __device__ __noinline__ uint4 block_bits(const AttnArgs& a, const Segment& g, int row, int i) {
    const RowView v = row_view(a, g, row);
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
    for (int h = 0; h < 8; ++h) {
        if (i + h >= g.n) break;
        const uint32_t bits = row_bits(a, g, v, segment_group(g, i + h) * kCacheGroup) << (16 * (h & 1));
        if (h < 2) r.x |= bits;
        else if (h < 4) r.y |= bits;
        else if (h < 6) r.z |= bits;
        else r.w |= bits;
    }
    return r;
}

// A row's sums times f, where they lie.
template <int D>
__device__ __forceinline__ void scale_sums(uint32_t oc, float f) {
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

// A warp's 32 rows of queries, from row r0 of the tile, to shared memory: whole
// rows in neighbouring lanes, as operands (flip: the sign bits, for a negative
// scale of the scores).  8-bit: in units that make a row's
// largest value lie in [128, 256), and what undoes that.
template <int D, bool FP8>
__device__ __forceinline__ void put_queries(const AttnArgs& a, const Segment& g, int r0, int row0, uint32_t flip, uint8_t* dst, float* unit) {
    constexpr int kLanes = D / 8, kEach = 32 / kLanes;   // lanes a row, rows at a time
    // several loads on their way at once; more would cost more in fetching the
    // instructions of a loop that is run a few times a segment
    constexpr int kAhead = FP8 ? 4 : 8;
    const int lane = threadIdx.x & 31, c = lane % kLanes;
    int64_t at = 0;   // of row r0 + lane
    if (r0 + lane < g.rows) {
        const int rho = g.rho0 + r0 + lane, tok = rho / a.G;
        at = (g.s.t0 + tok) * a.qt + (g.h * a.G + rho - tok * a.G) * a.qh;
    }
#pragma unroll 1
    for (int i0 = lane / kLanes; i0 < 32; i0 += kAhead * kEach) {
        uint4 q[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t from = __shfl_sync(0xffffffffu, at, i0 + k * kEach);
            q[k] = make_uint4(0, 0, 0, 0);
            if (r0 + i0 + k * kEach < g.rows) {
                const __nv_bfloat16* src = (const __nv_bfloat16*)a.q + from + 8 * c;
                if (a.q_wide) {
                    q[k] = __ldg(reinterpret_cast<const uint4*>(src));
                } else {
                    const uint16_t* h = reinterpret_cast<const uint16_t*>(src);
                    uint32_t* p = &q[k].x;
#pragma unroll
                    for (int i = 0; i < 4; ++i) p[i] = h[2 * i] | (uint32_t)h[2 * i + 1] << 16;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const uint4 v = make_uint4(q[k].x ^ flip, q[k].y ^ flip, q[k].z ^ flip, q[k].w ^ flip);
            const int i = i0 + k * kEach, row = row0 + i;
            if constexpr (FP8) {
                const uint32_t p[4] = {v.x, v.y, v.z, v.w};
                float top = 0.0f;
#pragma unroll
                for (int x = 0; x < 4; ++x) top = fmaxf(top, fmaxf(fabsf(bf16_lo(p[x])), fabsf(bf16_hi(p[x]))));
#pragma unroll
                for (int m = 1; m < kLanes; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
                // (codes hold no infinities: such a row's scores are NaN, as its softmax is)
                const float f = top < INFINITY ? inverse_power(top) : __uint_as_float(0x7fc00000u);
                uint32_t h[4], l[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) split_q(bf16_lo(p[x]) * f * 128.0f, bf16_hi(p[x]) * f * 128.0f, h[x], l[x]);
                const int to = cache_chunk(D, 7, row, c >> 1) + 8 * (c & 1);
                *reinterpret_cast<uint2*>(dst + to) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
                *reinterpret_cast<uint2*>(dst + 128 * D + to) = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
                if (c == 0) unit[i] = 0x1p-7f / f;
            } else {
                *reinterpret_cast<uint4*>(dst + row * 128 + (c >> 3) * kHalfBytes + (((c & 7) ^ (row & 7)) << 4)) = v;
            }
        }
    }
}

template <int D, bool FP8, int ACT>
__device__ __forceinline__ void tile_rows(const AttnArgs& a, uint8_t* smem, uint64_t* bars, Misc& misc, uint32_t tmem,
                                          Place& at, const Abort& ab) {
    using C = Cfg<D, FP8>;
    constexpr bool kSm = ACT == kSoftmax;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = (warp - C::kRows0) >> 2;
    const int quarter = warp & 3;
    static_assert(C::kRows0 % 4 == 0, "whole warpgroups");
    const int row = quarter * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t sc = trow + s * 128, oc = trow + 256 + s * 128;
    float2* const fin = reinterpret_cast<float2*>(smem + C::kOffFin) + row;
    // for outputs on their way: the place of the warp's own queries, which no other
    // warp writes to (8-bit rows of 64 are too short: a place apart)
    uint8_t* const stage = smem + (C::kStageApart ? C::kOffStage + (s * 4 + quarter) * 4096 : s * C::kTile + quarter * 4096);
    const auto scale_of = [&](float alpha) {
        ActScale k = act_scale<ACT>(alpha);
        // (a zero scale would make NaN of masked scores; the least normal number is none to any that are not)
        if (kSm) k.c0 = fmaxf(fabsf(k.c0), 0x1p-126f);
        return k;
    };
    ActScale ks = scale_of(a.alpha);
    const Segment& g = at.g;
    const Walk& w = at.w;
    uint32_t items = 0, used[2] = {0, 0}, fins = 0, q_ph = 1, block0 = 0;
    while (advance(a, at)) {
        const int n = w.blocks(s), n1 = w.n1, nb = w.nb, open0 = w.open0, open1 = w.open1;
        const bool dual = w.dual;
        const int tile0 = dual ? 0 : 128 * s;            // first row of the slot
        const int r = tile0 + row;                       // of the tile
        const bool real = r < g.rows;
        if (nb > 0) {
            if (!wg_wait<true>(&bars[C::kQEmpty], q_ph, ab, 61)) return;
            q_ph ^= 1;
            if (!(dual && s)) {
                put_queries<D, FP8>(a, g, tile0 + quarter * 32, quarter * 32, kSm && a.alpha < 0.0f ? 0x80008000u : 0u, smem + (dual ? 0 : s) * C::kTile,
                                    reinterpret_cast<float*>(smem + C::kOffUnit) + tile0 + quarter * 32);
                fence_proxy_async_smem();
            }
            mbar_arrive(&bars[C::kQFull]);
        }
        float ref = -INFINITY, sum = 0.0f;   // reference and sum of the weights
        for (int j = 0; j < n; ++j) {
            const int b = dual ? 2 * j + s : j;
            // what the row sees of the block, made while its scores are
            const bool masked = b < open0 || b >= open1;
            uint4 vis = make_uint4(~0u, ~0u, ~0u, ~0u);
            if (masked) vis = block_bits(a, g, r, 8 * b);
            if (!wg_wait<true>(&bars[C::kSFull + s], (items + j) & 1, ab, 71)) return;
            tc_fence_after();
            if (FP8 && j == 0) ks = scale_of(a.alpha * reinterpret_cast<const float*>(smem + C::kOffUnit)[r]);
            const uint32_t gone = *reinterpret_cast<volatile uint8_t*>(&misc.gone[(block0 + b) & 15]);
            const bool cut = masked || gone;
            if (gone) {
                const auto lost = [&](int i) { return (gone >> i & 1u ? 0xffffu : 0u) | (gone >> i & 2u ? 0xffff0000u : 0u); };
                vis.x &= ~lost(0);
                vis.y &= ~lost(2);
                vis.z &= ~lost(4);
                vis.w &= ~lost(6);
            }
            uint32_t x[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(sc + c * 32, *reinterpret_cast<uint32_t(*)[32]>(x + c * 32));
            tmem_ld_wait();
            if constexpr (FP8) {   // the keys' powers of two
                const float4* p = reinterpret_cast<const float4*>(smem + C::kOffScale) + ((block0 + b) & 7) * 32;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float4 y = p[e];
                    const float2 u = f2_split(f2_mul(f2_make(__uint_as_float(x[4 * e]), __uint_as_float(x[4 * e + 1])), f2_make(y.x, y.y)));
                    const float2 v = f2_split(f2_mul(f2_make(__uint_as_float(x[4 * e + 2]), __uint_as_float(x[4 * e + 3])), f2_make(y.z, y.w)));
                    x[4 * e] = __float_as_uint(u.x);
                    x[4 * e + 1] = __float_as_uint(u.y);
                    x[4 * e + 2] = __float_as_uint(v.x);
                    x[4 * e + 3] = __float_as_uint(v.y);
                }
            }
            if (cut) {
                const uint32_t see[4] = {vis.x, vis.y, vis.z, vis.w};
#pragma unroll
                for (int e = 0; e < 128; ++e)
                    if (!(see[e >> 5] >> (e & 31) & 1u)) x[e] = 0xff800000u;   // -inf
            }
            if constexpr (kSm) {
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 128; e += 8)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        m4[u] = max3_nan(m4[u], __uint_as_float(x[e + u]), __uint_as_float(x[e + 4 + u]));
                const float top = max3_nan(max3_nan(m4[0], m4[1], m4[2]), m4[3], m4[3]) * ks.c0;
                if (top != top) {
                    sum = top;
                    if (ref == -INFINITY) ref = 0.0f;   // the part counts
                }
                // the reference moves when it would be passed by more than 2^8 (that
                // the scores are complete says that the sums before them are)
                const bool up = real && top > ref + kRise;   // also from -inf
                if (__any_sync(0xffffffffu, up)) {
                    const float nref = up ? top : ref;
                    const float f = up ? ex2_approx(ref - nref) : 1.0f;   // 0 from -inf
                    ref = nref;
                    sum *= f;
                    if (j > 0) scale_sums<D>(oc, f);
                }
            }
            const float nref = kSm ? (ref == -INFINITY ? 0.0f : -ref) : 0.0f;
            uint64_t sum2 = f2_make(0.0f, 0.0f);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    float p0, p1;
                    const float s0 = __uint_as_float(x[c * 32 + e]), s1 = __uint_as_float(x[c * 32 + e + 1]);
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
                tmem_st16(sc + c * 16, pk);
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&bars[C::kPFull + s]);
            if constexpr (kSm) {
                const float2 y = f2_split(sum2);
                sum += y.x + y.y;
            }
        }
        items += n;
        block0 += (uint32_t)nb;
        const bool both = dual && n1 > 0;   // slot 0's threads join slot 1's sums to their own
        if (n > 0 && !wg_wait<true>(&bars[C::kOFull + s], used[s] & 1, ab, 73)) return;
        tc_fence_after();
        float f0 = 1.0f, f1 = 0.0f;
        if (both && s) {
            *fin = make_float2(ref, sum);
            tc_fence_before();
            mbar_arrive(&bars[C::kFin]);
        }
        if (both && !s) {
            if (!wg_wait<true>(&bars[C::kOFull + 1], used[1] & 1, ab, 74) || !wg_wait<true>(&bars[C::kFin], fins & 1, ab, 75)) return;
            tc_fence_after();
            f1 = 1.0f;
            if constexpr (kSm) {
                const float2 y = *fin;
                const float m = fmaxf(ref, y.x), m0 = m == -INFINITY ? 0.0f : m;
                f0 = ex2_approx(ref - m0);
                f1 = ex2_approx(y.x - m0);
                sum = sum * f0 + y.y * f1;
                ref = m;
            }
        }
        fins += both;
        if (!(dual && s)) {
            const bool dirty = *reinterpret_cast<volatile uint8_t*>(&misc.odd[used[0] & 7]) == odd_tag(used[0]);
            float* slot = nullptr;
            if (!g.whole) slot = a.part + (int64_t)(2 * blockIdx.x + (g.head ? 1 : 0)) * cache_slot(a.TM, D);
            const float inv = kSm ? (sum == 0.0f ? 0.0f : 1.0f / sum) : 1.0f;
            // outputs, 32 columns at a time, through shared memory, so that a row's
            // lie in neighbouring lanes (the queries' products are over)
            const int warp_rows = min(32, g.rows - tile0 - quarter * 32);
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                float y[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) y[e] = 0.0f;
                if (n > 0) {
                    tmem_ld32(oc + c, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(o[e]) * f0;
                }
                if (both) {
                    tmem_ld32(oc + 128 + c, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e) y[e] = fmaf(__uint_as_float(o[e]), f1, y[e]);
                }
                if (dirty && real) {
                    float z[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) z[e] = y[e];
                    add_odd<D, FP8, kSm>(a, g, w, r, c, z);
#pragma unroll
                    for (int e = 0; e < 32; ++e) y[e] = z[e];
                }
                if (slot) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<float4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                    __syncwarp();
                    float* to = slot + (tile0 + quarter * 32) * D + c;
                    for (int i = lane >> 3; i < warp_rows; i += 4)
                        reinterpret_cast<float4*>(to + i * D)[lane & 7] = *reinterpret_cast<const float4*>(stage + i * 128 + (((lane & 7) ^ (i & 7)) << 4));
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        *reinterpret_cast<uint4*>(stage + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4)) =
                            make_uint4(pack_bf16x2(y[8 * e] * inv, y[8 * e + 1] * inv), pack_bf16x2(y[8 * e + 2] * inv, y[8 * e + 3] * inv),
                                       pack_bf16x2(y[8 * e + 4] * inv, y[8 * e + 5] * inv), pack_bf16x2(y[8 * e + 6] * inv, y[8 * e + 7] * inv));
                    __syncwarp();
                    for (int i = lane >> 2; i < warp_rows; i += 8) {
                        const int rho = g.rho0 + tile0 + quarter * 32 + i, tok = rho / a.G;
                        const int64_t out = (int64_t)(g.s.t0 + tok) * a.H + g.h * a.G + (rho - tok * a.G);
                        reinterpret_cast<uint4*>((__nv_bfloat16*)a.o + out * D + c)[lane & 3] =
                            *reinterpret_cast<const uint4*>(stage + i * 64 + (((lane & 3) ^ ((i >> 1) & 3)) << 4));
                    }
                }
                __syncwarp();
            }
            if (kSm && real) {
                if (slot) {
                    slot[a.TM * D + r] = ref;
                    slot[a.TM * (D + 1) + r] = sum;
                } else if (a.lse) {
                    const int rho = g.rho0 + r, tok = rho / a.G;
                    a.lse[(int64_t)(g.s.t0 + tok) * a.H + g.h * a.G + (rho - tok * a.G)] =
                        sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * 0.693147180559945309f;
                }
            }
            if (slot && g.head && threadIdx.x == 32 * C::kRows0) {
                CacheDesc& t = a.desc[blockIdx.x];
                t.rows = g.rows;
                t.t0 = g.s.t0;
                t.h = g.h;
                t.rho0 = g.rho0;
                t.parts = g.parts;
            }
            tc_fence_before();
            if (n > 0) mbar_arrive(&bars[C::kOFree + s]);
            if (both) mbar_arrive(&bars[C::kOFree + 1]);
        }
        used[0] += nb > 0;
        used[1] += n1 > 0;
    }
}

template <int D, bool FP8, int ACT>
__global__ void __launch_bounds__(Cfg<D, FP8>::kThreads, 1)
cache_tc_kernel(const __grid_constant__ AttnArgs a) {
    using C = Cfg<D, FP8>;
    extern __shared__ __align__(1024) uint8_t smem[];   // (the operands' swizzle starts at 1024 bytes)
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    Misc& misc = *reinterpret_cast<Misc*>(smem + C::kOffMisc);
    const int warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.launch_dependents;");
    if (threadIdx.x == 32 * C::kRows0) a.desc[blockIdx.x].parts = 0;   // (the thread that may set it)
    if (threadIdx.x == 0) {
        for (int b = 0; b < C::kNumBars; ++b) {
            uint32_t n = 1;
            if (b == C::kQFull) n = 256;
            if (b == C::kKFull && a.stall) n = 2;   // (an arrival that never comes)
            if (b == C::kFin || (b >= C::kPFull && b < C::kPFull + 2) || (b >= C::kOFree && b < C::kOFree + 2)) n = 128;
            if ((b >= C::kKReady && b < C::kKEmpty) || (b >= C::kVReady && b < C::kVEmpty) || b >= C::kREmpty) n = C::kWorkers;
            mbar_init(&bars[b], n);
        }
        misc.abort_flag = 0;
        for (int i = 0; i < 8; ++i) misc.odd[i] = 0;
        fence_mbar_init();
    }
    const Share sh = find_share<C::kThreads>(a, reinterpret_cast<int64_t*>(smem + C::kOffScan));
    if (sh.u >= sh.u_end) return;   // the whole CTA
    if (warp == 1) tmem_alloc(&misc.tmem, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc.tmem;
    const Abort ab{&misc.abort_flag, a.c.err, a.wait_ns};
    Place& at = reinterpret_cast<Place*>(smem + C::kOffPlace)[warp];
    if ((threadIdx.x & 31) == 0) at.sh = sh;
    __syncwarp();
    if (warp < C::kRows0) {
        // 384 threads start with 168 registers: 88 + 2 * 208; 512 with 128: 2 * 64 + 2 * 192
        if constexpr (FP8) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 0) {
            load_tiles<D, FP8>(a, smem, bars, misc, at, ab);
        } else if (warp == 1) {
            Issuer<D, FP8> z;
            bool ok = true;
            while (ok && advance(a, at)) {
                if (at.w.nb == 0) continue;
                if (elect_one()) ok = issue_segment<D, FP8>(z, at.w, smem, bars, tmem, ab);
                // the elected lane keeps the state; all agree on whether to go on
                ok = __all_sync(0xffffffffu, ok);
            }
            if (elect_one()) {
                // all of its products complete before TMEM is released
                one_commit(&bars[C::kMmaDone]);
                mbar_wait_teardown(&bars[C::kMmaDone], 0);
            }
            __syncwarp();
        } else {
            work_tiles<D, FP8>(a, smem, bars, misc, at, ab);
        }
    } else {
        if constexpr (FP8) asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        tile_rows<D, FP8, ACT>(a, smem, bars, misc, tmem, at, ab);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D, bool FP8, int ACT>
gdpa_status launch(const AttnArgs& a, int grid, cudaStream_t st) {
    using C = Cfg<D, FP8>;
    static std::atomic<uint64_t> done{0};
    if (!cache_smem((const void*)cache_tc_kernel<D, FP8, ACT>, C::kSmem, done)) return GDPA_ERR_CUDA;
    cache_tc_kernel<D, FP8, ACT><<<grid, C::kThreads, C::kSmem, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? GDPA_OK : GDPA_ERR_CUDA;
}

template <bool FP8>
gdpa_status launch_any(const AttnArgs& a, int grid, cudaStream_t st) {
    gdpa_status s = GDPA_OK;
    if (a.c.d == 128) {
        if (a.act == kSoftmax) return launch<128, FP8, kSoftmax>(a, grid, st);
        GDPA_DISPATCH_ACT(a.act, A, s = launch<128, FP8, A>(a, grid, st))
    } else {
        if (a.act == kSoftmax) return launch<64, FP8, kSoftmax>(a, grid, st);
        GDPA_DISPATCH_ACT(a.act, A, s = launch<64, FP8, A>(a, grid, st))
    }
    return s;
}

}  // namespace cache_tc
}  // namespace gdpa
