// Shared-prefix attention backward on the tensor cores (bf16 rows, d = 64 or
// 128), as two kernels that each keep their result in TMEM until it is done:
//
//   dK, dV (prefix_dkv_kernel): a unit is a 128-key block of one key head
//     against every packed query row that sees it.  Scores are formed
//     transposed, S^T = K Q^T and dP^T = V dO^T, so that the weights leave the
//     warps as the TMEM operand of the next products, dV += P^T dO and dK +=
//     dS^T Q: nothing is staged in shared memory or transposed, and the keys'
//     gradients, summed over all rows and heads, are rounded once.
//   dQ (prefix_dq_kernel): a run is a row tile against a piece's key blocks,
//     S = Q K^T, dP = dO V^T, dQ += dS K; the parts are joined by the merge.
//
// Forming the scores twice (7 products a tile instead of 5) is what it costs
// to have no float32 dQ in memory: adding each tile's 64 KB to it atomically
// would move more bytes through L2 than all operands, in an order that
// changes the sums from run to run.  Results here are the same bits every time.
//
// dK and dV walk items of 64 query rows through two slots of TMEM columns
// [S^T | dP^T], a warpgroup each, thread = key: while one slot's weights are
// computed the tensor core runs the other slot's products, then item e's sums
// and the scores of item e + 2 into the same columns.  The sums leave through
// a warpgroup of their own, and the next unit's keys load into whichever of
// three pairs of buffers is free, so that short units follow one another
// without a gap (32 ragged users of 64 .. 2048 keys: 41 us; with the keys in
// one place and the two slots' warpgroups storing the sums 65 us, with stores
// of half sectors 46).
// dQ walks blocks of 128 keys: S and dP go into registers at once and the next
// block's scores into the freed columns, dS into one of two places of its own
// (99 us against 108 in the form above, 1024 rows x 8192 keys x 16 heads).
//
// What bounds them, on those 1024 rows x 8192 keys x 16 heads with GELU: dK
// and dV 128 us, the tensor pipe busy 46% of them: products 128 x 64 x 16 whose
// operands take 120 of the 128 bytes shared memory gives a cycle, and a slot's
// chain of scores, weights and sums; 128-row items would read less, but TMEM
// has no room for them beside 256 columns of sums.  dQ 99 us, tensor pipe 49%:
// 64 KB of K and V a block, 5.4 TB/s in all, arrive late for the issuer.
// Softmax batches of ragged users are bound by the few row tiles a unit has.
//
// Rows behind the last one of an item share its 16-row step: their weights are
// zero by selection, and the rows themselves are cleared in shared memory so
// that what lies there does not enter as 0 * inf.
//
// Every wait is bounded (csrc/tc_common.cuh).
#include <cuda_bf16.h>

#include "act.cuh"
#include "prefix_tc.cuh"

namespace gdpa {
namespace {

using namespace tc;

constexpr int kThreads = 384;   // producer and issuer (and two idle warps), a warpgroup per slot
constexpr int kKvThreads = 512; // and one that drains dK and dV
constexpr int kHalfBytes = 128 * 128;
constexpr uint32_t kTmemCols = 512;
constexpr int kItem = 64;   // columns of an item
// Items of every tile but a unit's last: tiles of 128 / r whole tokens of r rows
// have more rows than one.
constexpr int kTileItems = 2;
constexpr int fewest_tile_rows() {
    int n = kBM;
    for (int r = 1; r <= kBM; ++r) n = kBM / r * r < n ? kBM / r * r : n;
    return n;
}
static_assert(fewest_tile_rows() > kItem && kBM <= kTileItems * kItem, "items of a tile");

struct BwArgs {
    const PrefixUnit* units;
    const PrefixPiece* pieces;
    const int32_t* seg;
    const float* lse;
    const float* delta;
    float* parts;
    float* unit_parts;
    __nv_bfloat16 *dkp, *dvp, *dk, *dv;
    int H, Hkv, r, tpt, windowed, window;
    int q_bytes;
    float alpha;
    int32_t* err;
    uint64_t wait_ns;
    int stall;   // test hook: CTA 0 never loads its first query tile
};

// weights and score gradients of two pairs
template <int ACT>
__device__ __forceinline__ void weights2(float s0, float s1, float dp0, float dp1, const ActScale& k,
                                         float l0, float l1, float d0, float d1, float& p0, float& p1,
                                         float& ds0, float& ds1) {
    if constexpr (ACT == kSoftmax) {
        const float2 t = f2_split(f2_fma(f2_make(s0, s1), f2_make(k.c0, k.c0), f2_make(-l0, -l1)));
        p0 = ex2_approx(t.x);
        p1 = ex2_approx(t.y);
        ds0 = p0 * (dp0 - d0);
        ds1 = p1 * (dp1 - d1);
    } else {
        float a0, a1;
        act_dact_s2<ACT>(s0, s1, k, p0, p1, a0, a1);
        const float2 d = f2_split(f2_mul(f2_make(dp0, dp1), f2_make(a0, a1)));
        ds0 = d.x;
        ds1 = d.y;
    }
}

// clear rows [r0, r1) of a [128][D] tile in shared memory (128 threads)
template <int D>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int r0, int r1, int tid) {
    for (int i = tid; i < (r1 - r0) * (D / 8); i += 128) {
        const int row = r0 + i / (D / 8), ch = i % (D / 8);
        *reinterpret_cast<uint4*>(tile + (ch >> 3) * kHalfBytes + row * 128 + ((ch & 7) << 4)) =
            make_uint4(0u, 0u, 0u, 0u);
    }
}

// ----------------------------------------------------------------- dK and dV

template <int D>
struct KvCfg {
    static constexpr int kHalves = D / 64;
    static constexpr int kTile = 128 * D * 2;
    static constexpr int kPair = 2 * kTile;      // K and V of a unit, or Q and dO of a tile; 3 of them
    static constexpr int kOffStat = 3 * kPair;   // [8 warps][2][64] (lse, delta) pairs
    static constexpr int kOffBar = kOffStat + 8 * 2 * 64 * 8;
    enum { kFull = 0, kEmpty = kFull + 3, kSDFull = kEmpty + 3, kPFull = kSDFull + 2,
           kAccFull = kPFull + 2, kAccFree, kMmaDone, kNumBars };
    static constexpr int kSmem = kOffBar + kNumBars * 8 + 16 + 1024;
};

// rows of tile m of a unit, and its 64-row items
__device__ __forceinline__ int tile_rows(const PrefixUnit& u, const BwArgs& a, int m) {
    return min(a.tpt, u.ntok - m * a.tpt) * a.r;
}

// Items of a unit (0: no row sees its keys).
__device__ __forceinline__ int unit_items(const PrefixUnit& u, const BwArgs& a) {
    const int tiles = (u.ntok + a.tpt - 1) / a.tpt;
    return tiles == 0 ? 0 : (tiles - 1) * kTileItems + (tile_rows(u, a, tiles - 1) + kItem - 1) / kItem;
}

// Which of the three pairs of buffers hold a unit's keys and its tiles (in
// turn).  The next unit's keys go where no recent tile is, so that they load
// while this unit is worked on; its first tile where this unit's keys were.
struct Places {
    uint32_t kv = 0, x = 1, y = 2;
    __device__ __forceinline__ uint32_t tile(int m) const { return m & 1 ? y : x; }
    __device__ __forceinline__ void next(int tiles) {
        const uint32_t last = tiles & 1 ? x : y, other = tiles & 1 ? y : x;
        x = kv;
        kv = other;
        y = last;
    }
};

template <int D>
__device__ __forceinline__ void kv_producer(const CUtensorMap* tmQ, const CUtensorMap* tmDO, const CUtensorMap* tmKp,
                                            const CUtensorMap* tmVp, const CUtensorMap* tmK, const CUtensorMap* tmV,
                                            const BwArgs& a, uint8_t* smem, uint64_t* bars, int seg0, int seg1,
                                            const Abort& ab) {
    using C = KvCfg<D>;
    const uint64_t keep = policy_evict_last(), once = policy_evict_first();
    int32_t armed[3] = {-1, -1, -1};
    uint32_t ph = 7;   // per pair: the parity of "empty" to wait for
    Places at;
    bool stall = a.stall && blockIdx.x == 0;
    // a pair is free: arm it for the next load (of nothing: it stays empty)
    auto take = [&](uint32_t pair, uint32_t bytes) -> bool {
        if (!mbar_wait<true>(&bars[C::kEmpty + pair], (ph >> pair) & 1, ab, 81)) return false;
        ph ^= 1u << pair;
        if (bytes == 0) return true;
        mbar_arrive_expect_tx(&bars[C::kFull + pair], bytes);
        armed[pair] = (int32_t)((ph >> pair) & 1);
        return true;
    };
    for (int t = seg0; t < seg1; ++t) {
        const PrefixUnit u = load_unit(a.units + t);
        const int tiles = (u.ntok + a.tpt - 1) / a.tpt;
        if (tiles == 0) continue;
        const bool own = u.flags & kPieceOwn;
        const CUtensorMap *mk = own ? tmK : tmKp, *mv = own ? tmV : tmVp;
        if (!take(at.kv, 2 * C::kTile)) goto unwind;
#pragma unroll
        for (int hf = 0; hf < C::kHalves; ++hf) {
            uint8_t* dst = smem + at.kv * C::kPair + hf * kHalfBytes;
            tma_load_2d(mk, &bars[C::kFull + at.kv], dst, u.hk * D + hf * 64, u.k0, once);
            tma_load_2d(mv, &bars[C::kFull + at.kv], dst + C::kTile, u.hk * D + hf * 64, u.k0, once);
        }
        for (int m = 0; m < tiles; ++m) {
            const uint32_t pair = at.tile(m);
            if (!take(pair, stall ? 0 : 2 * (uint32_t)a.q_bytes)) goto unwind;
            if (stall) {
                stall = false;
                continue;
            }
#pragma unroll
            for (int hf = 0; hf < C::kHalves; ++hf) {
                uint8_t* dst = smem + pair * C::kPair + hf * kHalfBytes;
                tma_load_3d(tmQ, &bars[C::kFull + pair], dst, hf * 64, u.hk * a.r, u.tok + m * a.tpt, keep);
                tma_load_3d(tmDO, &bars[C::kFull + pair], dst + C::kTile, hf * 64, u.hk * a.r, u.tok + m * a.tpt, keep);
            }
        }
        at.next(tiles);
    }
unwind:
    // never leave the CTA with a TMA write still in flight
    for (int s = 0; s < 3; ++s)
        if (armed[s] >= 0) mbar_wait_teardown(&bars[C::kFull + s], (uint32_t)armed[s]);
}

// A walk over the items of a CTA's units, for the issuer: it runs one for the
// scores and, two items behind, one for the sums, across units.
struct ItemWalk {
    PrefixUnit u;
    Places at;
    int t, tiles, items, x, last_rows;
    __device__ __forceinline__ void load(const BwArgs& a, int seg1) {
        for (; t < seg1; ++t) {   // units without rows have no items
            u = load_unit(a.units + t);
            tiles = (u.ntok + a.tpt - 1) / a.tpt;
            if (tiles > 0) break;
        }
        x = 0;
        if (t < seg1) {
            last_rows = tile_rows(u, a, tiles - 1);
            items = (tiles - 1) * kTileItems + (last_rows + kItem - 1) / kItem;
        }
    }
    __device__ __forceinline__ bool last() const { return x == items - 1; }
    __device__ __forceinline__ void next(const BwArgs& a, int seg1) {
        if (++x < items) return;
        at.next(tiles);
        ++t;
        load(a, seg1);
    }
};

// The issuer (one lane).
template <int D>
__device__ __forceinline__ void kv_mma(const BwArgs& a, uint8_t* smem, uint64_t* bars, uint32_t tmem, int seg0,
                                       int seg1, const Abort& ab) {
    using C = KvCfg<D>;
    constexpr uint32_t idesc_acc = idesc_bf16(128, D, false, true);
    constexpr uint64_t kPairDesc = C::kPair >> 4, kTileDesc = C::kTile >> 4, kItemDesc = (kItem * 128) >> 4;
    const uint64_t k_major = smem_desc_sw128(smem_u32(smem), 16, 1024);
    const uint64_t mn_major = smem_desc_sw128(smem_u32(smem), kHalfBytes, 1024);
    // rows of an item, in 16s
    auto rows16 = [&](const ItemWalk& w, int half) {
        const int n = w.x >= (w.tiles - 1) * kTileItems ? w.last_rows : a.tpt * a.r;
        return (uint32_t)((min(kItem, n - half * kItem) + 15) & ~15);
    };
    ItemWalk A, B;
    A.t = B.t = seg0;
    A.load(a, seg1);
    B.load(a, seg1);
    uint32_t slotA = 0, slotB = 0, p_ph = 0, acc_ph = 1, ph = 0;
    auto landed = [&](uint32_t pair) -> bool {
        if (!mbar_wait<true>(&bars[C::kFull + pair], (ph >> pair) & 1, ab, 83)) return false;
        ph ^= 1u << pair;
        return true;
    };
    auto scores = [&]() -> bool {
        const int m = A.x >> 1, half = A.x & 1;
        const uint32_t pair = A.at.tile(m);
        if (A.x == 0 && !landed(A.at.kv)) return false;
        if (half == 0 && !landed(pair)) return false;
        tc_fence_after();
        const uint64_t kd = k_major + A.at.kv * kPairDesc, qd = k_major + pair * kPairDesc + half * kItemDesc;
        const uint32_t id = idesc_bf16(128, rows16(A, half), false, false), col = tmem + slotA * 128;
        one_scores<D>(col, kd, qd, id);
        one_scores<D>(col + 64, kd + kTileDesc, qd + kTileDesc, id);
        one_commit(&bars[C::kSDFull + slotA]);
        if (A.last()) one_commit(&bars[C::kEmpty + A.at.kv]);
        slotA ^= 1;
        A.next(a, seg1);
        return true;
    };
    for (int i = 0; i < 2; ++i)
        if (A.t < seg1 && !scores()) return;
    while (B.t < seg1) {
        const int m = B.x >> 1, half = B.x & 1;
        const uint32_t pair = B.at.tile(m), col = tmem + slotB * 128;
        const bool last = B.last();
        if (B.x == 0) {   // the accumulators of the unit before have been read
            if (!mbar_wait<true>(&bars[C::kAccFree], acc_ph, ab, 85)) return;
            acc_ph ^= 1;
        }
        if (!mbar_wait<true>(&bars[C::kPFull + slotB], p_ph, ab, 86)) return;
        tc_fence_after();
        const uint64_t qd = mn_major + pair * kPairDesc + half * kItemDesc;
        const uint32_t steps = rows16(B, half) >> 4;
        one_sums(tmem + 256, col, col + 16, qd + kTileDesc, idesc_acc, steps, B.x > 0);
        one_sums(tmem + 384, col + 64, col + 80, qd, idesc_acc, steps, B.x > 0);
        p_ph ^= slotB;
        slotB ^= 1;
        if (half || last) one_commit(&bars[C::kEmpty + pair]);
        if (last) one_commit(&bars[C::kAccFull]);
        B.next(a, seg1);
        if (A.t < seg1 && !scores()) return;
    }
}

// The (lse, delta) of row 32 half + lane of item x of a unit.
template <bool kSm>
__device__ __forceinline__ float2 row_stats(const PrefixUnit& u, const BwArgs& a, int items, int x,
                                            int half, int lane) {
    float2 v = make_float2(INFINITY, 0.0f);
    if (kSm && x < items) {
        const int m = x >> 1, row = (x & 1) * kItem + 32 * half + lane;
        if (row < tile_rows(u, a, m)) {
            const int tt = row / a.r;
            const int64_t at = (int64_t)(u.tok + m * a.tpt + tt) * a.H + u.hk * a.r + (row - tt * a.r);
            const float l = a.lse[at];
            v.x = l == -INFINITY ? INFINITY : l * kLog2e;   // a row without keys: weights 0
            v.y = a.delta[at];
        }
    }
    return v;
}

template <int D, int ACT>
__device__ __forceinline__ void kv_rows(const BwArgs& a, uint8_t* smem, uint64_t* bars, uint32_t tmem, int seg0,
                                        int seg1, const Abort& ab) {
    using C = KvCfg<D>;
    constexpr bool kSm = ACT == kSoftmax;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = (warp - 4) >> 2, quarter = warp & 3;
    const int key = quarter * 32 + lane;   // TMEM lane
    const uint32_t col = tmem + ((uint32_t)(quarter * 32) << 16) + s * 128;
    // a warp's row statistics, two items' in turn
    float2* stat = reinterpret_cast<float2*>(smem + C::kOffStat) + (warp - 4) * 128;
    const ActScale ks = act_scale<ACT>(a.alpha);
    uint32_t e0 = 0;
    Places at;
    PrefixUnit u = load_unit(a.units + seg0);
    int items = unit_items(u, a);
    // the statistics of this slot's next item, on their way while the one
    // before it is worked on
    float2 next0 = row_stats<kSm>(u, a, items, s, 0, lane);
    float2 next1 = row_stats<kSm>(u, a, items, s, 1, lane);
    for (int t = seg0; t < seg1; ++t) {
        const PrefixUnit coming = load_unit(a.units + min(t + 1, seg1 - 1));
        const bool banded = (u.flags & kPieceOwn) && a.windowed;
        const int jpos = u.j0 + key;
        // this slot's items of the unit: those with e0 + x of its parity
        int x = (int)((e0 ^ (uint32_t)s) & 1);
        const int coming_items = unit_items(coming, a), coming_x = (int)((e0 + items) ^ (uint32_t)s) & 1;
        if (x >= items) {   // none: the next unit's instead
            next0 = row_stats<kSm>(coming, a, coming_items, coming_x, 0, lane);
            next1 = row_stats<kSm>(coming, a, coming_items, coming_x, 1, lane);
        }
        for (; x < items; x += 2) {
            const uint32_t e = e0 + x;
            const int m = x >> 1, r0 = (x & 1) * kItem;
            const int n = min(kItem, tile_rows(u, a, m) - r0);
            float2* sb = stat + ((e >> 1) & 1) * 64;
            if (kSm) {
                sb[lane] = next0;
                sb[32 + lane] = next1;
                const bool more = x + 2 < items;
                next0 = row_stats<kSm>(more ? u : coming, a, more ? items : coming_items, more ? x + 2 : coming_x,
                                       0, lane);
                next1 = row_stats<kSm>(more ? u : coming, a, more ? items : coming_items, more ? x + 2 : coming_x,
                                       1, lane);
                __syncwarp();
            }
            if (!wg_wait<true>(&bars[C::kSDFull + s], (e >> 1) & 1, ab, 91)) return;
            tc_fence_after();
            const bool cut = banded || n < kItem;
            int lo = 0, hi = n;   // rows that see this key: positions jpos .. jpos + window - 1
            if (banded) {
                const int64_t first = (int64_t)(jpos - u.i0 - m * a.tpt) * a.r - r0;
                lo = (int)max((int64_t)0, first);
                hi = (int)max((int64_t)0, min((int64_t)n, first + (int64_t)a.window * a.r));
            }
#pragma unroll 1
            for (int c0 = 0; c0 < 64; c0 += 32) {   // (registers, and half the code)
                uint32_t sv[32], pv[32];
                tmem_ld32(col + c0, sv);
                tmem_ld32(col + 64 + c0, pv);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 32; c += 16) {
                    uint32_t pk[8], dk8[8];
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        float l0 = 0.f, l1 = 0.f, d0 = 0.f, d1 = 0.f, p0, p1, g0, g1;
                        if constexpr (kSm) {
                            const float4 st = *reinterpret_cast<const float4*>(sb + c0 + c + i);
                            l0 = st.x; d0 = st.y; l1 = st.z; d1 = st.w;
                        }
                        weights2<ACT>(__uint_as_float(sv[c + i]), __uint_as_float(sv[c + i + 1]),
                                      __uint_as_float(pv[c + i]), __uint_as_float(pv[c + i + 1]), ks, l0, l1, d0,
                                      d1, p0, p1, g0, g1);
                        if (cut) {
                            const int j = c + i, lo0 = lo - c0, hi0 = hi - c0;
                            const bool ok0 = j >= lo0 && j < hi0, ok1 = j + 1 >= lo0 && j + 1 < hi0;
                            p0 = ok0 ? p0 : 0.0f;
                            g0 = ok0 ? g0 : 0.0f;
                            p1 = ok1 ? p1 : 0.0f;
                            g1 = ok1 ? g1 : 0.0f;
                        }
                        pk[i >> 1] = pack_bf16x2(p0, p1);
                        dk8[i >> 1] = pack_bf16x2(g0, g1);
                    }
                    tmem_st8(col + (c0 + c) / 2, pk);   // over scores that have been read
                    tmem_st8(col + 64 + (c0 + c) / 2, dk8);
                }
            }
            tmem_st_wait();
            if (n & 15) {
                uint8_t* rows = smem + at.tile(m) * C::kPair;
                clear_rows<D>(rows, r0 + n, r0 + ((n + 15) & ~15), key);
                clear_rows<D>(rows + C::kTile, r0 + n, r0 + ((n + 15) & ~15), key);
                fence_proxy_async_smem();
            }
            tc_fence_before();
            mbar_arrive(&bars[C::kPFull + s]);
        }
        if (items > 0) at.next((u.ntok + a.tpt - 1) / a.tpt);
        e0 += items;
        u = coming;
        items = coming_items;
    }
}

// The units' dV and dK from TMEM to memory (a warpgroup of its own: short
// units would otherwise wait for it before their weights).
template <int D>
__device__ __forceinline__ void kv_drain(const BwArgs& a, uint64_t* bars, uint32_t tmem, int seg0, int seg1,
                                         const Abort& ab) {
    using C = KvCfg<D>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quarter = warp & 3;
    const int key = quarter * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16);
    uint32_t ph = 0;
    for (int t = seg0; t < seg1; ++t) {
        const PrefixUnit u = load_unit(a.units + t);
        const bool own = u.flags & kPieceOwn, real = key < u.nk;
        const int split = u.flags / kUnitPart;
        const int64_t at = ((int64_t)(u.k0 + key) * a.Hkv + u.hk) * D;
        __nv_bfloat16 *dv = (own ? a.dv : a.dvp) + at, *dk = (own ? a.dk : a.dkp) + at;
        const bool wide = !(((uintptr_t)dv | (uintptr_t)dk) & 31);
        if (u.ntok == 0) {   // keys that no row sees
            if (real)
                for (int c = 0; c < D / 8; ++c)
                    reinterpret_cast<uint4*>(dv)[c] = reinterpret_cast<uint4*>(dk)[c] = make_uint4(0u, 0u, 0u, 0u);
            continue;
        }
        if (!wg_wait<true>(&bars[C::kAccFull], ph, ab, 92)) return;
        ph ^= 1;
        tc_fence_after();
#pragma unroll 1
        for (int x = 0; x < 2 * D; x += 32) {
            const bool second = x >= D;
            const int c = second ? x - D : x;
            uint32_t v[32];
            tmem_ld32(trow + (second ? 384 : 256) + c, v);
            tmem_ld_wait();
            if (x + 32 == 2 * D) {
                tc_fence_before();
                mbar_arrive(&bars[C::kAccFree]);
            }
            const float f = second ? a.alpha : 1.0f;
            if (real && split) {   // one of several ranges of the rows
                float4* to = reinterpret_cast<float4*>(a.unit_parts + ((int64_t)(split - 1) * 256 + (second ? 128 : 0) + key) * D + c);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    to[i] = make_float4(__uint_as_float(v[4 * i]) * f, __uint_as_float(v[4 * i + 1]) * f,
                                        __uint_as_float(v[4 * i + 2]) * f, __uint_as_float(v[4 * i + 3]) * f);
            } else if (real) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t o[8];
#pragma unroll
                    for (int w = 0; w < 8; ++w)
                        o[w] = pack_bf16x2(__uint_as_float(v[16 * i + 2 * w]) * f,
                                           __uint_as_float(v[16 * i + 2 * w + 1]) * f);
                    store_sector((second ? dk : dv) + c + 16 * i, o, wide);
                }
            }
        }
    }
}

template <int D, int ACT>
__global__ void __launch_bounds__(kKvThreads, 1)
prefix_dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDO,
                  const __grid_constant__ CUtensorMap tmKp, const __grid_constant__ CUtensorMap tmVp,
                  const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const BwArgs a) {
    using C = KvCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_let_next();
    const int seg0 = a.seg[blockIdx.x], seg1 = a.seg[blockIdx.x + 1];
    if (seg0 == seg1) {
        grid_wait_previous();
        return;
    }
    if (threadIdx.x == 0) {
        for (int b = 0; b < C::kNumBars; ++b)
            mbar_init(&bars[b], b == C::kPFull || b == C::kPFull + 1 ? 128u : b == C::kAccFree ? 128u : 1u);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Abort ab{abort_flag, a.err, a.wait_ns};
    // 512 threads start with 128 registers: 2 * 80 + 2 * 176 four of them
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (warp == 0) {
            if (lane == 0) kv_producer<D>(&tmQ, &tmDO, &tmKp, &tmVp, &tmK, &tmV, a, smem, bars, seg0, seg1, ab);
            __syncwarp();
        } else if (warp == 1) {
            if (elect_one()) {
                kv_mma<D>(a, smem, bars, tmem, seg0, seg1, ab);
                // all of its products complete before TMEM is released
                one_commit(&bars[C::kMmaDone]);
                mbar_wait_teardown(&bars[C::kMmaDone], 0);
            }
            __syncwarp();
        }
    } else if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        kv_drain<D>(a, bars, tmem, seg0, seg1, ab);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        kv_rows<D, ACT>(a, smem, bars, tmem, seg0, seg1, ab);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    grid_wait_previous();   // (a kernel that nothing here reads from)
}

// ------------------------------------------------------------------------ dQ

template <int D>
struct DqCfg {
    static constexpr int kHalves = D / 64;
    static constexpr int kTile = 128 * D * 2;
    // V and K tiles in turn: V first, as it is done with after the scores and
    // K only after the sums, so that with 5 places both tiles of a block wait
    // for ones that were done with a block ago (K first: 109 us, not 99, where
    // 1024 rows meet 8192 keys in 16 heads)
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int kOffQ = 0, kOffDO = kTile, kOffKV = 2 * kTile;
    static constexpr int kOffBar = kOffKV + kStages * kTile;
    enum { kQFull = 0, kQEmpty, kFull, kEmpty = kFull + kStages, kSDFull = kEmpty + kStages, kSDFree,
           kPFull, kAccFull = kPFull + 2, kAccFree, kMmaDone, kNumBars };
    static constexpr int kSmem = kOffBar + kNumBars * 8 + 16 + 1024;
};

// A run: one row tile against the key blocks of one slot of a piece.
struct Run {
    int tok, rows, i0, part, blocks, step, first;
    int nk;
    __device__ __forceinline__ Run(const PrefixPiece& p, int s, int r) {
        const int nb = (p.nk + kBN - 1) / kBN;
        const bool dual = p.flags & kPieceDual;
        const bool second = s && !dual;
        tok = p.tok + (second ? p.nA : 0);
        i0 = p.i0 + (second ? p.nA : 0);
        rows = (second ? p.nB : p.nA) * r;
        part = s ? p.part1 : p.part0;
        step = dual ? 2 : 1;
        first = dual ? s : 0;
        blocks = part < 0 ? 0 : dual ? (s ? nb >> 1 : (nb + 1) >> 1) : nb;
        nk = p.nk;
    }
    __device__ __forceinline__ int block(int j) const { return first + j * step; }
    __device__ __forceinline__ int keys(int j) const { return min(kBN, nk - block(j) * kBN); }
};

template <int D>
__device__ __forceinline__ void dq_producer(const CUtensorMap* tmQ, const CUtensorMap* tmDO, const CUtensorMap* tmKp,
                            const CUtensorMap* tmVp, const CUtensorMap* tmK, const CUtensorMap* tmV,
                            const BwArgs& a, uint8_t* smem, uint64_t* bars, int seg0, int seg1,
                            const Abort& ab) {
    using C = DqCfg<D>;
    const uint64_t keep = policy_evict_last(), once = policy_evict_first();
    int32_t q_armed = -1, armed[C::kStages];
    for (int s = 0; s < C::kStages; ++s) armed[s] = -1;
    uint32_t nr = 0, c = 0;
    for (int t = 2 * seg0; t < 2 * seg1; ++t) {
        const PrefixPiece p = load_piece(a.pieces + (t >> 1));
        const Run run(p, t & 1, a.r);
        if (run.blocks == 0) continue;
        if (!mbar_wait<true>(&bars[C::kQEmpty], (nr & 1) ^ 1, ab, 101)) goto unwind;
        if (!(a.stall && blockIdx.x == 0 && nr == 0)) {
            mbar_arrive_expect_tx(&bars[C::kQFull], 2 * (uint32_t)a.q_bytes);
            q_armed = (int32_t)(nr & 1);
#pragma unroll
            for (int hf = 0; hf < C::kHalves; ++hf) {
                tma_load_3d(tmQ, &bars[C::kQFull], smem + C::kOffQ + hf * kHalfBytes, hf * 64, p.hk * a.r, run.tok, once);
                tma_load_3d(tmDO, &bars[C::kQFull], smem + C::kOffDO + hf * kHalfBytes, hf * 64, p.hk * a.r, run.tok, once);
            }
        }
        const bool own = p.flags & kPieceOwn;
        for (int j = 0; j < run.blocks; ++j)
            for (int kv = 0; kv < 2; ++kv, ++c) {
                const CUtensorMap* map = kv ? (own ? tmK : tmKp) : (own ? tmV : tmVp);
                const uint32_t st = c % C::kStages, ph = (c / C::kStages) & 1;
                if (!mbar_wait<true>(&bars[C::kEmpty + st], ph ^ 1, ab, 102)) goto unwind;
                mbar_arrive_expect_tx(&bars[C::kFull + st], C::kTile);
                armed[st] = (int32_t)ph;
#pragma unroll
                for (int hf = 0; hf < C::kHalves; ++hf)
                    tma_load_2d(map, &bars[C::kFull + st], smem + C::kOffKV + st * C::kTile + hf * kHalfBytes,
                                p.hk * D + hf * 64, p.k0 + run.block(j) * kBN, keep);
            }
        ++nr;
    }
unwind:
    if (q_armed >= 0) mbar_wait_teardown(&bars[C::kQFull], (uint32_t)q_armed);
    for (int s = 0; s < C::kStages; ++s)
        if (armed[s] >= 0) mbar_wait_teardown(&bars[C::kFull + s], (uint32_t)armed[s]);
}

// The issuer (one lane).
template <int D>
__device__ __forceinline__ void dq_mma(const BwArgs& a, uint8_t* smem, uint64_t* bars, uint32_t tmem, int seg0,
                                       int seg1, const Abort& ab) {
    using C = DqCfg<D>;
    constexpr uint32_t idesc_acc = idesc_bf16(128, D, false, true), idesc_full = idesc_bf16(128, kBN, false, false);
    constexpr uint64_t kTileDesc = C::kTile >> 4, kHalfDesc = (64 * 128) >> 4;
    const uint64_t qd = smem_desc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
    const uint64_t dd = smem_desc_sw128(smem_u32(smem + C::kOffDO), 16, 1024);
    const uint64_t kv_k = smem_desc_sw128(smem_u32(smem + C::kOffKV), 16, 1024);
    const uint64_t kv_mn = smem_desc_sw128(smem_u32(smem + C::kOffKV), kHalfBytes, 1024);
    // ring places of the V whose scores come next (its K is behind it) and of
    // the K whose sums do
    RingAt<C::kStages> v, kB;
    kB.next();
    uint32_t slot = 0, p_ph = 0, q_ph = 0, acc_ph = 1, s_ph = 1;
    for (int t = 2 * seg0; t < 2 * seg1; ++t) {
        const PrefixPiece p = load_piece(a.pieces + (t >> 1));
        const Run run(p, t & 1, a.r);
        if (run.blocks == 0) continue;
        const uint32_t last16 = (uint32_t)((run.keys(run.blocks - 1) + 15) & ~15);
        const uint32_t idesc_last = idesc_bf16(128, last16, false, false);
        auto scores = [&](bool last) -> bool {
            RingAt<C::kStages> k = v;
            k.next();
            if (!mbar_wait<true>(&bars[C::kFull + v.st], v.ph, ab, 104) ||
                !mbar_wait<true>(&bars[C::kFull + k.st], k.ph, ab, 105) ||
                !mbar_wait<true>(&bars[C::kSDFree], s_ph, ab, 108))
                return false;
            s_ph ^= 1;
            tc_fence_after();
            const uint32_t id = last ? idesc_last : idesc_full;
            one_scores<D>(tmem, qd, kv_k + k.st * kTileDesc, id);
            one_scores<D>(tmem + 128, dd, kv_k + v.st * kTileDesc, id);
            one_commit(&bars[C::kSDFull]);
            one_commit(&bars[C::kEmpty + v.st]);
            if (last) one_commit(&bars[C::kQEmpty]);
            v = k;
            v.next();
            return true;
        };
        if (!mbar_wait<true>(&bars[C::kQFull], q_ph, ab, 103)) return;
        q_ph ^= 1;
        if (!scores(run.blocks == 1)) return;
        for (int j = 0; j < run.blocks; ++j) {
            const bool last = j == run.blocks - 1;
            if (!last && !scores(j == run.blocks - 2)) return;
            if (j == 0) {
                if (!mbar_wait<true>(&bars[C::kAccFree], acc_ph, ab, 106)) return;
                acc_ph ^= 1;
            }
            if (!mbar_wait<true>(&bars[C::kPFull + slot], p_ph, ab, 107)) return;
            tc_fence_after();
            const uint32_t col = tmem + 384 + slot * 64;
            const uint64_t kd = kv_mn + kB.st * kTileDesc;
            const uint32_t steps = (last ? last16 : (uint32_t)kBN) >> 4;
            one_sums(tmem + 256, col, col + 16, kd, idesc_acc, min(steps, 4u), j > 0);
            if (steps > 4) one_sums(tmem + 256, col + 32, col + 48, kd + kHalfDesc, idesc_acc, steps - 4, 1);
            one_commit(&bars[C::kEmpty + kB.st]);
            if (last) one_commit(&bars[C::kAccFull]);
            p_ph ^= slot;
            slot ^= 1;
            kB.next();
            kB.next();
        }
    }
}

template <int D, int ACT>
__device__ __forceinline__ void dq_rows(const BwArgs& a, uint8_t* smem, uint64_t* bars, uint32_t tmem, int seg0,
                                        int seg1, const Abort& ab) {
    using C = DqCfg<D>;
    constexpr bool kSm = ACT == kSoftmax;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = (warp - 4) >> 2, quarter = warp & 3;   // s: which 64 keys of a block
    const int row = quarter * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t col = trow + s * 64;
    const ActScale ks = act_scale<ACT>(a.alpha);
    const int rt = row / a.r, rj = row - rt * a.r;
    uint32_t acc_ph = 0, e = 0;
    RingAt<C::kStages> ring;   // of K
    ring.next();
    for (int t = 2 * seg0; t < 2 * seg1; ++t) {
        const PrefixPiece p = load_piece(a.pieces + (t >> 1));
        const Run run(p, t & 1, a.r);
        if (run.blocks == 0) continue;
        const bool real = row < run.rows;
        const bool banded = (p.flags & kPieceOwn) && a.windowed;
        const int ipos = run.i0 + rt;
        float lse2 = INFINITY, delta = 0.0f;
        if (kSm && real) {
            const int64_t at = (int64_t)(run.tok + rt) * a.H + p.hk * a.r + rj;
            const float l = a.lse[at];
            lse2 = l == -INFINITY ? INFINITY : l * kLog2e;
            delta = a.delta[at];
        }
        for (int j = 0; j < run.blocks; ++j, ++e) {
            const int n = run.keys(j) - s * 64;   // of this warpgroup's 64
            const bool cut = banded || n < 64;
            int lo = 0, hi = n;   // columns this row sees
            if (banded) {
                const int at = ipos - (p.j0 + run.block(j) * kBN + s * 64);
                hi = min(hi, at + 1);
                lo = at >= a.window ? at - a.window + 1 : 0;
            }
            if (!wg_wait<true>(&bars[C::kSDFull], e & 1, ab, 111)) return;
            tc_fence_after();
            uint32_t sv[64], pv[64];
#pragma unroll
            for (int c = 0; c < 64; c += 32) {
                tmem_ld32(col + c, *reinterpret_cast<uint32_t(*)[32]>(sv + c));
                tmem_ld32(col + 128 + c, *reinterpret_cast<uint32_t(*)[32]>(pv + c));
            }
            tmem_ld_wait();
            tc_fence_before();
            mbar_arrive(&bars[C::kSDFree]);   // the next block's scores may come
            if (n > 0) {
                const uint32_t to = trow + 384 + (e & 1) * 64 + s * 32;
#pragma unroll
                for (int c = 0; c < 64; c += 16) {
                    uint32_t dk8[8];
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        float p0, p1, g0, g1;
                        weights2<ACT>(__uint_as_float(sv[c + i]), __uint_as_float(sv[c + i + 1]),
                                      __uint_as_float(pv[c + i]), __uint_as_float(pv[c + i + 1]), ks, lse2, lse2,
                                      delta, delta, p0, p1, g0, g1);
                        if (cut) {
                            if (c + i < lo || c + i >= hi) g0 = 0.0f;
                            if (c + i + 1 < lo || c + i + 1 >= hi) g1 = 0.0f;
                        }
                        dk8[i >> 1] = pack_bf16x2(g0, g1);
                    }
                    // (the sums two blocks before, which read this place, were
                    // issued before this block's scores and are complete)
                    tmem_st8(to + c / 2, dk8);
                }
                tmem_st_wait();
                if (n < 64 && (n & 15)) {
                    clear_rows<D>(smem + C::kOffKV + ring.st * C::kTile, s * 64 + n, s * 64 + ((n + 15) & ~15), row);
                    fence_proxy_async_smem();
                }
            }
            ring.next();
            ring.next();
            tc_fence_before();
            mbar_arrive(&bars[C::kPFull + (e & 1)]);
        }
        if (!wg_wait<true>(&bars[C::kAccFull], acc_ph, ab, 112)) return;
        acc_ph ^= 1;
        tc_fence_after();
        float4* out = reinterpret_cast<float4*>(a.parts) + (int64_t)run.part * (D / 4) + row;
        {   // this warpgroup's half of the columns
            const int c0 = s * (D / 2);
            uint32_t o[D / 2];
#pragma unroll
            for (int c = 0; c < D / 2; c += 32) tmem_ld32(trow + 256 + c0 + c, *reinterpret_cast<uint32_t(*)[32]>(o + c));
            tmem_ld_wait();
            tc_fence_before();
            mbar_arrive(&bars[C::kAccFree]);
            if (real) {
#pragma unroll
                for (int e = 0; e < D / 8; ++e)
                    out[(int64_t)(c0 / 4 + e) * run.rows] =
                        make_float4(__uint_as_float(o[4 * e]) * a.alpha, __uint_as_float(o[4 * e + 1]) * a.alpha,
                                    __uint_as_float(o[4 * e + 2]) * a.alpha, __uint_as_float(o[4 * e + 3]) * a.alpha);
            }
        }
    }
}

template <int D, int ACT>
__global__ void __launch_bounds__(kThreads, 1)
prefix_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDO,
                 const __grid_constant__ CUtensorMap tmKp, const __grid_constant__ CUtensorMap tmVp,
                 const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                 const BwArgs a) {
    using C = DqCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_let_next();
    const int seg0 = a.seg[blockIdx.x], seg1 = a.seg[blockIdx.x + 1];
    if (seg0 == seg1) {
        grid_wait_previous();
        return;
    }
    if (threadIdx.x == 0) {
        for (int b = 0; b < C::kNumBars; ++b)
            mbar_init(&bars[b], b == C::kPFull || b == C::kPFull + 1 || b == C::kSDFree || b == C::kAccFree ? 256u : 1u);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Abort ab{abort_flag, a.err, a.wait_ns};
    // 384 threads start with 168 registers: 88 + 2 * 208 a triple
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 0) {
            if (lane == 0) dq_producer<D>(&tmQ, &tmDO, &tmKp, &tmVp, &tmK, &tmV, a, smem, bars, seg0, seg1, ab);
            __syncwarp();
        } else if (warp == 1) {
            if (elect_one()) {
                dq_mma<D>(a, smem, bars, tmem, seg0, seg1, ab);
                // all of its products complete before TMEM is released
                one_commit(&bars[C::kMmaDone]);
                mbar_wait_teardown(&bars[C::kMmaDone], 0);
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        dq_rows<D, ACT>(a, smem, bars, tmem, seg0, seg1, ab);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    grid_wait_previous();   // (a kernel that nothing here reads from)
}

template <typename K>
gdpa_status go(K kern, int threads, int smem, std::atomic<uint64_t>& done, PrefixPlan& p, const CUtensorMap* m, const BwArgs& a,
               cudaStream_t st) {
    if (!allow_smem(kern, smem, p.device, done)) return GDPA_ERR_CUDA;
    const bool ok = launch_kernel(kern, dim3((unsigned)p.S), threads, smem, st, p.chain > 0, m[0], m[1], m[2], m[3],
                                  m[4], m[5], a);
    p.launches += 1;
    p.chain += 1;
    return ok ? GDPA_OK : GDPA_ERR_CUDA;
}

template <int D, int ACT>
gdpa_status launch(PrefixPlan& p, const CUtensorMap* m, BwArgs& a, cudaStream_t st) {
    gdpa_status s = GDPA_OK;
    if (p.useg[p.S] > 0) {
        a.seg = p.dev_useg();
        a.stall = p.stall == 1;
        static std::atomic<uint64_t> done{0};
        s = go(prefix_dkv_kernel<D, ACT>, kKvThreads, KvCfg<D>::kSmem, done, p, m, a, st);
    }
    if (s == GDPA_OK && p.seg[p.S] > 0) {
        a.seg = p.dev_seg();
        a.stall = p.stall == 2;
        static std::atomic<uint64_t> done{0};
        s = go(prefix_dq_kernel<D, ACT>, kThreads, DqCfg<D>::kSmem, done, p, m, a, st);
    }
    return s;
}

}  // namespace

gdpa_status launch_prefix_tc_bwd(PrefixPlan& p, const PrefixIO& io, const float* delta, cudaStream_t st) {
    if (p.seg[p.S] == 0 && p.useg[p.S] == 0) return GDPA_OK;
    CUtensorMap m[6];
    const uint64_t krow = (uint64_t)p.Hkv * p.d;
    // tensors without rows are never loaded from: any map will do
    const void* kp = p.Tp ? io.kp : io.k;
    const void* vp = p.Tp ? io.vp : io.v;
    const void* k = p.Tkv ? io.k : io.kp;
    const void* v = p.Tkv ? io.v : io.vp;
    const uint64_t np = p.Tp ? p.Tp : p.Tkv, nk = p.Tkv ? p.Tkv : p.Tp;
    const uint64_t nq = p.Tq ? p.Tq : 1;
    if (!tc::make_tmap_rows(&m[0], p.Tq ? io.q : kp, nq, p.Tq ? p.H : p.Hkv, p.d, p.Tq ? p.r : 1, p.tpt) ||
        !tc::make_tmap_rows(&m[1], p.Tq ? io.d_o : kp, nq, p.Tq ? p.H : p.Hkv, p.d, p.Tq ? p.r : 1, p.tpt) ||
        !tc::make_tmap_bf16(&m[2], kp, np, krow, 128) || !tc::make_tmap_bf16(&m[3], vp, np, krow, 128) ||
        !tc::make_tmap_bf16(&m[4], k, nk, krow, 128) || !tc::make_tmap_bf16(&m[5], v, nk, krow, 128))
        return GDPA_ERR_CUDA;
    BwArgs a;
    a.units = p.dev_units();
    a.pieces = p.dev_pieces();
    a.seg = nullptr;
    a.lse = io.lse;
    a.delta = delta;
    a.parts = p.d_parts;
    a.unit_parts = p.d_grad;
    a.dkp = (__nv_bfloat16*)io.dkp;
    a.dvp = (__nv_bfloat16*)io.dvp;
    a.dk = (__nv_bfloat16*)io.dk;
    a.dv = (__nv_bfloat16*)io.dv;
    a.H = p.H;
    a.Hkv = p.Hkv;
    a.r = p.r;
    a.tpt = p.tpt;
    a.windowed = p.mask == GDPA_MASK_CAUSAL_WINDOW;
    a.window = p.window;
    a.q_bytes = p.tpt * p.r * p.d * 2;
    a.alpha = io.alpha;
    a.err = p.dev_err();
    a.wait_ns = tc::wait_limit_ns(p.wait_limit_us);
    a.stall = 0;
    gdpa_status s = GDPA_OK;
    if (p.d == 128) {
        if (io.act == kSoftmax)
            s = launch<128, kSoftmax>(p, m, a, st);
        else
            GDPA_DISPATCH_ACT(io.act, A, s = launch<128, A>(p, m, a, st))
    } else {
        if (io.act == kSoftmax)
            s = launch<64, kSoftmax>(p, m, a, st);
        else
            GDPA_DISPATCH_ACT(io.act, A, s = launch<64, A>(p, m, a, st))
    }
    return s;
}

}  // namespace gdpa
