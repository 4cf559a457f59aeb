// Host planner of shared-prefix attention.
//
// Forward units are (group, key head, one or two row tiles) against the
// group's prefix, and (sample, key head, one or two row tiles) against the
// sample's own keys, in steps of one 128-key block for two row tiles, or of
// two blocks for a single tile (whose two slots take alternate blocks).  All
// units' steps are dealt in equal shares, one per CTA, so that ragged groups
// balance and a short batch spreads a long prefix over every SM; a cut inside
// a unit costs another part of its rows to merge, which the shares allow for
// (kPieceCost steps a piece).
#include <algorithm>

#include "prefix_internal.h"

namespace gdpa {
namespace {

// Steps a piece costs beside its own.  (Forward of 512 rows on 16384 keys, 8
// heads: 60 us; 81 with 0, 69 with 1, 62 with 6.  2 x 2048 rows on 32768 keys:
// 423 us; 437, 434, 427.)
constexpr int kPieceCost = 3;

// Own keys of samples with at most this many packed rows, keys, and pairs of
// them are streamed by warp-level kernels (prefix_own.cu), without a tile's
// latency; with more pairs the tensor core's products are worth it.  Forward
// and backward in us, d = 128, 4 heads, with this limit of pairs, with 512 and
// with none: 300 samples of 16 to 64 rows on 8 to 64 keys, d = 64: 58, 141; 88,
// 166; 57, 140.  500 of 6 to 8 rows on 100 to 500 keys, d = 64: 56, 86; 94, 170;
// 55, 86.  200 of 48 to 64 rows on 64 to 400 keys: 69, 144; 62, 116; 115, 311.
constexpr int kSmallRows = 64;
constexpr int kSmallKeys = 512;
constexpr int kSmallPairs = 4096;

// Rows of a kind: a walk in blocks steps past the last one by less than two
// blocks, in 32 bits.
constexpr int64_t kMaxRows = 0x7fffffff - 4095;

constexpr int kSplitTiles = 4;   // row tiles that a range of a split backward unit has at least

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Unit {
    PrefixPiece p;       // the whole unit as one piece
    int64_t steps;
    int32_t tileA, tileB;   // merge tiles (prefix units)
};

bool good_offsets(const int32_t* off, int n) {
    if (!off || off[0] != 0) return false;
    for (int i = 0; i < n; ++i)
        if (off[i + 1] < off[i]) return false;
    return true;
}

bool is_small(const PrefixPlan& p, int32_t lq, int32_t lk) {
    const int64_t rows = (int64_t)lq * p.r;
    return (p.d == 64 || p.d == 128) && rows <= kSmallRows && lk <= kSmallKeys && rows * lk <= kSmallPairs;
}

int64_t steps_of(const PrefixPiece& p) {
    const int64_t nb = cdiv(p.nk, kBN);
    return p.flags & kPieceDual ? cdiv(nb, 2) : nb;
}

// The CUDA-core kernels' row blocks: 8 rows (2 a warp) or 32 (8 a warp).
//
// 2 rows a warp: a quarter of the instructions on a warp's way, for four times
// the reads of keys.  Better where few blocks are there to hide them (4 users of
// 40 rows, 500 keys, d = 32: 21 us, 25 with 8 rows; one row against 4096 keys, d
// = 128: 26 and 42), where the keys meet few rows, and up to 48 columns always (8
// users of 256 rows, 2000 keys, 4 heads, d = 48: 272 and 384; samples of 36 rows
// and 120 own keys, d = 32: 312 and 401); from 64 on 8 rows (256 rows, 2000 keys,
// d = 64: 248, 303 with 2; 512 rows, d = 128: 431, 663).
void make_row_blocks(PrefixPlan& p) {
    int64_t blocks = 0, work = 0, work8 = 0;
    auto rows_of = [&](const PrefixPiece& q, int slot) -> int64_t {
        if ((slot ? q.part1 : q.part0) < 0) return 0;
        return (int64_t)(slot && !(q.flags & kPieceDual) ? q.nB : q.nA) * p.r;
    };
    for (const PrefixPiece& q : p.pieces)
        for (int slot = 0; slot < 2; ++slot) {
            const int64_t rows = rows_of(q, slot), keys = q.flags & kPieceDual ? cdiv(q.nk, 2) : q.nk;
            blocks += cdiv(rows, 32);
            work += cdiv(rows, 32) * keys;
            work8 += cdiv(rows, 8) * keys;
        }
    p.warp_rows = p.d < 64 || blocks <= 2 * p.S || work8 <= 2 * work ? 2 : 8;
    p.blocks.clear();
    for (size_t i = 0; i < p.pieces.size(); ++i)
        for (int slot = 0; slot < 2; ++slot) {
            const int64_t n = cdiv(rows_of(p.pieces[i], slot), 4 * p.warp_rows);
            for (int64_t sub = 0; sub < n; ++sub)
                p.blocks.push_back(RowBlock{(int32_t)i, (int32_t)(2 * sub + slot)});
        }
}

// Cut units with more rows than a share of all (few keys, many rows) into
// ranges of their tokens, so that every SM has work: each writes float32 sums
// of its own, which a kernel joins in order.  (Backward of 4 users, 2000 rows a
// head, on 100 keys: 8 heads sharing one, d = 128, 131 us, whole 331; 8 key
// heads 137 and 152; 17 users, 18144 rows on 40 keys of one float32 head, d =
// 32, 1055 and 3283.)
void split_units(PrefixPlan& p) {
    p.joins.clear();
    p.n_unit_parts = 0;
    // the tensor-core kernel has one CTA an SM, the others several
    const int64_t lanes = p.d == 64 || p.d == 128 ? p.S : 4 * (int64_t)p.S;
    int64_t total = 0;
    for (const PrefixUnit& u : p.units) total += cdiv(u.ntok, p.tpt);
    const int64_t share = std::max<int64_t>(cdiv(total, lanes), kSplitTiles);
    std::vector<PrefixUnit> out;
    for (const PrefixUnit& u : p.units) {
        const int64_t tiles = cdiv(u.ntok, p.tpt);
        if (2 * tiles <= 3 * share || p.n_unit_parts > 1 << 20) {   // (flags hold part numbers up to 2^23)
            out.push_back(u);
            continue;
        }
        const int64_t each = cdiv(tiles, cdiv(tiles, share)) * p.tpt;   // tokens
        PrefixUnit j = u;
        j.tok = (int32_t)p.n_unit_parts;
        for (int64_t at = 0; at < u.ntok; at += each) {
            PrefixUnit c = u;
            c.tok += (int32_t)at;
            c.i0 += (int32_t)at;
            c.ntok = (int32_t)std::min<int64_t>(each, u.ntok - at);
            c.flags |= (int32_t)(++p.n_unit_parts) * kUnitPart;
            out.push_back(c);
        }
        j.ntok = (int32_t)p.n_unit_parts - j.tok;
        p.joins.push_back(j);
    }
    p.units.swap(out);
}

}  // namespace

gdpa_status build_prefix_plan(PrefixPlan& p, const int32_t* q_off, const int32_t* kv_off,
                              const int32_t* group_off, const int32_t* prefix_off) {
    if (!good_offsets(q_off, p.B) || !good_offsets(kv_off, p.B) || !good_offsets(group_off, p.G) ||
        !good_offsets(prefix_off, p.G) || group_off[p.G] != p.B)
        return GDPA_ERR_INVALID_ARG;
    p.Tq = q_off[p.B];
    p.Tkv = kv_off[p.B];
    p.Tp = prefix_off[p.G];
    if (p.Tq > kMaxRows || p.Tkv > kMaxRows || p.Tp > kMaxRows) return GDPA_ERR_UNSUPPORTED;
    const int tpt = p.tpt;
    int64_t parts = 0;   // rows of the workspace given out
    std::vector<Unit> units;
    p.own.assign((size_t)p.Tq, PrefixOwn{0, 0, 0, 0});
    for (int g = 0; g < p.G; ++g) {
        const int32_t t0 = q_off[group_off[g]], nt = q_off[group_off[g + 1]] - t0;
        const int32_t np = prefix_off[g + 1] - prefix_off[g];
        const int nm = (int)cdiv(nt, tpt);
        for (int hk = 0; hk < p.Hkv; ++hk) {
            const int32_t first = (int32_t)p.tiles.size();
            for (int m = 0; m < nm; ++m)
                p.tiles.push_back(PrefixTile{t0 + m * tpt, std::min(tpt, nt - m * tpt), hk, 0, 0, {}});
            if (np == 0) continue;
            for (int m = 0; m < nm; m += 2) {
                Unit u{};
                u.tileA = first + m;
                u.tileB = m + 1 < nm ? first + m + 1 : -1;
                u.p.tok = p.tiles[u.tileA].tok;
                u.p.nA = p.tiles[u.tileA].n;
                u.p.nB = u.tileB >= 0 ? p.tiles[u.tileB].n : 0;
                u.p.hk = hk;
                u.p.k0 = prefix_off[g];
                u.p.nk = np;
                u.p.flags = u.tileB >= 0 ? 0 : kPieceDual;
                u.steps = steps_of(u.p);
                units.push_back(u);
            }
        }
    }
    const size_t n_prefix = units.size();
    // own keys: row tiles counted from the sample's first token
    const bool windowed = p.mask == GDPA_MASK_CAUSAL_WINDOW;
    std::vector<Unit> small_units;
    for (int b = 0; b < p.B; ++b) {
        const int32_t lq = q_off[b + 1] - q_off[b], lk = kv_off[b + 1] - kv_off[b];
        if (lq == 0 || lk == 0) continue;
        const bool small = is_small(p, lq, lk);
        std::vector<Unit>& to = small ? small_units : units;
        for (int32_t i = 0; i < lq;) {
            const int32_t nA = std::min(tpt, lq - i), nB = std::min(tpt, lq - i - nA);
            // hull of the keys these rows see
            const int32_t lo = windowed ? std::max(0, i - p.window + 1) : 0;
            const int32_t hi = windowed ? std::min(lk, i + nA + nB) : lk;
            if (hi > lo) {
                Unit u{};
                u.tileA = u.tileB = -1;
                u.p.tok = q_off[b] + i;
                u.p.nA = nA;
                u.p.nB = nB;
                u.p.k0 = kv_off[b] + lo;
                u.p.nk = hi - lo;
                u.p.flags = kPieceOwn | (nB > 0 || small ? 0 : kPieceDual);
                u.p.i0 = i;
                u.p.j0 = lo;
                u.steps = steps_of(u.p);
                const int layers = u.p.flags & kPieceDual && u.p.nk > kBN ? 2 : 1;
                const int32_t ra = nA * p.r, rb = nB * p.r;
                const size_t u0 = to.size();
                for (int hk = 0; hk < p.Hkv; ++hk) {
                    u.p.hk = hk;
                    u.p.part0 = (int32_t)(parts + (int64_t)hk * layers * ra);
                    u.p.part1 = layers == 2 ? u.p.part0 + ra : -1;
                    to.push_back(u);
                }
                for (int32_t t = 0; t < nA; ++t) {
                    PrefixOwn& o = p.own[u.p.tok + t];
                    o.part = (int32_t)parts;
                    o.row0 = t * p.r;
                    o.layers = layers;
                    o.rows = ra;
                }
                parts += (int64_t)p.Hkv * layers * ra;
                if (nB > 0) {
                    for (int hk = 0; hk < p.Hkv; ++hk)
                        to[u0 + hk].p.part1 = (int32_t)(parts + (int64_t)hk * rb);
                    for (int32_t t = 0; t < nB; ++t) {
                        PrefixOwn& o = p.own[u.p.tok + nA + t];
                        o.part = (int32_t)parts;
                        o.row0 = t * p.r;
                        o.layers = 1;
                        o.rows = rb;
                    }
                    parts += (int64_t)p.Hkv * rb;
                }
                if (parts > 0x7fffffff) return GDPA_ERR_UNSUPPORTED;
            }
            i += nA + nB;
        }
    }
    // Cut the steps into S shares.  A prefix unit gives as many whole shares as
    // it has; those of one (group, key head) start on the same keys at the same
    // time, so that its row tiles read them from L2 once.  What is left of the
    // units, and the own units, form one line that is cut into the remaining
    // shares.
    int64_t total = 0;
    for (const Unit& u : units) total += u.steps + kPieceCost;
    auto piece_of = [&](size_t n, int64_t done, int64_t take) {
        const Unit& u = units[n];
        const int64_t unit_keys = u.p.flags & kPieceDual ? 2 * kBN : kBN;
        PrefixPiece q = u.p;
        q.k0 = (int32_t)(u.p.k0 + done * unit_keys);
        q.nk = (int32_t)std::min<int64_t>(u.p.nk - done * unit_keys, take * unit_keys);
        if (n < n_prefix) q.pad = (int32_t)n;
        return q;
    };
    const int64_t base = cdiv(total, p.S);
    for (int64_t budget = std::max<int64_t>(base, kPieceCost + 1);; budget += 1 + budget / 64) {
        p.pieces.clear();
        p.seg.assign((size_t)p.S + 1, 0);
        int cta = 0;
        bool ok = true;
        const int64_t share = budget - kPieceCost;
        // whole shares, the units of a (group, key head) side by side
        for (size_t n = 0; n < n_prefix && ok;) {
            size_t e = n + 1;
            while (e < n_prefix && units[e].p.k0 == units[n].p.k0 && units[e].p.hk == units[n].p.hk) ++e;
            int64_t most = 0;
            for (size_t i = n; i < e; ++i) most = std::max(most, units[i].steps / share);
            for (int64_t c = 0; c < most && ok; ++c)
                for (size_t i = n; i < e; ++i) {
                    if (units[i].steps / share <= c) continue;
                    if (cta >= p.S) {
                        ok = false;
                        break;
                    }
                    p.pieces.push_back(piece_of(i, c * share, share));
                    p.seg[(size_t)++cta] = (int32_t)p.pieces.size();
                }
            n = e;
        }
        // the line
        int64_t left = budget;
        bool open = false;   // the current share has pieces
        for (size_t n = 0; n < units.size() && ok; ++n) {
            const Unit& u = units[n];
            const bool own = n >= n_prefix;   // own units stay whole (their parts are laid out above)
            int64_t done = own ? 0 : u.steps / share * share;
            while (done < u.steps) {
                int64_t take = left - kPieceCost;
                if (open && (take < 1 || (own && take < u.steps))) {
                    p.seg[(size_t)++cta] = (int32_t)p.pieces.size();
                    left = budget;
                    open = false;
                    continue;
                }
                if (cta >= p.S) {
                    ok = false;
                    break;
                }
                take = own ? u.steps : std::min(take, u.steps - done);
                p.pieces.push_back(piece_of(n, done, take));
                open = true;
                done += take;
                left -= take + kPieceCost;
            }
        }
        if (ok) {
            if (open) ++cta;
            for (int c = cta; c <= p.S; ++c) p.seg[(size_t)c] = (int32_t)p.pieces.size();
            break;
        }
    }
    // a unit's pieces, in order of keys, for its parts
    std::vector<std::vector<int32_t>> of_unit(n_prefix);
    for (size_t i = 0; i < p.pieces.size(); ++i)
        if (!(p.pieces[i].flags & kPieceOwn)) of_unit[(size_t)p.pieces[i].pad].push_back((int32_t)i);
    for (size_t n = 0; n < n_prefix; ++n) {
        const Unit& u = units[n];
        const bool dual = u.p.flags & kPieceDual;
        const int32_t ra = u.p.nA * p.r, rb = u.p.nB * p.r;
        PrefixTile& ta = p.tiles[u.tileA];
        ta.part = (int32_t)parts;
        for (int32_t i : of_unit[n]) {
            PrefixPiece& q = p.pieces[(size_t)i];
            q.part0 = (int32_t)parts;
            parts += ra;
            q.part1 = -1;
            if (dual && q.nk > kBN) {
                q.part1 = (int32_t)parts;
                parts += ra;
            }
        }
        ta.layers = (int32_t)((parts - ta.part) / ra);
        if (!dual) {
            p.tiles[u.tileB].part = (int32_t)parts;
            p.tiles[u.tileB].layers = (int32_t)of_unit[n].size();
            for (int32_t i : of_unit[n]) {
                p.pieces[(size_t)i].part1 = (int32_t)parts;
                parts += rb;
            }
        }
        if (parts > 0x7fffffff) return GDPA_ERR_UNSUPPORTED;
    }
    for (PrefixPiece& q : p.pieces) q.pad = 0;
    for (const Unit& u : small_units) p.pieces.push_back(u.p);
    p.n_part_rows = parts;
    p.max_layers = 0;
    for (const PrefixTile& t : p.tiles) p.max_layers = std::max(p.max_layers, t.layers);
    make_row_blocks(p);

    // backward: one unit per 128-key block, against all rows that see it
    p.units.clear();
    for (int g = 0; g < p.G; ++g) {
        const int32_t t0 = q_off[group_off[g]], nt = q_off[group_off[g + 1]] - t0;
        for (int32_t k = prefix_off[g]; k < prefix_off[g + 1]; k += kBN)
            for (int hk = 0; hk < p.Hkv; ++hk)
                p.units.push_back(PrefixUnit{k, std::min(kBN, prefix_off[g + 1] - k), t0, nt, hk, 0, 0, 0});
    }
    std::vector<PrefixUnit> small_blocks, more;
    for (int b = 0; b < p.B; ++b) {
        const int32_t lq = q_off[b + 1] - q_off[b], lk = kv_off[b + 1] - kv_off[b];
        const bool small = lq > 0 && is_small(p, lq, lk);
        for (int32_t j = 0; j < lk; j += kBN) {
            const int32_t nk = std::min(kBN, lk - j);
            // queries j <= i < j + nk - 1 + window
            const int32_t lo = windowed ? std::min(lq, j) : 0;
            const int32_t hi = windowed ? (int32_t)std::min<int64_t>(lq, (int64_t)j + nk - 1 + p.window) : lq;
            for (int hk = 0; hk < p.Hkv; ++hk)
                (small ? small_blocks : p.units)
                    .push_back(PrefixUnit{kv_off[b] + j, nk, q_off[b] + lo, std::max(0, hi - lo), hk, kPieceOwn,
                                          lo, j});
        }
        if (small && lk > 0)
            for (int hk = 0; hk < p.Hkv; ++hk) {
                const PrefixUnit u{kv_off[b], lk, q_off[b], lq, hk, kPieceOwn, 0, 0};
                (lq * p.r <= 8 ? p.smalls : more).push_back(u);
                p.eights.push_back(u);
                for (int32_t row = 8; row < lq * p.r; row += 8) {
                    p.eights.push_back(u);
                    p.eights.back().j0 = row;
                }
            }
    }
    p.n_small8 = (int64_t)p.smalls.size();
    p.smalls.insert(p.smalls.end(), more.begin(), more.end());
    split_units(p);
    // deal them by their row tiles (and a unit's own loads and stores) in
    // snake order, longest first
    const int64_t n = (int64_t)p.units.size();
    std::vector<std::vector<PrefixUnit>> queue((size_t)p.S);
    std::stable_sort(p.units.begin(), p.units.end(),
                     [](const PrefixUnit& x, const PrefixUnit& y) { return x.ntok > y.ntok; });
    for (int64_t i = 0; i < n; ++i) {
        const int64_t round = i / p.S, at = i % p.S;
        queue[(size_t)(round & 1 ? p.S - 1 - at : at)].push_back(p.units[(size_t)i]);
    }
    p.units.clear();
    p.useg.assign((size_t)p.S + 1, 0);
    for (int c = 0; c < p.S; ++c) {
        p.units.insert(p.units.end(), queue[(size_t)c].begin(), queue[(size_t)c].end());
        p.useg[(size_t)c + 1] = (int32_t)p.units.size();
    }
    p.units.insert(p.units.end(), small_blocks.begin(), small_blocks.end());
    return GDPA_OK;
}

}  // namespace gdpa
