// What the kernels of the attention over the history cache share: how all work
// is cut into equal shares on the device, and where a share's results go.
//
// An item is one tile of a sample's query rows that share a key head (row rho =
// token * G + head of the G query heads, TM rows a tile) against all the groups
// of 16 events that its sample's rows look at.  The lengths are only known on
// the device, so every CTA sums the units (groups of all items, and `lead` more
// an item for what starting and ending one costs) itself, takes the blockIdx-th
// equal share of them and walks the items that it meets: a segment is what a
// share holds of an item (shares that would start among an item's first `lead`
// units start at the item).  (Without `lead`, 128 users with 1 to 100000 events
// and a window of 1024: 64 us, the SMs busy for 43% of them.)  A segment that is a whole item
// gives outputs; other segments give parts (float32 sums, running maximum and
// sum) in the workspace, two slots a CTA: 2 c + 1 for the item that starts in
// CTA c and goes on in c + 1, c + 2, ..., whose slots 2 (c + 1), 2 (c + 2), ...
// hold the rest.  The merge kernel joins them in that order, so that results
// repeat bit for bit.
#pragma once

#include <atomic>

#include "act.cuh"
#include "cache_internal.h"

namespace gdpa {

// Floats of a slot of the workspace: a tile's sums, maxima and sums of weights, in
// whole 16-byte pieces (tiles of one row are not).
__host__ __device__ __forceinline__ int cache_slot(int TM, int d) { return (TM * (d + 2) + 3) & ~3; }

struct CacheDesc {
    int32_t parts;      // parts of the item that starts in this CTA (0: none to join)
    int32_t rows;       // real rows of its tile
    int32_t t0, h;      // the sample's first token, the key head
    int32_t rho0;       // first row of the tile
    int32_t pad[3];
};

struct AttnArgs {
    CacheView c;
    CacheWhere w;
    const void* q;
    int64_t qt, qh;     // strides in elements
    int q_wide;         // rows in 16-byte pieces
    void* o;
    float* lse;
    const int32_t* parents;
    float alpha;        // softmax: times log2 e
    int H, G, mask, window, sinks, act;
    int TM, RT;         // rows of a tile; row tiles of 16 side by side in a CTA
    int min_share, lead;
    uint64_t wait_ns;   // limit of a wait
    int stall;          // test hook: no CTA's first keys are ever complete
    float* part;
    CacheDesc* desc;
};

struct Sample {
    int t0, n;          // first token, tokens
    int start, end;     // events before the first row; events there are
    int lo_g, sink_g;   // first group of the window; groups of sinks before it
    int groups;         // >= 1
    int tiles;
};

__device__ __forceinline__ Sample sample_info(const AttnArgs& a, int b) {
    Sample s;
    const int T = (int)a.w.T;
    s.t0 = min(max(__ldg(a.w.off + b), 0), T);
    s.n = min(max(__ldg(a.w.off + b + 1), s.t0), T) - s.t0;
    s.start = a.w.starts ? min(__ldg(a.w.starts + b), kCacheMost) : 0;   // (behind every table: so that sums fit 32 bits)
    const int64_t cap = (int64_t)a.w.width << a.c.page_log;
    int64_t end = (int64_t)s.start + (a.mask == GDPA_CACHE_HISTORY ? 0 : s.n);
    if (s.start < 0) end = 0;
    s.end = (int)min(end, cap);
    const int lo = a.window > 0 ? (int)min((int64_t)s.end, max((int64_t)0, (int64_t)s.start - a.window + 1)) : 0;
    s.lo_g = lo / kCacheGroup;
    s.sink_g = (min(a.sinks, lo) + kCacheGroup - 1) / kCacheGroup;
    if (s.sink_g >= s.lo_g) s.lo_g = s.sink_g = 0;   // no gap between them
    const int end_g = (s.end + kCacheGroup - 1) / kCacheGroup;
    s.groups = max(1, s.sink_g + end_g - s.lo_g);
    s.tiles = (int)(((int64_t)s.n * a.G + a.TM - 1) / a.TM);
    return s;
}

__device__ __forceinline__ int64_t sample_units(const AttnArgs& a, int b) {
    const Sample s = sample_info(a, b);
    return (int64_t)s.tiles * a.c.heads * (s.groups + a.lead);
}

// What of a sample lies outside the cache is recorded once a launch.
__device__ __forceinline__ void sample_check(const AttnArgs& a, int b) {
    const Sample s = sample_info(a, b);
    if (s.n == 0) return;
    if (s.start < 0) cache_bad(a.c.err, kCacheBadStart, b, s.start);
    else if ((int64_t)s.start + (a.mask == GDPA_CACHE_HISTORY ? 0 : s.n) > s.end)
        cache_bad(a.c.err, kCacheBadEvent, b, s.end);
}

// x / y for x >= 0, y > 0: in 32 bits where they fit (a fifth of the instructions)
__device__ __forceinline__ int64_t divide(int64_t x, int64_t y) {
    if ((x | y) >> 32 == 0) return (uint32_t)x / (uint32_t)y;
    return x / y;
}

// A CTA's place in the work: its share [u, u_end) of the units, the sample b
// that holds u, and the unit at which b starts.  Where it starts inside an item,
// the `last` units that are left of that item come last: then the CTAs that hold
// tiles of the same sample read the same events at about the same time, from L2 (8 x
// 512 rows on 16384 bf16 events: 219 us, 229 in the order of the units).  Only in
// long shares: finding out costs a microsecond.
constexpr int kLongShare = 512;   // units
struct Share {
    int64_t u, u_end, size, b_first;
    int b, last;
    __device__ __forceinline__ bool more() const { return u < u_end || last > 0; }
};

template <int NT>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* tmp, int64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, m);
        if (lane >= m) x += y;
    }
    if (lane == 31) tmp[warp] = x;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
        if (i < warp) before += tmp[i];
        total += tmp[i];
    }
    __syncthreads();
    return before + x;   // inclusive
}

// tmp: shared, NT / 32 + 2 words.
template <int NT>
__device__ __forceinline__ Share find_share(const AttnArgs& a, int64_t* tmp) {
    int64_t mine = 0, first = 0;
#pragma unroll 4
    for (int b = threadIdx.x; b < a.w.B; b += NT) {
        const int64_t n = sample_units(a, b);
        if (b < NT) first = n;
        mine += n;
        if (blockIdx.x == 0) sample_check(a, b);
    }
    int64_t total, all;
    const int64_t scan0 = block_scan<NT>(first, tmp, total);   // of the first NT samples
    if (a.w.B > NT) block_scan<NT>(mine, tmp, all); else all = total;
    Share s;
    s.size = max(divide(all + gridDim.x - 1, gridDim.x), (int64_t)a.min_share);
    s.u = min((int64_t)blockIdx.x * s.size, all);
    s.u_end = min(s.u + s.size, all);
    if (threadIdx.x == 0) tmp[NT / 32] = -1;
    __syncthreads();
    if (s.u < s.u_end) {
        int64_t base = 0, scan = scan0, v = first;
        for (int b0 = 0;;) {
            if (base + scan > s.u && base + scan - v <= s.u) {
                tmp[NT / 32] = b0 + threadIdx.x;
                tmp[NT / 32 + 1] = base + scan - v;
            }
            base += total;
            b0 += NT;
            if (base > s.u || b0 >= a.w.B) break;
            v = b0 + (int)threadIdx.x < a.w.B ? sample_units(a, b0 + threadIdx.x) : 0;
            scan = block_scan<NT>(v, tmp, total);
        }
        __syncthreads();
    }
    s.b = (int)tmp[NT / 32];
    s.b_first = tmp[NT / 32 + 1];
    if (s.b < 0) s.u_end = s.u;
    s.last = 0;
    if (s.u < s.u_end && s.size >= kLongShare) {
        const Sample x = sample_info(a, s.b);
        const int64_t size = x.groups + a.lead, in = s.u - s.b_first, item = divide(in, size);
        const int64_t end = s.b_first + (item + 1) * size;
        if (in - item * size > a.lead && end < s.u_end && s.u_end <= s.b_first + x.tiles * a.c.heads * size) {
            s.last = (int)(end - s.u);
            s.u = end;
        }
    }
    __syncthreads();
    return s;
}

// One segment: a tile of rows, and which groups of events.
struct Segment {
    Sample s;
    int b, h, rho0, rows;     // rows: real ones of the tile
    int n;                    // groups to look at
    int na, a0, b0;           // group i is a0 + i (i < na), b0 + i (else)
    bool head, whole;         // starts its item; is all of it
    int parts;                // head: CTAs that the item spans
};

__device__ __forceinline__ int segment_group(const Segment& g, int i) { return i < g.na ? g.a0 + i : g.b0 + i; }

// The segment at s.u; moves s behind it.  Every thread of the CTA alike, whole
// warps together.  rows 0: the share has no more.
__device__ __forceinline__ Segment next_segment(const AttnArgs& a, Share& s) {
    Segment g;
    const int lane = threadIdx.x & 31;
    g.rows = g.n = g.na = g.parts = 0;
    const auto rest = [&] {   // on to what comes last; false: nothing does
        if (s.last <= 0) return false;
        s.u = (int64_t)blockIdx.x * s.size;
        s.u_end = s.u + s.last;
        s.last = 0;
        return true;
    };
    if (s.u >= s.u_end && !rest()) return g;
    for (;;) {   // the sample of s.u, 32 at a time over samples without rows
        g.s = sample_info(a, s.b);
        const int64_t n = (int64_t)g.s.tiles * a.c.heads * (g.s.groups + a.lead);
        if (s.u < s.b_first + n) break;
        s.b_first += n;
        if (++s.b >= a.w.B) {   // (lengths that changed under the call)
            s.u = s.u_end;
            return g;
        }
        for (;;) {
            const int b = s.b + lane;
            const unsigned some = __ballot_sync(0xffffffffu, b >= a.w.B - 1 || __ldg(a.w.off + b + 1) > __ldg(a.w.off + b));
            if (some) {
                s.b = min(s.b + __ffs(some) - 1, a.w.B - 1);
                break;
            }
            s.b += 32;
        }
    }
    const int size = g.s.groups + a.lead;
    int item, u0;
    for (;;) {
        const int64_t in = s.u - s.b_first;
        item = (int)divide(in, size);
        u0 = (int)(in - (int64_t)item * size);
        if (u0 > a.lead) break;
        s.u -= u0;                   // (the share's first segment, or an item's start)
        u0 = 0;
        if (s.u_end - s.u > a.lead) break;
        s.u = s.u_end;               // the next share starts here
        if (!rest()) return g;
    }
    int u1 = (int)min((int64_t)size, u0 + (s.u_end - s.u));
    g.b = s.b;
    g.h = item / g.s.tiles;
    g.rho0 = (item - g.h * g.s.tiles) * a.TM;
    const int all = g.s.n * a.G;
    g.rows = min(a.TM, all - g.rho0);
    g.head = u0 == 0;
    g.whole = g.head && u1 == size;
    // up to the CTA that holds the item's last unit
    g.parts = g.head ? (int)(divide(s.u + size - 1, s.size) - blockIdx.x) + 1 : 0;
    s.u += u1 - u0;
    u0 = max(0, u0 - a.lead);
    u1 -= a.lead;
    // groups that this tile's rows see none of are left out
    const int i0 = g.rho0 / a.G, i1 = (g.rho0 + g.rows - 1) / a.G;
    int end = g.s.end, lo_g = g.s.lo_g;
    if (a.mask != GDPA_CACHE_HISTORY) end = min(end, g.s.start + i1 + 1);
    if (a.mask == GDPA_CACHE_CAUSAL && a.window > 0 && (g.s.sink_g > 0 || a.sinks <= 0))
        lo_g = max(lo_g, max(0, g.s.start + i0 - a.window + 1) / kCacheGroup);
    const int end_g = (end + kCacheGroup - 1) / kCacheGroup;
    const int b0 = max(max(u0, g.s.sink_g) - g.s.sink_g + g.s.lo_g, lo_g);
    const int b1 = min(u1 - g.s.sink_g + g.s.lo_g, end_g);
    g.a0 = u0;
    g.na = max(0, min(u1, g.s.sink_g) - u0);
    g.n = g.na + max(0, b1 - b0);
    g.b0 = b0 - g.na;
    return g;
}

// What one row sees: events below `hi` that are at or above `lo` or below the
// sinks; in a tree, also its path (depth steps long) among the new rows.
struct RowView {
    int hi, lo, tok, depth;   // tok -1: not a row
};

__device__ __forceinline__ int tree_parent(const AttnArgs& a, const Sample& s, int i) {
    const int p = __ldg(a.parents + s.t0 + i);
    return p >= 0 && p < i ? p : -1;
}

__device__ __forceinline__ RowView row_view(const AttnArgs& a, const Segment& g, int r) {
    RowView v;
    v.tok = v.depth = -1;
    v.hi = v.lo = 0;
    if (r >= g.rows) return v;
    v.tok = (g.rho0 + r) / a.G;
    int pos = g.s.start;
    if (a.mask == GDPA_CACHE_CAUSAL) {
        pos += v.tok;
        v.hi = pos + 1;
    } else {
        v.hi = g.s.start;
        if (a.mask == GDPA_CACHE_TREE) {
            v.depth = 0;
            if (a.window > 0)   // (what positions are for)
                for (int i = tree_parent(a, g.s, v.tok); i >= 0; i = tree_parent(a, g.s, i)) ++v.depth;
            pos += v.depth;
        }
    }
    v.hi = min(v.hi, g.s.end);
    v.lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
    return v;
}

// Bit j: the row sees event e0 + j (j < 16).
__device__ __forceinline__ uint32_t row_bits(const AttnArgs& a, const Segment& g, const RowView& v, int e0) {
    if (v.tok < 0) return 0;
    const auto below = [&](int n) { return n <= e0 ? 0u : n >= e0 + 16 ? 0xffffu : (1u << (n - e0)) - 1u; };
    uint32_t bits = below(v.hi) & (~below(v.lo) | below(a.window > 0 ? a.sinks : 0));
    if (a.mask == GDPA_CACHE_TREE && e0 + 16 > g.s.start && e0 <= g.s.start + v.tok) {
        int depth = v.depth;
        for (int i = v.tok; i >= 0 && g.s.start + i >= e0; i = tree_parent(a, g.s, i), --depth) {
            const int e = g.s.start + i;
            if (e >= e0 + 16 || e >= g.s.end) continue;
            if (a.window <= 0 || v.depth - depth < a.window || g.s.start + depth < a.sinks) bits |= 1u << (e - e0);
        }
    }
    return bits;
}

// the power of two 2^(to - floor(log2 x)), x > 0 finite and normal; kept within f32
__device__ __forceinline__ float inverse_power(float x, int to = 0) {
    const uint32_t e = __float_as_uint(x) >> 23;
    return __uint_as_float((uint32_t)(min(max(254 + to - (int)e, 1), 254)) << 23);
}

// two values of a query row (below 256) as E4M3 codes, and what these leave of
// them as E5M2 ones
__device__ __forceinline__ void split_q(float x, float y, uint32_t& hi, uint32_t& lo) {
    uint16_t h, l;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(y), "f"(x));
    uint32_t f;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"(h));
    const float2 v = __half22float2(*reinterpret_cast<__half2*>(&f));
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(l) : "f"(y - v.y), "f"(x - v.x));
    hi = h;
    lo = l;
}

// sum += x with what the rounding leaves of it kept in `lost` (Kahan's compensated
// sum): thousands of equal weights on a larger sum would drift by 2^-24 of it each.
__device__ __forceinline__ void add_compensated(float& sum, float& lost, float x) {
    const float y = x - lost, t = sum + y;
    lost = (t - sum) - y;
    sum = t;
}

// values of 16 bytes of a cache row
__host__ __device__ constexpr int cache_per_chunk(int store) {
    return store == GDPA_STORE_F32 ? 4 : store == GDPA_STORE_BF16 ? 8 : 16;
}

// the values of a word of 16 bytes of a cache row
template <int STORE>
__device__ __forceinline__ void expand_word(uint32_t w, float (&x)[cache_per_chunk(STORE) / 4]) {
    if constexpr (STORE == GDPA_STORE_F32) {
        x[0] = __uint_as_float(w);
    } else if constexpr (STORE == GDPA_STORE_BF16) {
        x[0] = __uint_as_float(w << 16);
        x[1] = __uint_as_float(w & 0xffff0000u);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t h;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w >> (16 * i))));
            const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

// value by value of 16 bytes of a cache row (8-bit: as its code's value)
template <int STORE>
__device__ __forceinline__ void expand(const uint4& q, float (&x)[cache_per_chunk(STORE)]) {
    constexpr int V = cache_per_chunk(STORE) / 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) expand_word<STORE>((&q.x)[i], *reinterpret_cast<float(*)[V]>(x + V * i));
}

// Four values to the row type.
__device__ __forceinline__ void put4(float* p, const float (&x)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void put4(__nv_bfloat16* p, const float (&x)[4]) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]), hi = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// The sums over a segment of a tile, from the warps that took turns over its
// groups, to the outputs or to the workspace.  at(w, r, c): address of 4 columns
// of warp w's row r; ml(w, r): its maximum and sum.  Warps ks * RT + rt hold rows
// 16 rt .. of the tile.
template <typename E, bool SM, int NT, typename At, typename Ml>
__device__ __forceinline__ void finish_segment(const AttnArgs& a, const Segment& g, int ks, At at, Ml ml) {
    const int d = a.c.d, d4 = d / 4;
    float* slot = nullptr;
    if (!g.whole) {
        slot = a.part + (int64_t)(2 * blockIdx.x + (g.head ? 1 : 0)) * cache_slot(a.TM, d);
        if (g.head && threadIdx.x == 0) {
            CacheDesc& t = a.desc[blockIdx.x];
            t.rows = g.rows;
            t.t0 = g.s.t0;
            t.h = g.h;
            t.rho0 = g.rho0;
            t.parts = g.parts;
        }
    }
    for (int i = threadIdx.x; i < g.rows * d4; i += NT) {
        const int r = i / d4, c = (i - r * d4) * 4;
        const int w0 = r >> 4, rr = r & 15;
        float m = -INFINITY, l = 0.0f, x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (SM)
            for (int k = 0; k < ks; ++k) m = fmaxf(m, ml(w0 + k * a.RT, rr).x);
        for (int k = 0; k < ks; ++k) {
            const float4 y = *at(w0 + k * a.RT, rr, c);
            float f = 1.0f;
            if constexpr (SM) {
                const float2 s = ml(w0 + k * a.RT, rr);
                f = s.x == -INFINITY ? 0.0f : ex2_approx(s.x - m);
                // a part without events holds zeros; a NaN maximum never gets here (fmaxf)
                l += s.y * f;
                if (s.x == -INFINITY && s.y == 0.0f) continue;
            }
            x[0] += y.x * f;
            x[1] += y.y * f;
            x[2] += y.z * f;
            x[3] += y.w * f;
        }
        if (slot) {
            put4(slot + r * d + c, x);
            if (SM && c == 0) {
                slot[a.TM * d + r] = m;
                slot[a.TM * (d + 1) + r] = l;
            }
            continue;
        }
        const int rho = g.rho0 + r, tok = rho / a.G;
        const int64_t row = (int64_t)(g.s.t0 + tok) * a.H + g.h * a.G + (rho - tok * a.G);
        if constexpr (SM) {
            const float f = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] *= f;
            if (c == 0 && a.lse) a.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
        }
        put4((E*)a.o + row * d + c, x);
    }
}

// Let a kernel take `bytes` of shared memory; once a kernel and device.
inline bool cache_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

gdpa_status launch_cache_mma(const AttnArgs& a, int grid, cudaStream_t st);
gdpa_status launch_cache_tc_bf16(const AttnArgs& a, int grid, cudaStream_t st);
gdpa_status launch_cache_tc_e4m3(const AttnArgs& a, int grid, cudaStream_t st);
// CTAs an SM that the registers of R rows' queries and sums leave room for.
__host__ __device__ constexpr int cache_few_per_sm(int store, int R) {
    return R * cache_per_chunk(store) <= 16 ? 4 : R * cache_per_chunk(store) <= 32 ? 3 : 2;
}
gdpa_status launch_cache_few(const AttnArgs& a, gdpa_dtype dt, int grid, cudaStream_t st);
gdpa_status launch_cache_simt(const AttnArgs& a, gdpa_dtype dt, int grid, cudaStream_t st);

}  // namespace gdpa
