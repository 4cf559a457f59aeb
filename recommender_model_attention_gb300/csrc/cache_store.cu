// The history cache's rows: written to their pages, in 8 bits or as they are,
// and read back.
//
// 8-bit rows.  A row x of one head (d values) is held as E4M3 codes c_i and
// one power of two, x_i ~ c_i 2^e, with the least e >= -126 that brings the
// row's largest magnitude to 448 or less.  A power of two costs no precision
// that a freely chosen scale would keep (E4M3's steps are relative), and makes
// every product by it exact: a value is rounded once, x_i 2^-e to the nearest
// code, ties to the even one, at most 2^-4 of it (2^-10 2^e near zero).  At e = 120
// the code 256 stands for 2^128, which float32 does not hold: values from 248 2^120 on
// take 240, the largest whose value it does.  One
// scale a row and not one a block of columns, because then the attention that
// reads the cache may multiply whole scores and weights by it.  A row that
// holds an infinity or a NaN is all NaN.
//
// What bounds it: every value is read and written once, so device memory; for
// a handful of rows, the launch.  A thread owns 16 bytes of a bf16 or float32
// row, neighbouring lanes the rest of the row, so that its largest value is a
// few shuffles away and both sides are whole sectors; kPasses such pieces, whose
// loads are all on their way before anything is done with the first (one after the
// other: 156 us for the 430 MB of 256 histories written and read back).
#include <string.h>

#include <atomic>

#include "cache_internal.h"

namespace gdpa {
namespace {

constexpr int kThreads = 256;
// Pieces a thread takes (430 MB of 8-bit and bf16 rows: 88 us with 2, 82 with 4, 95
// with 8; 64 bytes each, of float32 rows to write in 8 bits: 123 us with 2, 130 with 4)
constexpr int kPasses = 4, kPassesLong = 2;
constexpr int kMaxTokens = 512;  // of a block: two rows of one piece each
constexpr int kCounted = 1023;   // samples whose offsets a block counts through (as rotary positions do)

constexpr int kTopExponent = 120;   // of the largest finite rows

struct StoreArgs {
    CacheView c;
    CacheWhere w;
    const void *k, *v;            // rows; written by reads
    int64_t kt, kh, vt, vh;       // strides in elements
    int items, lanes;             // 16-byte pieces of a cache row; rounded up to a power of two
    int sectors;                  // rows in whole sectors of 32 bytes
    int tokens, rows;             // of a block: tokens, and of the heads' K and V rows of each
    int step_tok, step_row;       // a pass further on: tokens, rows (a pass's rows in tokens and the rest)
};

// The last sample that starts at or before `row`, among [lo, hi).
__device__ __forceinline__ int sample_of(const int32_t* off, int64_t row, int lo, int hi) {
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(off + mid) <= row) lo = mid; else hi = mid;
    }
    return lo;
}

// Where the block's tokens lie: a thread a token.  (The samples that they can
// belong to by looking at all offsets at once.)
struct Tokens {
    int page[kMaxTokens], e[kMaxTokens];   // -1: no row of a sample, or outside the cache
};

__device__ __forceinline__ void find_tokens(const StoreArgs& a, int64_t row0, Tokens& t) {
    const CacheWhere& w = a.w;
    int lo = 0, hi = w.B;
    if (w.B <= kCounted) {
        int n0 = 0, n1 = 0;
        for (int i = threadIdx.x; i - (int)threadIdx.x <= w.B; i += kThreads) {
            const int64_t o = i <= w.B ? w.off[i] : INT64_MAX;
            n0 += __syncthreads_count(o <= row0);
            n1 += __syncthreads_count(o <= row0 + a.tokens - 1);
        }
        lo = max(n0 - 1, 0);
        hi = min(n1, w.B);
    }
    const int64_t last = min(w.T, (int64_t)__ldg(w.off + w.B));
    for (int i = threadIdx.x; i < a.tokens; i += kThreads) {
        const int64_t row = row0 + i;
        t.page[i] = t.e[i] = -1;
        if (row >= last) continue;
        const int b = sample_of(w.off, row, lo, hi);
        const int first = __ldg(w.off + b);
        if (row < first) continue;   // (before the first sample)
        const int64_t ev = row - first + (w.starts ? __ldg(w.starts + b) : 0);
        const int64_t page = cache_block(a.c, w, b, ev, 0);
        t.e[i] = 0;   // (a row, if not one with a page)
        if (page < 0) continue;
        t.page[i] = (int)(page / a.c.heads);
        t.e[i] = (int)(ev & ((1 << a.c.page_log) - 1));
    }
    __syncthreads();
}

// What a thread's pieces are of, one pass after the other.
struct Walk {
    int tok, hv;      // token of the block, row of the token's 2 heads
    const StoreArgs& a;
    const int hv0;
    __device__ __forceinline__ Walk(const StoreArgs& a, int first) : a(a), hv0(blockIdx.y * a.rows) {
        tok = first / a.rows;
        hv = first - tok * a.rows;
    }
    __device__ __forceinline__ void next() {
        tok += a.step_tok;
        hv += a.step_row;
        if (hv >= a.rows) {
            hv -= a.rows;
            ++tok;
        }
    }
    __device__ __forceinline__ bool is_v() const { return hv0 + hv >= a.c.heads; }
    __device__ __forceinline__ int head() const { return hv0 + hv - (is_v() ? a.c.heads : 0); }
    __device__ __forceinline__ bool inside() const { return tok < a.tokens && hv0 + hv < 2 * a.c.heads; }
};

__device__ __forceinline__ uint16_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float2 from_e4m3x2(uint16_t v) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
    return __half22float2(*reinterpret_cast<__half2*>(&h));
}

__device__ __forceinline__ void put(float& y, float v) { y = v; }
__device__ __forceinline__ void put(__nv_bfloat16& y, float v) { y = __float2bfloat16_rn(v); }

// N values at p, in 16-byte loads.
template <typename E, int N>
__device__ __forceinline__ void load_piece(const E* p, E (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N * (int)sizeof(E) / 16; ++i) reinterpret_cast<uint4*>(x)[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
}
// N values to p: whole sectors in one store where they are aligned to them.
template <typename E, int N>
__device__ __forceinline__ void store_piece(E* p, const E (&x)[N], bool sectors) {
    const uint32_t* v = reinterpret_cast<const uint32_t*>(x);
    if constexpr (N * sizeof(E) >= 32) {
        if (sectors) {
#pragma unroll
            for (int i = 0; i < N * (int)sizeof(E) / 32; ++i)
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"((char*)p + 32 * i), "r"(v[8 * i]),
                             "r"(v[8 * i + 1]), "r"(v[8 * i + 2]), "r"(v[8 * i + 3]), "r"(v[8 * i + 4]), "r"(v[8 * i + 5]),
                             "r"(v[8 * i + 6]), "r"(v[8 * i + 7])
                             : "memory");
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < N * (int)sizeof(E) / 16; ++i) reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(x)[i];
}

// E: the rows' type; FP8: 8-bit cache; WIDE: rows in 16-byte loads.
template <typename E, bool FP8, bool WIDE>
__global__ void __launch_bounds__(kThreads)
cache_write_kernel(const __grid_constant__ StoreArgs a) {
    constexpr int N = FP8 ? 16 : 16 / (int)sizeof(E);    // values of a piece
    __shared__ Tokens at;
    const int64_t row0 = (int64_t)blockIdx.x * a.tokens;
    const int sub = threadIdx.x / a.lanes, c = threadIdx.x - sub * a.lanes;
    constexpr int kN = FP8 && sizeof(E) == 4 ? kPassesLong : kPasses;
    alignas(16) E xs[kN][N];
    const Walk start(a, sub);
    Walk w = start;
#pragma unroll
    for (int k = 0; k < kN; ++k, w.next()) {
        const int64_t row = row0 + w.tok;
#pragma unroll
        for (int j = 0; j < N * (int)sizeof(E) / 16; ++j) reinterpret_cast<uint4*>(xs[k])[j] = make_uint4(0, 0, 0, 0);
        if (w.inside() && row < a.w.T && c < a.items) {
            const E* src = w.is_v() ? (const E*)a.v + row * a.vt + w.head() * a.vh : (const E*)a.k + row * a.kt + w.head() * a.kh;
            if constexpr (WIDE) {
                load_piece<E, N>(src + c * N, xs[k]);
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) xs[k][j] = src[c * N + j];
            }
        }
    }
    find_tokens(a, row0, at);
    Walk v = start;
#pragma unroll
    for (int k = 0; k < kN; ++k, v.next()) {        // whole warps stay together
        const bool live = v.inside() && c < a.items && at.page[v.tok] >= 0;
        const bool is_v = v.is_v();
        const E (&x)[N] = xs[k];
        const int64_t blk = live ? (int64_t)at.page[v.tok] * a.c.heads + v.head() : 0;
        const int e = live ? at.e[v.tok] : 0;
        uint8_t* dst = (is_v ? a.c.v : a.c.k) + blk * a.c.block;
        if constexpr (FP8) {
            // the row's largest magnitude as float32 bits: those of an infinity or
            // a NaN are above every number's
            uint32_t top = 0;
            if constexpr (sizeof(E) == 2) {
                const uint32_t* p = reinterpret_cast<const uint32_t*>(x);
#pragma unroll
                for (int j = 0; j < N / 2; ++j) top = __vmaxu2(top, p[j] & 0x7fff7fffu);
                for (int m = 1; m < a.lanes; m <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, m));
                top = max(top & 0xffff0000u, top << 16);
            } else {
                const uint32_t* p = reinterpret_cast<const uint32_t*>(x);
#pragma unroll
                for (int j = 0; j < N; ++j) top = max(top, p[j] & 0x7fffffffu);
                for (int m = 1; m < a.lanes; m <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
            }
            const bool odd = top >= 0x7f800000u;
            // top = m 2^x with m in [1, 2): 448 = 1.75 2^8
            const int ex = max((int)(top >> 23) - 127 - ((top & 0x7fffffu) <= 0x600000u ? 8 : 7), -126);
            const float inv = odd ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(127 - ex) << 23);
            alignas(16) uint16_t p[N / 2];
#pragma unroll
            for (int j = 0; j < N / 2; ++j) p[j] = to_e4m3x2(to_f(x[2 * j]) * inv, to_f(x[2 * j + 1]) * inv);
            if (ex == kTopExponent) {   // (above it there are no finite rows)
                uint32_t* w = reinterpret_cast<uint32_t*>(p);
#pragma unroll
                for (int j = 0; j < N / 4; ++j) w[j] -= __vcmpeq4(w[j] & 0x7f7f7f7fu, 0x78787878u) & 0x01010101u;
            }
            if (live) {
                *reinterpret_cast<uint4*>(dst + cache_chunk(a.c.row, a.c.page_log, e, c)) = *reinterpret_cast<const uint4*>(p);
                if (c == 0) (is_v ? a.c.vs : a.c.ks)[(blk << a.c.page_log) + e] = (uint8_t)(odd ? 255 : ex + 127);
            }
        } else {
            if (live) *reinterpret_cast<uint4*>(dst + cache_chunk(a.c.row, a.c.page_log, e, c)) = *reinterpret_cast<const uint4*>(x);
        }
    }
}

// The other way: piece c of a row to its place among the rows.
template <typename E, bool FP8>
__global__ void __launch_bounds__(kThreads)
cache_read_kernel(const __grid_constant__ StoreArgs a) {
    constexpr int N = FP8 ? 16 : 16 / (int)sizeof(E);
    __shared__ Tokens at;
    const int64_t row0 = (int64_t)blockIdx.x * a.tokens;
    find_tokens(a, row0, at);
    const int sub = threadIdx.x / a.items, c = threadIdx.x - sub * a.items;
    if (sub >= kThreads / a.items) return;               // (threads that a pass leaves over)
    uint4 qs[kPasses];
    uint32_t sc[kPasses];
    const Walk start(a, sub);
    Walk w = start;
#pragma unroll
    for (int k = 0; k < kPasses; ++k, w.next()) {
        qs[k] = make_uint4(0, 0, 0, 0);                  // rows without a page read as zeros
        sc[k] = 127;
        if (w.inside() && at.page[w.tok] >= 0) {
            const int64_t blk = (int64_t)at.page[w.tok] * a.c.heads + w.head();
            const int e = at.e[w.tok];
            qs[k] = *reinterpret_cast<const uint4*>((w.is_v() ? a.c.v : a.c.k) + blk * a.c.block + cache_chunk(a.c.row, a.c.page_log, e, c));
            if constexpr (FP8) sc[k] = (w.is_v() ? a.c.vs : a.c.ks)[(blk << a.c.page_log) + e];
        }
    }
    Walk v = start;
#pragma unroll
    for (int k = 0; k < kPasses; ++k, v.next()) {
        if (!v.inside() || at.e[v.tok] < 0) continue;
        const int64_t row = row0 + v.tok;
        alignas(16) E x[N];
        if constexpr (FP8) {
            const float s = cache_scale(sc[k]);
            alignas(16) uint16_t p[8];
            *reinterpret_cast<uint4*>(p) = qs[k];
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                const float2 f = from_e4m3x2(p[j]);
                put(x[2 * j], f.x * s);
                put(x[2 * j + 1], f.y * s);
            }
        } else {
            *reinterpret_cast<uint4*>(x) = qs[k];
        }
        E* dst = v.is_v() ? (E*)a.v + row * a.vt + v.head() * a.vh : (E*)a.k + row * a.kt + v.head() * a.kh;
        store_piece<E, N>(dst + c * N, x, a.sectors);
    }
}

// A block's part: as many of a token's rows as its passes hold (`width` threads a
// row), and then as many tokens, fewer while that leaves SMs idle.
gdpa_status launch(void (*f)(const StoreArgs), StoreArgs& a, int width, int passes, cudaStream_t st) {
    const int heads2 = 2 * a.c.heads, room = passes * (kThreads / width);
    a.rows = heads2 < room ? heads2 : room;
    a.tokens = room / a.rows;
    const int sms = cache_sms();
    if (sms == 0) return GDPA_ERR_CUDA;
    while (a.tokens > 1 && (a.w.T + a.tokens - 1) / a.tokens < 4 * sms) a.tokens = (a.tokens + 1) / 2;
    a.step_tok = kThreads / width / a.rows;
    a.step_row = kThreads / width - a.step_tok * a.rows;
    const int64_t blocks = (a.w.T + a.tokens - 1) / a.tokens;
    if (blocks > 0x7fffffff) return GDPA_ERR_UNSUPPORTED;
    f<<<dim3((unsigned)blocks, (unsigned)((heads2 + a.rows - 1) / a.rows)), kThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? GDPA_OK : GDPA_ERR_CUDA;
}

// What both directions check; `wide`: all rows in 16-byte pieces.
gdpa_status store_args(const gdpa_cache* cache, gdpa_dtype dtype, int64_t T, const gdpa_cache_rows* k,
                       const gdpa_cache_rows* v, const gdpa_cache_where* w, StoreArgs& a, bool& wide) {
    gdpa_status s;
    if (!cache_view(cache, a.c, &s)) return s;
    if (dtype != GDPA_BF16 && dtype != GDPA_F32) return GDPA_ERR_INVALID_ARG;
    if ((a.c.store == GDPA_STORE_BF16 && dtype != GDPA_BF16) || (a.c.store == GDPA_STORE_F32 && dtype != GDPA_F32))
        return GDPA_ERR_INVALID_ARG;
    if (T < 0 || !k || !v) return GDPA_ERR_INVALID_ARG;
    s = cache_where(w, T, a.c, a.w);
    if (s != GDPA_OK) return s;
    const size_t es = dtype == GDPA_BF16 ? 2 : 4;
    const gdpa_cache_rows* r[2] = {k, v};
    wide = true;
    a.sectors = 1;
    for (int i = 0; i < 2; ++i) {
        if (T > 0 && (!r[i]->x || (uintptr_t)r[i]->x % es)) return GDPA_ERR_INVALID_ARG;
        // strides that are never stepped: a single row's, a single head's
        const int64_t t = T > 1 ? r[i]->token : 0, h = a.c.heads > 1 ? r[i]->head : 0;
        if ((uintptr_t)r[i]->x % 16 || t * es % 16 || h * es % 16) wide = false;
        if ((uintptr_t)r[i]->x % 32 || t * es % 32 || h * es % 32) a.sectors = 0;
        (i ? a.v : a.k) = r[i]->x;
        (i ? a.vt : a.kt) = t;
        (i ? a.vh : a.kh) = h;
    }
    a.items = a.c.row / 16;
    for (a.lanes = 1; a.lanes < a.items; a.lanes *= 2) {}
    return GDPA_OK;
}

}  // namespace

bool cache_view(const gdpa_cache* c, CacheView& v, gdpa_status* s) {
    *s = GDPA_ERR_INVALID_ARG;
    if (!c || c->pages < 0 || c->heads < 1 || c->d < 1 || c->page < 1) return false;
    if (c->store < GDPA_STORE_BF16 || c->store > GDPA_STORE_E4M3) return false;
    const bool fp8 = c->store == GDPA_STORE_E4M3;
    if (c->pages > 0 && (!c->k || !c->v || (fp8 && (!c->k_scale || !c->v_scale)))) return false;
    if (!c->error || (uintptr_t)c->error % 4) return false;
    if (((uintptr_t)c->k | (uintptr_t)c->v | (uintptr_t)c->k_scale | (uintptr_t)c->v_scale) % 128) return false;
    *s = GDPA_ERR_UNSUPPORTED;
    const int es = c->store == GDPA_STORE_BF16 ? 2 : c->store == GDPA_STORE_F32 ? 4 : 1;
    if (c->d > 128 || c->d * es % 16 || c->heads > 4096) return false;
    if (c->page < kCacheGroup || c->page > 1024 || (c->page & (c->page - 1))) return false;
    v.k = (uint8_t*)c->k;
    v.v = (uint8_t*)c->v;
    v.ks = c->k_scale;
    v.vs = c->v_scale;
    v.err = c->error;
    v.pages = c->pages;
    v.heads = c->heads;
    v.d = c->d;
    v.store = c->store;
    v.row = c->d * es;
    for (v.page_log = 4; (1 << v.page_log) < c->page; ++v.page_log) {}
    v.block = (int64_t)v.row << v.page_log;
    *s = GDPA_OK;
    return true;
}

int cache_sms() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
    if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

gdpa_status cache_where(const gdpa_cache_where* w, int64_t T, const CacheView& c, CacheWhere& o) {
    if (!w || w->B < 0 || w->width < 0 || w->stride < 0 || !w->off || (uintptr_t)w->off % 4) return GDPA_ERR_INVALID_ARG;
    if (w->B > 0 && w->width > 0 && (!w->table || (uintptr_t)w->table % 4)) return GDPA_ERR_INVALID_ARG;
    if ((uintptr_t)w->starts % 4) return GDPA_ERR_INVALID_ARG;
    if (((int64_t)w->width << c.page_log) > kCacheMost || T > kCacheMost) return GDPA_ERR_UNSUPPORTED;
    o.table = w->table;
    o.stride = w->B > 1 ? w->stride : 0;
    o.width = w->width;
    o.off = w->off;
    o.starts = w->starts;
    o.B = w->B;
    o.T = T;
    return GDPA_OK;
}

}  // namespace gdpa

extern "C" {

gdpa_status gdpa_cache_bytes(const gdpa_cache* cache, int64_t* rows, int64_t* scales) {
    if (!cache || !rows || !scales) return GDPA_ERR_INVALID_ARG;
    // only the sizes are looked at
    gdpa_cache c = *cache;
    c.k = c.v = c.k_scale = c.v_scale = (uint8_t*)128;
    c.error = (int32_t*)128;
    gdpa::CacheView v;
    gdpa_status s;
    if (!gdpa::cache_view(&c, v, &s)) return s;
    *rows = v.block * v.heads * v.pages;
    *scales = v.store == GDPA_STORE_E4M3 ? ((int64_t)v.pages * v.heads << v.page_log) : 0;
    return GDPA_OK;
}

gdpa_status gdpa_cache_write(const gdpa_cache* cache, gdpa_dtype dtype, int64_t T, const gdpa_cache_rows* k,
                             const gdpa_cache_rows* v, const gdpa_cache_where* where, void* stream) {
    using namespace gdpa;
    StoreArgs a;
    memset(&a, 0, sizeof(a));
    bool wide;
    const gdpa_status s = store_args(cache, dtype, T, k, v, where, a, wide);
    if (s != GDPA_OK || T == 0 || a.w.B == 0) return s;
    const bool fp8 = a.c.store == GDPA_STORE_E4M3;
    void (*f)(const StoreArgs);
    if (dtype == GDPA_BF16) {
        using E = __nv_bfloat16;
        f = fp8 ? wide ? cache_write_kernel<E, true, true> : cache_write_kernel<E, true, false>
                : wide ? cache_write_kernel<E, false, true> : cache_write_kernel<E, false, false>;
    } else {
        using E = float;
        f = fp8 ? wide ? cache_write_kernel<E, true, true> : cache_write_kernel<E, true, false>
                : wide ? cache_write_kernel<E, false, true> : cache_write_kernel<E, false, false>;
    }
    return launch(f, a, a.lanes, fp8 && dtype == GDPA_F32 ? kPassesLong : kPasses, (cudaStream_t)stream);
}

gdpa_status gdpa_cache_read(const gdpa_cache* cache, gdpa_dtype dtype, int64_t T, const gdpa_cache_rows* k,
                            const gdpa_cache_rows* v, const gdpa_cache_where* where, void* stream) {
    using namespace gdpa;
    StoreArgs a;
    memset(&a, 0, sizeof(a));
    bool wide;
    const gdpa_status s = store_args(cache, dtype, T, k, v, where, a, wide);
    if (s != GDPA_OK || T == 0 || a.w.B == 0) return s;
    if (!wide) return GDPA_ERR_INVALID_ARG;
    const bool fp8 = a.c.store == GDPA_STORE_E4M3;
    void (*f)(const StoreArgs);
    if (dtype == GDPA_BF16)
        f = fp8 ? cache_read_kernel<__nv_bfloat16, true> : cache_read_kernel<__nv_bfloat16, false>;
    else
        f = fp8 ? cache_read_kernel<float, true> : cache_read_kernel<float, false>;
    return launch(f, a, a.items, kPasses, (cudaStream_t)stream);
}

gdpa_status gdpa_cache_check(const gdpa_cache* cache, int32_t* detail, void* stream) {
    gdpa::CacheView v;
    gdpa_status s;
    if (!gdpa::cache_view(cache, v, &s)) return s;
    if (!detail) return GDPA_ERR_INVALID_ARG;
    int32_t e[4];
    cudaStream_t st = (cudaStream_t)stream;
    if (cudaMemcpyAsync(e, v.err, sizeof(e), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return GDPA_ERR_CUDA;
    memcpy(detail, e, sizeof(e));
    if (e[0] == 0) return GDPA_OK;
    if (cudaMemsetAsync(v.err, 0, sizeof(e), st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess)
        return GDPA_ERR_CUDA;
    return e[0] == gdpa::kDevTimeout ? GDPA_ERR_TIMEOUT : GDPA_ERR_DEVICE;
}

}  // extern "C"
