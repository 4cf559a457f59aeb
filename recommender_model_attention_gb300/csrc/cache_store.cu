// The history cache's rows: written to their pages, in 8 bits or as they are,
// and read back.
//
// 8-bit rows.  A row x of one head (d values) is held as E4M3 codes c_i and
// one power of two, x_i ~ c_i 2^e, with the least e >= -126 that brings the
// row's largest magnitude to 448 or less.  A power of two costs no precision
// that a freely chosen scale would keep (E4M3's steps are relative), and makes
// every product by it exact: a value is rounded once, x_i 2^-e to the nearest
// code, ties to the even one, at most 2^-4 of it (2^-10 2^e near zero).  One
// scale a row and not one a block of columns, because then the attention that
// reads the cache may multiply whole scores and weights by it.  A row that
// holds an infinity or a NaN is all NaN.
//
// What bounds it: every value is read and written once, so device memory; for
// a handful of rows, the launch.  A thread owns 16 bytes of a bf16 or float32
// row, neighbouring lanes the rest of the row, so that its largest value is a
// few shuffles away and both sides are whole sectors.
#include <string.h>

#include "cache_internal.h"

namespace gdpa {
namespace {

constexpr int kThreads = 256;
constexpr int kCounted = 1023;   // samples whose offsets a block counts through (as rotary positions do)

struct StoreArgs {
    CacheView c;
    CacheWhere w;
    const void *k, *v;            // rows; written by reads
    int64_t kt, kh, vt, vh;       // strides in elements
    int items, lanes;             // 16-byte pieces of a row; rounded up to a power of two
    int tokens;                   // of a block
};

// The last sample that starts at or before `row`, among [lo, hi).
__device__ __forceinline__ int sample_of(const int32_t* off, int64_t row, int lo, int hi) {
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(off + mid) <= row) lo = mid; else hi = mid;
    }
    return lo;
}

// The samples that the block's rows [row0, row0 + n) can belong to.
__device__ __forceinline__ void block_samples(const CacheWhere& w, int64_t row0, int n, int& lo, int& hi) {
    lo = 0;
    hi = w.B;
    if (w.B > kCounted) return;
    int n0 = 0, n1 = 0;
    for (int i = threadIdx.x; i - (int)threadIdx.x <= w.B; i += kThreads) {
        const int64_t o = i <= w.B ? w.off[i] : INT64_MAX;
        n0 += __syncthreads_count(o <= row0);
        n1 += __syncthreads_count(o <= row0 + n - 1);
    }
    lo = max(n0 - 1, 0);
    hi = min(n1, w.B);
}

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

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float& y, float v) { y = v; }
__device__ __forceinline__ void put(__nv_bfloat16& y, float v) { y = __float2bfloat16_rn(v); }

// Where the N values of piece c of a row's N-value pieces lie within a block.
template <bool FP8, int N>
__device__ __forceinline__ int piece_at(const CacheView& v, int e, int c) {
    if constexpr (!FP8) return cache_chunk(v.row, v.page_log, e, c);
    constexpr int P = 16 / N;   // pieces of a chunk
    return cache_chunk(v.row, v.page_log, e, c / P) + (c % P) * N;
}
template <int N> struct Codes;
template <> struct Codes<8> { using T = uint2; };
template <> struct Codes<4> { using T = uint32_t; };

// E: the rows' type; FP8: 8-bit cache; WIDE: rows in 16-byte loads.
template <typename E, bool FP8, bool WIDE>
__global__ void __launch_bounds__(kThreads)
cache_write_kernel(const __grid_constant__ StoreArgs a) {
    constexpr int N = 16 / (int)sizeof(E);               // values of a piece
    const int64_t row0 = (int64_t)blockIdx.x * a.tokens;
    int lo, hi;
    block_samples(a.w, row0, a.tokens, lo, hi);
    const int sub = threadIdx.x / a.lanes, c = threadIdx.x % a.lanes;
    const int per = kThreads / a.lanes;                  // rows a pass
    const int heads2 = 2 * a.c.heads;
    const int64_t last = min(a.w.T, (int64_t)__ldg(a.w.off + a.w.B));
    const int n = a.tokens * heads2;
    for (int i0 = 0; i0 < n; i0 += per) {                // whole warps stay together
        const int i = i0 + sub;
        const int tok = i / heads2, hv = i - tok * heads2;
        const bool is_v = hv >= a.c.heads;
        const int h = is_v ? hv - a.c.heads : hv;
        const int64_t row = row0 + tok;
        bool live = i < n && row < last && c < a.items;
        alignas(16) E x[N] = {};
        int64_t blk = -1;
        int e = 0;
        if (live) {
            const E* src = is_v ? (const E*)a.v + row * a.vt + h * a.vh : (const E*)a.k + row * a.kt + h * a.kh;
            if constexpr (WIDE) {
                *reinterpret_cast<uint4*>(x) = __ldg(reinterpret_cast<const uint4*>(src) + c);
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) x[j] = src[c * N + j];
            }
            const int b = sample_of(a.w.off, row, lo, hi);
            const int64_t ev = row - __ldg(a.w.off + b) + (a.w.starts ? __ldg(a.w.starts + b) : 0);
            blk = cache_block(a.c, a.w, b, ev, h);
            e = (int)(ev & ((1 << a.c.page_log) - 1));
        }
        uint8_t* dst = (is_v ? a.c.v : a.c.k) + blk * a.c.block;
        if constexpr (FP8) {
            float top = 0.0f;
            bool odd = false;                            // an infinity or a NaN
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float f = fabsf(to_f(x[j]));
                odd |= !(f <= 3.402823466e38f);
                top = fmaxf(top, f);
            }
            for (int m = 1; m < a.lanes; m <<= 1) {
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
                odd |= __shfl_xor_sync(0xffffffffu, (int)odd, m) != 0;
            }
            // top = m 2^x with m in [1, 2): 448 = 1.75 2^8
            const uint32_t bits = __float_as_uint(top);
            const int ex = max((int)(bits >> 23) - 127 - ((bits & 0x7fffffu) <= 0x600000u ? 8 : 7), -126);
            const float inv = odd ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(127 - ex) << 23);
            alignas(8) uint16_t p[N / 2];
#pragma unroll
            for (int j = 0; j < N / 2; ++j) p[j] = to_e4m3x2(to_f(x[2 * j]) * inv, to_f(x[2 * j + 1]) * inv);
            if (live && blk >= 0) {
                using T = typename Codes<N>::T;
                *reinterpret_cast<T*>(dst + piece_at<true, N>(a.c, e, c)) = *reinterpret_cast<const T*>(p);
                if (c == 0) (is_v ? a.c.vs : a.c.ks)[(blk << a.c.page_log) + e] = (uint8_t)(odd ? 255 : ex + 127);
            }
        } else {
            if (live && blk >= 0)
                *reinterpret_cast<uint4*>(dst + piece_at<false, N>(a.c, e, c)) = *reinterpret_cast<const uint4*>(x);
        }
    }
}

// The other way: piece c of a row to its place among the rows.
template <typename E, bool FP8>
__global__ void __launch_bounds__(kThreads)
cache_read_kernel(const __grid_constant__ StoreArgs a) {
    constexpr int N = 16 / (int)sizeof(E);
    const int64_t row0 = (int64_t)blockIdx.x * a.tokens;
    int lo, hi;
    block_samples(a.w, row0, a.tokens, lo, hi);
    const int heads2 = 2 * a.c.heads;
    const int64_t last = min(a.w.T, (int64_t)__ldg(a.w.off + a.w.B));
    const int n = a.tokens * heads2 * a.items;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int r = i / a.items, c = i - r * a.items;
        const int tok = r / heads2, hv = r - tok * heads2;
        const bool is_v = hv >= a.c.heads;
        const int h = is_v ? hv - a.c.heads : hv;
        const int64_t row = row0 + tok;
        if (row >= last) break;                          // (rows ascend with i)
        const int b = sample_of(a.w.off, row, lo, hi);
        const int64_t ev = row - __ldg(a.w.off + b) + (a.w.starts ? __ldg(a.w.starts + b) : 0);
        const int64_t blk = cache_block(a.c, a.w, b, ev, h);
        alignas(16) E x[N] = {};                         // rows without a page read as zeros
        if (blk >= 0) {
            const int e = (int)(ev & ((1 << a.c.page_log) - 1));
            const uint8_t* src = (is_v ? a.c.v : a.c.k) + blk * a.c.block;
            const uint8_t* q = src + piece_at<FP8, N>(a.c, e, c);
            if constexpr (FP8) {
                using T = typename Codes<N>::T;
                const float s = cache_scale((is_v ? a.c.vs : a.c.ks)[(blk << a.c.page_log) + e]);
                alignas(8) uint16_t p[N / 2];
                *reinterpret_cast<T*>(p) = *reinterpret_cast<const T*>(q);
#pragma unroll
                for (int j = 0; j < N / 2; ++j) {
                    const float2 f = from_e4m3x2(p[j]);
                    put(x[2 * j], f.x * s);
                    put(x[2 * j + 1], f.y * s);
                }
            } else {
                *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(q);
            }
        }
        E* dst = is_v ? (E*)a.v + row * a.vt + h * a.vh : (E*)a.k + row * a.kt + h * a.kh;
        reinterpret_cast<uint4*>(dst)[c] = *reinterpret_cast<const uint4*>(x);
    }
}

// Tokens a block: about 4 passes of its threads, fewer while that leaves SMs idle.
int block_tokens(int64_t T, int items) {
    int64_t tok = 4 * kThreads / items;
    while (tok > 1 && (T + tok - 1) / tok < 4 * 152) tok = (tok + 1) / 2;
    return (int)(tok < 1 ? 1 : tok);
}

gdpa_status launch(void (*f)(const StoreArgs), StoreArgs& a, int items, cudaStream_t st) {
    a.tokens = block_tokens(a.w.T, items);
    const int64_t blocks = (a.w.T + a.tokens - 1) / a.tokens;
    if (blocks > 0x7fffffff) return GDPA_ERR_UNSUPPORTED;
    f<<<(unsigned)blocks, kThreads, 0, st>>>(a);
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
    for (int i = 0; i < 2; ++i) {
        if (T > 0 && (!r[i]->x || (uintptr_t)r[i]->x % es)) return GDPA_ERR_INVALID_ARG;
        // strides that are never stepped: a single row's, a single head's
        const int64_t t = T > 1 ? r[i]->token : 0, h = a.c.heads > 1 ? r[i]->head : 0;
        if ((uintptr_t)r[i]->x % 16 || t * es % 16 || h * es % 16) wide = false;
        (i ? a.v : a.k) = r[i]->x;
        (i ? a.vt : a.kt) = t;
        (i ? a.vh : a.kh) = h;
    }
    a.items = a.c.d * (int)es / 16;
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

gdpa_status cache_where(const gdpa_cache_where* w, int64_t T, const CacheView& c, CacheWhere& o) {
    if (!w || w->B < 0 || w->width < 0 || !w->off || (uintptr_t)w->off % 4) return GDPA_ERR_INVALID_ARG;
    if (w->B > 0 && w->width > 0 && (!w->table || (uintptr_t)w->table % 4)) return GDPA_ERR_INVALID_ARG;
    if ((uintptr_t)w->starts % 4) return GDPA_ERR_INVALID_ARG;
    if (((int64_t)w->width << c.page_log) > 0x7fffffff - 65536 || T > 0x7fffffff) return GDPA_ERR_UNSUPPORTED;
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
    return launch(f, a, 2 * a.c.heads * a.lanes, (cudaStream_t)stream);
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
    return launch(f, a, 2 * a.c.heads * a.items, (cudaStream_t)stream);
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
    return GDPA_ERR_DEVICE;
}

}  // extern "C"
