// The paged history cache: where a row lies, and what the store kernels and
// the attention over it share.
//
// A page holds `page` consecutive events of one user for every key head; K and
// V each have an array [pages][heads] of blocks of page * row bytes, and 8-bit
// caches one scale byte a row in [pages][heads][page].  Rows are laid out for
// the kernels that read 16 of them as operands of a matrix product: a block is
// split into columns of 128 bytes, [column][event][128 bytes], and the 16-byte
// chunk c of event e lies at c ^ (e & 7), so that 8 lanes that read the same
// chunk of 8 events, or 8 chunks of every second one, meet no bank twice.  It
// is also the 128-byte swizzle of tcgen05 operands, which a plain copy of
// whole events therefore brings into shared memory ready to use.  Rows of 64
// bytes lie row after row, chunk c of event e at c ^ ((e >> 1) & 3), the 64-byte
// swizzle; all other widths plainly.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdpa_internal.h"

namespace gdpa {

constexpr int kCacheMost = 0x3fffffff;   // events of a sample, rows of a call
constexpr int kCacheGroup = 16;   // events read together; a page is a multiple of it

struct CacheView {
    uint8_t *k, *v, *ks, *vs;
    int32_t* err;
    int64_t block;      // bytes of a (page, head) block: page << row bytes
    int pages, heads, d, store;
    int page_log;       // page = 1 << page_log
    int row;            // bytes of a row
};

// Where the new rows of a jagged batch lie: sample b's are rows [off[b],
// off[b + 1]), at the events starts[b], starts[b] + 1, ...  of the pages in
// row b of the table.
struct CacheWhere {
    const int32_t *table, *off, *starts;
    int64_t stride;     // of the table's rows
    int width, B;
    int64_t T;
};

// bytes of chunk c (16 bytes) of event e within its block
__host__ __device__ __forceinline__ int cache_chunk(int row, int page_log, int e, int c) {
    if ((row & 127) == 0)
        return ((((c >> 3) << page_log) + e) << 7) + (((c & 7) ^ (e & 7)) << 4);
    if (row == 64) return (e << 6) + ((c ^ ((e >> 1) & 3)) << 4);
    return e * row + (c << 4);
}

// Records a table entry or an event outside the cache (the access is skipped).
__device__ __forceinline__ void cache_bad(int32_t* err, int where, int sample, int value) {
    if (atomicCAS(err, 0, (int)kDevBad) == 0) {
        err[1] = where;
        err[2] = sample;
        err[3] = value;
    }
}
enum : int { kCacheBadPage = 1, kCacheBadEvent = 2, kCacheBadStart = 3 };

// The block of `head` in the page of event e of sample b, -1 if there is none.
__device__ __forceinline__ int64_t cache_block(const CacheView& c, const CacheWhere& w, int b, int64_t e,
                                               int head) {
    const int64_t i = e >> c.page_log;
    if (e < 0 || i >= w.width) {
        cache_bad(c.err, kCacheBadEvent, b, (int)e);
        return -1;
    }
    const int p = __ldg(w.table + b * w.stride + i);
    if ((unsigned)p >= (unsigned)c.pages) {
        cache_bad(c.err, kCacheBadPage, b, p);
        return -1;
    }
    return (int64_t)p * c.heads + head;
}

// 2^(byte - 127) of a scale byte (1 .. 247; 255, of a row of NaNs, gives infinity)
__device__ __forceinline__ float cache_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

bool cache_view(const gdpa_cache* c, CacheView& v, gdpa_status* s);
gdpa_status cache_where(const gdpa_cache_where* w, int64_t T, const CacheView& c, CacheWhere& o);
int cache_sms();   // SMs of the current device (looked up once a device), 0 if there is none

}  // namespace gdpa
