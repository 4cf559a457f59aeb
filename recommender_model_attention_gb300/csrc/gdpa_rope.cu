// Rotary positions of Q and K rows: the C entry points and the kernel.
//
// Each pair (a, b) of a row's rotated columns is turned by the angle
// t = position * f_i of its frequency:
//     a' = A (a cos t - b sin t),   b' = A (a sin t + b cos t),
// and the gradient is the same turn by -t.
//
// Angles.  A position of 10^9 times a frequency near 1 leaves float32 no
// digit of the angle.  Frequencies are therefore kept as turns per position
// in 64-bit fixed point (the fraction of a turn, 2^64 = one turn), so that
// the integer product with the position, which wraps, is the angle reduced
// to one turn without error: |frequency error| <= 2^-64 turns, 2^-33 turns
// at a position of 2^31.  The top 32 bits, as a signed fraction of half a
// turn, go to sincospif (float32 rows: error of a few 2^-24) or, for bf16
// rows, to the hardware sine and cosine on [-pi, pi] (absolute error about
// 2^-21, against the row's own rounding of 2^-8).
//
// What bounds it: every value is read and written once, so device memory;
// for a handful of rows, the launch.  A thread owns one 16-byte column item
// of a token (two of them, half a head apart, in the half layout), makes the
// item's sines and cosines once, and walks `hp` heads of Q and K with them;
// a warp's accesses are runs of whole 128-byte lines.  2.7 GB of float32 rows:
// 392 us, 6.9 TB/s; 286 MB of packed bf16 rows: 64 us a call, 58 in the kernel
// (4.9 TB/s).  There the blocks are resident for three rounds of loads in all;
// fewer heads a thread (more blocks: 68 us at 4, 73 at 2), two or four heads'
// loads ahead of their stores (64 to 81 us: registers cost resident blocks)
// and the first loads ahead of the angles (63) were no faster.
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include "gdpa_internal.h"
#include "tc_common.cuh"

namespace gdpa {
namespace {

constexpr int kThreads = 256;
// Samples whose offsets a block counts through; with more, each thread searches
// them.  (One head of Q and K, d = 128, bf16, counting and searching: 16 samples
// 9.0 and 10.2 us, 256 30.7 and 31.6, 1024 84.4 and 86.0, 2047 100.5 and 94.6,
// 8192 148 and 88; positions given 8.2, 28.7, 74, 80, 67.)
constexpr int kCounted = 1023;

struct RopeArgs {
    uint64_t turns[GDPA_ROPE_MAX_PAIRS];
    gdpa_rope_tensor t[2];
    const void* pos;      // int32 or int64 [T], or NULL: positions from `off`
    const int32_t* off;   // [B + 1] sample offsets
    const int32_t* start; // [B] position of each sample's first row, or NULL
    int64_t T;
    int B, pos64;
    int heads;            // of both tensors
    int hp;               // heads a thread walks
    int half;             // rot_dim / 2
    int items, rot_items; // column items of a row, and those that turn
    int tokens;           // tokens of a block
    float scale, sine;    // amplitude of the cosines; of the sines (- for the gradient)
    int copy0, copy1;     // whether the columns behind rot_dim are written (not in place)
};

template <typename E, int V>
struct alignas(sizeof(E) * V) Vec {
    E e[V];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float& y, float v) { y = v; }
__device__ __forceinline__ void put(__nv_bfloat16& y, float v) { y = __float2bfloat16_rn(v); }

template <typename E>
__device__ __forceinline__ void sincos_turns(uint64_t p, float& s, float& c) {
    // nearest 2^-32 turn, as a signed fraction of half a turn
    const int32_t t = (int32_t)(uint32_t)((p + 0x80000000ull) >> 32);
    const float x = (float)t * 4.656612873077392578125e-10f;   // 2^-31
    if constexpr (sizeof(E) == 4) {
        sincospif(x, &s, &c);
    } else {
        const float r = x * 3.14159265358979f;
        s = __sinf(r);
        c = __cosf(r);
    }
}

// E: row type, V: elements of a column item, INTER: pairs (2i, 2i + 1)
// rather than (i, i + rot_dim / 2).
template <typename E, int V, bool INTER>
__global__ void __launch_bounds__(kThreads)
rope_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int kPairs = INTER ? V / 2 : V;
    using X = Vec<E, V>;
    __shared__ uint64_t turns[GDPA_ROPE_MAX_PAIRS];
    if (threadIdx.x < a.half) turns[threadIdx.x] = a.turns[threadIdx.x];
    const int64_t row0 = (int64_t)blockIdx.x * a.tokens;
    int lo = 0, hi = a.B;   // off[lo] <= rows of this block < off[hi]
    if (!a.pos && a.B <= kCounted) {
        // the block looks at all offsets at once rather than each thread at
        // log2(B) of them one after the other
        int n0 = 0, n1 = 0;
        for (int i = threadIdx.x; i - (int)threadIdx.x <= a.B; i += kThreads) {
            const int64_t o = i <= a.B ? a.off[i] : INT64_MAX;
            n0 += __syncthreads_count(o <= row0);
            n1 += __syncthreads_count(o <= row0 + a.tokens - 1);
        }
        lo = max(n0 - 1, 0);
        hi = min(n1, a.B);
    }
    __syncthreads();
    const int tok = threadIdx.x / a.items, item = threadIdx.x - tok * a.items;
    const int64_t row = row0 + tok;
    if (tok >= a.tokens || row >= a.T) return;
    int64_t pos;
    if (a.pos) {
        pos = a.pos64 ? ((const int64_t*)a.pos)[row] : (int64_t)((const int32_t*)a.pos)[row];
    } else {
        // the last sample that starts at or before this row
        if (a.B == 0 || row >= a.off[a.B]) return;   // behind the last sample
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.off[mid] <= row) lo = mid; else hi = mid;
        }
        pos = row - a.off[lo] + (a.start ? a.start[lo] : 0);
    }
    const int h0 = blockIdx.y * a.hp, h1 = min(h0 + a.hp, a.heads);
    const bool turn = item < a.rot_items;
    int ca, cb = 0;   // first column of the item, and of its partner
    float cs[kPairs], sn[kPairs];
    if (turn) {
        ca = item * V;
        cb = ca + a.half;
        const int i0 = INTER ? ca / 2 : ca;
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            float s, c;
            sincos_turns<E>((uint64_t)pos * turns[i0 + j], s, c);
            sn[j] = s * a.sine;
            cs[j] = c * a.scale;
        }
    } else {
        ca = 2 * a.half + (item - a.rot_items) * V;
    }
#pragma unroll 4
    for (int h = h0; h < h1; ++h) {
        const bool second = h >= a.t[0].heads;
        const gdpa_rope_tensor& t = a.t[second ? 1 : 0];
        const int hh = second ? h - a.t[0].heads : h;
        const E* x = (const E*)t.x + row * t.x_token + hh * t.x_head;
        E* y = (E*)t.y + row * t.y_token + hh * t.y_head;
        const X xa = *reinterpret_cast<const X*>(x + ca);
        if (!turn) {
            if (second ? a.copy1 : a.copy0) *reinterpret_cast<X*>(y + ca) = xa;
            continue;
        }
        if constexpr (INTER) {
            X ya;
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                const float u = to_f(xa.e[2 * j]), v = to_f(xa.e[2 * j + 1]);
                put(ya.e[2 * j], u * cs[j] - v * sn[j]);
                put(ya.e[2 * j + 1], u * sn[j] + v * cs[j]);
            }
            *reinterpret_cast<X*>(y + ca) = ya;
        } else {
            const X xb = *reinterpret_cast<const X*>(x + cb);
            X ya, yb;
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                const float u = to_f(xa.e[j]), v = to_f(xb.e[j]);
                put(ya.e[j], u * cs[j] - v * sn[j]);
                put(yb.e[j], u * sn[j] + v * cs[j]);
            }
            *reinterpret_cast<X*>(y + ca) = ya;
            *reinterpret_cast<X*>(y + cb) = yb;
        }
    }
}

template <typename E, int V, bool INTER>
gdpa_status launch(RopeArgs& a, int d, cudaStream_t st) {
    a.rot_items = INTER ? 2 * a.half / V : a.half / V;
    a.items = a.rot_items + (a.copy0 || a.copy1 ? (d - 2 * a.half) / V : 0);
    a.tokens = kThreads / a.items;
    // Heads per thread: as many as leave about 2048 threads per SM (the
    // sines are then made once per token), down to one head for a few rows,
    // where the latency of one load and store is all there is.  (Half and
    // twice as many: the same times from 16 to 30000 samples, 1 and 4 heads.)
    const int64_t want = 152 * 2048;
    int hp = 1;
    while (hp < a.heads && hp < 16 && a.T * a.items * (a.heads / (2 * hp)) >= want) hp *= 2;
    a.hp = hp;
    const int64_t blocks = (a.T + a.tokens - 1) / a.tokens;
    if (blocks > 0x7fffffff) return GDPA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)blocks, (unsigned)((a.heads + hp - 1) / hp));
    rope_kernel<E, V, INTER><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? GDPA_OK : GDPA_ERR_CUDA;
}

// The widest item (16 bytes, then 8, then single elements or pairs) that
// divides the rotated columns, the rest of the row, the strides and the
// addresses.  Half a head's columns (half layout) or a head's (interleaved)
// split into such items.
template <typename E, int V>
bool fits(const RopeArgs& a, int d, bool inter) {
    if (inter ? (2 * a.half) % V : a.half % V) return false;
    if ((d - 2 * a.half) % V) return false;
    for (const gdpa_rope_tensor& t : a.t) {
        if (t.heads == 0) continue;
        if ((t.x_token | t.x_head | t.y_token | t.y_head) % V) return false;
        if (((uintptr_t)t.x | (uintptr_t)t.y) % (V * sizeof(E))) return false;
    }
    return true;
}

template <typename E>
gdpa_status dispatch(RopeArgs& a, int d, bool inter, cudaStream_t st) {
    constexpr int W = 16 / (int)sizeof(E);
    if (inter) {
        if (fits<E, W>(a, d, true)) return launch<E, W, true>(a, d, st);
        if (fits<E, W / 2>(a, d, true)) return launch<E, W / 2, true>(a, d, st);
        if (fits<E, 2>(a, d, true)) return launch<E, 2, true>(a, d, st);
        return GDPA_ERR_INVALID_ARG;
    }
    if (fits<E, W>(a, d, false)) return launch<E, W, false>(a, d, st);
    if (fits<E, W / 2>(a, d, false)) return launch<E, W / 2, false>(a, d, st);
    return launch<E, 1, false>(a, d, st);
}

// f / (2 pi) turns in 64-bit fixed point, modulo one turn, rounded to
// nearest: integer arithmetic on f's 53-bit mantissa and the first 128 bits
// of 1 / (2 pi), so that every host gives the same bits.
uint64_t turns_of(double f) {
    if (f == 0.0) return 0;
    int e;
    const double m = frexp(fabs(f), &e);                       // f = m 2^e, m in [1/2, 1)
    const uint64_t mant = (uint64_t)ldexp(m, 53);              // f = mant 2^(e - 53)
    const uint64_t c_hi = 0x28be60db9391054aull, c_lo = 0x7f09d5f47d4d3770ull;
    // mant * c (192 bits): w2 2^128 + w1 2^64 + w0
    const unsigned __int128 lo = (unsigned __int128)mant * c_lo;
    const unsigned __int128 hi = (unsigned __int128)mant * c_hi + (uint64_t)(lo >> 64);
    const uint64_t w1 = (uint64_t)hi, w2 = (uint64_t)(hi >> 64);
    // turns 2^64 = mant c 2^(e - 53 - 128 + 64) = (w2 w1 w0) >> (117 - e);
    // |f| <= 2^20, so the shift is at least 97: w0 only lies below the result
    const int shift = 117 - e - 64;   // of (w2 w1), >= 33
    if (shift > 128) return 0;        // below 2^-65 turns per position
    const unsigned __int128 w = ((unsigned __int128)w2 << 64) | w1;
    const unsigned __int128 r = shift == 128 ? (unsigned __int128)(w >> 127)
                                             : (w >> shift) + ((w >> (shift - 1)) & 1);
    const uint64_t t = (uint64_t)r;
    return f < 0.0 ? (uint64_t)0 - t : t;
}

bool rope_ok(const gdpa_rope* r) {
    return r && r->rot_dim >= 2 && r->rot_dim <= 2 * GDPA_ROPE_MAX_PAIRS && r->rot_dim % 2 == 0 &&
           (r->layout == GDPA_ROPE_HALF || r->layout == GDPA_ROPE_INTERLEAVED);
}

}  // namespace
}  // namespace gdpa

extern "C" {

gdpa_status gdpa_rope_init_freqs(gdpa_rope* rope, int rot_dim, gdpa_rope_layout layout,
                                 const double* freqs, float scale) {
    if (!rope || !freqs || rot_dim < 2 || rot_dim % 2 || !isfinite(scale)) return GDPA_ERR_INVALID_ARG;
    if (layout != GDPA_ROPE_HALF && layout != GDPA_ROPE_INTERLEAVED) return GDPA_ERR_INVALID_ARG;
    if (rot_dim > 2 * GDPA_ROPE_MAX_PAIRS) return GDPA_ERR_UNSUPPORTED;
    for (int i = 0; i < rot_dim / 2; ++i)
        if (!(fabs(freqs[i]) <= 1048576.0)) return GDPA_ERR_INVALID_ARG;   // also NaN
    memset(rope, 0, sizeof(*rope));
    rope->rot_dim = rot_dim;
    rope->layout = layout;
    rope->scale = scale;
    for (int i = 0; i < rot_dim / 2; ++i) rope->turns[i] = gdpa::turns_of(freqs[i]);
    return GDPA_OK;
}

gdpa_status gdpa_rope_init(gdpa_rope* rope, int rot_dim, gdpa_rope_layout layout, double base,
                           gdpa_rope_scaling scaling, double factor, double orig_len, double lo,
                           double hi, float scale) {
    if (rot_dim < 2 || rot_dim % 2) return GDPA_ERR_INVALID_ARG;
    if (rot_dim > 2 * GDPA_ROPE_MAX_PAIRS) return GDPA_ERR_UNSUPPORTED;
    if (!(base >= 1.0) || !isfinite(base)) return GDPA_ERR_INVALID_ARG;
    if (scaling < GDPA_ROPE_SCALING_NONE || scaling > GDPA_ROPE_SCALING_BY_PARTS)
        return GDPA_ERR_INVALID_ARG;
    if (scaling != GDPA_ROPE_SCALING_NONE && (!(factor >= 1.0) || !isfinite(factor)))
        return GDPA_ERR_INVALID_ARG;
    if (scaling == GDPA_ROPE_SCALING_BY_PARTS &&
        (!(orig_len > 0.0) || !isfinite(orig_len) || !(lo < hi) || !isfinite(lo) || !isfinite(hi)))
        return GDPA_ERR_INVALID_ARG;
    double f[GDPA_ROPE_MAX_PAIRS];
    if (scaling == GDPA_ROPE_SCALING_NTK && rot_dim > 2)
        base *= pow(factor, rot_dim / (rot_dim - 2.0));
    for (int i = 0; i < rot_dim / 2; ++i) {
        f[i] = pow(base, -2.0 * i / rot_dim);
        if (scaling == GDPA_ROPE_SCALING_LINEAR) f[i] /= factor;
        if (scaling == GDPA_ROPE_SCALING_BY_PARTS) {
            const double turns = orig_len * f[i] / 6.283185307179586476925;
            const double keep = fmin(1.0, fmax(0.0, (turns - lo) / (hi - lo)));
            f[i] = f[i] / factor * (1.0 - keep) + f[i] * keep;
        }
    }
    return gdpa_rope_init_freqs(rope, rot_dim, layout, f, scale);
}

gdpa_status gdpa_rope_apply(const gdpa_rope* rope, int inverse, gdpa_dtype dtype, int64_t T, int d,
                            const gdpa_rope_tensor* tensors, int n, const void* positions,
                            int position_bits, const int32_t* off, const int32_t* starts, int B,
                            void* stream) {
    if (!gdpa::rope_ok(rope) || T < 0 || !tensors || n < 1 || n > 2) return GDPA_ERR_INVALID_ARG;
    if (dtype != GDPA_BF16 && dtype != GDPA_F32) return GDPA_ERR_INVALID_ARG;
    if (d < rope->rot_dim) return GDPA_ERR_INVALID_ARG;
    if (d > 2 * GDPA_ROPE_MAX_PAIRS) return GDPA_ERR_UNSUPPORTED;
    if (positions ? (position_bits != 32 && position_bits != 64) || off
                  : !off || B < 0)
        return GDPA_ERR_INVALID_ARG;
    if ((uintptr_t)positions % (position_bits == 64 ? 8 : 4)) return GDPA_ERR_INVALID_ARG;
    gdpa::RopeArgs a;
    memset(&a, 0, sizeof(a));
    const size_t esize = dtype == GDPA_BF16 ? 2 : 4;
    for (int i = 0; i < n; ++i) {
        const gdpa_rope_tensor& t = tensors[i];
        if (t.heads < 0) return GDPA_ERR_INVALID_ARG;
        if (t.heads > 4096) return GDPA_ERR_UNSUPPORTED;
        if (t.heads > 0 && T > 0 &&
            (!t.x || !t.y || (uintptr_t)t.x % esize || (uintptr_t)t.y % esize))
            return GDPA_ERR_INVALID_ARG;
        a.t[i] = t;
        // strides that are never stepped: a single row's, a single head's
        if (T <= 1) a.t[i].x_token = a.t[i].y_token = 0;
        if (t.heads <= 1) a.t[i].x_head = a.t[i].y_head = 0;
        a.heads += t.heads;
    }
    if (T == 0 || a.heads == 0) return GDPA_OK;
    memcpy(a.turns, rope->turns, sizeof(a.turns));
    a.pos = positions;
    a.pos64 = position_bits == 64;
    a.off = off;
    a.start = positions ? nullptr : starts;
    a.T = T;
    a.B = B;
    a.half = rope->rot_dim / 2;
    a.scale = rope->scale;
    a.sine = inverse ? -rope->scale : rope->scale;
    auto moved = [](const gdpa_rope_tensor& t) {
        return t.heads > 0 &&
               (t.x != t.y || t.x_token != t.y_token || t.x_head != t.y_head);
    };
    a.copy0 = moved(a.t[0]);
    a.copy1 = moved(a.t[1]);
    const bool inter = rope->layout == GDPA_ROPE_INTERLEAVED;
    // the interleaved layout takes pairs of columns at a time
    if (inter)
        for (int i = 0; i < n; ++i) {
            const gdpa_rope_tensor& t = a.t[i];
            if (t.heads == 0) continue;
            if ((t.x_token | t.x_head | t.y_token | t.y_head | d) % 2 ||
                ((uintptr_t)t.x | (uintptr_t)t.y) % (2 * esize))
                return GDPA_ERR_INVALID_ARG;
        }
    cudaStream_t st = (cudaStream_t)stream;
    return dtype == GDPA_BF16 ? gdpa::dispatch<__nv_bfloat16>(a, d, inter, st)
                              : gdpa::dispatch<float>(a, d, inter, st);
}

}  // extern "C"
