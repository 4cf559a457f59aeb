// Attention over the history cache: the C entry points and the kernel that
// joins the parts of items that several CTAs share.
#include <string.h>

#include <atomic>

#include "cache_attn.cuh"
#include "tc_common.cuh"

namespace gdpa {
namespace {

constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
constexpr int kMaxGrid = 2048;   // CTAs of an attention kernel at most (their records fit a block's shared memory)

// Rows of few parts are a warp each, eight a block; a row of many parts is a
// block's, whose warps take turns over the parts and add up in shared memory.
// Both always add in the same order.  (A block a row throughout: 120 us for the
// 38400 rows of 2 or 3 parts that 8 x 512 rows on 16384 events leave.)
constexpr int kFewParts = 8;

template <typename E, bool SM>
__device__ __forceinline__ void put_row(const AttnArgs& a, const CacheDesc& t, int r, int lane, const float4& x, float M, float l) {
    const int rho = t.rho0 + r, tok = rho / a.G;
    const int64_t row = (int64_t)(t.t0 + tok) * a.H + t.h * a.G + (rho - tok * a.G);
    float f = 1.0f;
    if (SM) {
        f = l == 0.0f ? 0.0f : 1.0f / l;
        if (lane == 0 && a.lse) a.lse[row] = l == 0.0f ? -INFINITY : (M + log2f(l)) * 0.693147180559945309f;
    }
    const float y[4] = {x.x * f, x.y * f, x.z * f, x.w * f};
    if (4 * lane < a.c.d) put4((E*)a.o + row * a.c.d + 4 * lane, y);
}

// a part's factor and sum, given the row's maximum
__device__ __forceinline__ float part_factor(float m, float n, float M) {
    return m == -INFINITY ? (n == 0.0f ? 0.0f : n) : ex2_approx(m - M);   // (n: a NaN)
}

template <typename E, bool SM>
__global__ void __launch_bounds__(kJoinThreads, 4)   // (one wave of them)
cache_join_kernel(const __grid_constant__ AttnArgs a, int ctas) {
    __shared__ int first[kMaxGrid + 1];   // units of the items before: rows, or eights of them
    __shared__ int tmp[kJoinWarps];
    __shared__ float4 sums[kJoinWarps][32];
    __shared__ float2 ml[kJoinWarps];
    __shared__ float factor[kMaxGrid];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int d = a.c.d, ld = cache_slot(a.TM, d);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int base = 0;
    for (int c0 = 0; c0 < ctas; c0 += kJoinThreads) {
        const int c = c0 + tid;
        int n = 0;
        if (c < ctas) {
            const int parts = a.desc[c].parts;
            n = parts > 1 ? a.desc[c].rows : 0;
            if (parts <= kFewParts) n = (n + 7) >> 3;
        }
        int x = n;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, m);
            if (lane >= m) x += y;
        }
        if (lane == 31) tmp[warp] = x;
        __syncthreads();
        int before = base;
        for (int i = 0; i < kJoinWarps; ++i) {
            if (i < warp) before += tmp[i];
            base += tmp[i];
        }
        if (c < ctas) first[c] = before + x - n;
        __syncthreads();
    }
    if (tid == 0) first[ctas] = base;
    __syncthreads();
    for (int i = blockIdx.x; i < base; i += gridDim.x) {
        int lo = 0, hi = ctas;   // the item whose rows hold i (the last one with first <= i and rows)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first[mid] <= i) lo = mid; else hi = mid;
        }
        const CacheDesc t = a.desc[lo];
        // part p: slot 2 lo + 1, then 2 (lo + 1), 2 (lo + 2), ...
        const auto slot = [&](int p) { return a.part + (int64_t)(p == 0 ? 2 * lo + 1 : 2 * (lo + p)) * ld; };
        if (t.parts <= kFewParts) {
            const int r = 8 * (i - first[lo]) + warp;
            if (r >= t.rows) continue;
            float m = -INFINITY, n = 0.0f;
            if (SM && lane < t.parts) {
                m = slot(lane)[a.TM * d + r];
                n = slot(lane)[a.TM * (d + 1) + r];
            }
            float4 y[kFewParts];
#pragma unroll
            for (int p = 0; p < kFewParts; ++p)
                if (p < t.parts && 4 * lane < d) y[p] = *reinterpret_cast<const float4*>(slot(p) + r * d + 4 * lane);
            float M = m;
#pragma unroll
            for (int k = 1; k < kFewParts; k <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
            M = __shfl_sync(0xffffffffu, M, 0);
            const float f = SM ? part_factor(m, n, M) : 1.0f;
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float l = 0.0f;
#pragma unroll
            for (int p = 0; p < kFewParts; ++p) {
                if (p >= t.parts) break;
                const float g = __shfl_sync(0xffffffffu, f, p);
                l += __shfl_sync(0xffffffffu, n, p) * g;
                x.x += y[p].x * g;
                x.y += y[p].y * g;
                x.z += y[p].z * g;
                x.w += y[p].w * g;
            }
            put_row<E, SM>(a, t, r, lane, x, M, l);
            continue;
        }
        const int r = i - first[lo];
        float M = -INFINITY, l = 0.0f;
        if (SM) {   // a thread a part: the largest maximum, the parts' factors and the sum
            float m = -INFINITY, n = 0.0f;
            if (tid < t.parts) {
                m = slot(tid)[a.TM * d + r];
                n = slot(tid)[a.TM * (d + 1) + r];
            }
            M = m;
            for (int p = tid + kJoinThreads; p < t.parts; p += kJoinThreads) M = fmaxf(M, slot(p)[a.TM * d + r]);
#pragma unroll
            for (int k = 1; k < 32; k <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
            if (lane == 0) ml[warp].x = M;
            __syncthreads();
            for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, ml[w].x);
            for (int p = tid; p < t.parts; p += kJoinThreads) {
                if (p != tid) {
                    m = slot(p)[a.TM * d + r];
                    n = slot(p)[a.TM * (d + 1) + r];
                }
                const float f = part_factor(m, n, M);
                factor[p] = f;
                l += n * f;
            }
#pragma unroll
            for (int k = 1; k < 32; k <<= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
            if (lane == 0) ml[warp].y = l;
            __syncthreads();
        }
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (int p = warp; p < t.parts; p += kJoinWarps) {
            if (4 * lane < d) {
                const float4 y = *reinterpret_cast<const float4*>(slot(p) + r * d + 4 * lane);
                const float f = SM ? factor[p] : 1.0f;
                x.x += y.x * f;
                x.y += y.y * f;
                x.z += y.z * f;
                x.w += y.w * f;
            }
        }
        sums[warp][lane] = x;
        __syncthreads();
        if (warp == 0) {
            l = 0.0f;
            for (int w = 0; w < kJoinWarps; ++w) {
                if (w > 0) {
                    const float4 y = sums[w][lane];
                    x.x += y.x;
                    x.y += y.y;
                    x.z += y.z;
                    x.w += y.w;
                }
                if (SM) l += ml[w].y;
            }
            put_row<E, SM>(a, t, r, lane, x, M, l);
        }
        __syncthreads();
    }
}

template <typename E, bool SM>
gdpa_status launch_join(const AttnArgs& a, int ctas, int sms, cudaStream_t st) {
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3((unsigned)(4 * sms));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute at;
    memset(&at, 0, sizeof(at));
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cache_join_kernel<E, SM>, a, ctas) == cudaSuccess ? GDPA_OK : GDPA_ERR_CUDA;
}

// gdpa_cache_set_wait_test
std::atomic<uint32_t> wait_limit_us{0};
std::atomic<int> wait_stall{0};

enum Kind { kFew, kSimt, kMma, kTc };
struct Shape {
    Kind kind;
    int RT, TM, grid, sms, min_share, lead;
    int64_t bytes;
};

// Rows and heads (a multiple of the cache's) that the kernels' counts hold.
bool sizes_fit(const CacheView& c, int64_t T, int H) { return T <= kCacheMost && H / c.heads <= 128 && T * H <= 0x7fffffff; }

// The kernel, its tile and its workspace: rules on types and sizes alone.
gdpa_status shape(const CacheView& c, gdpa_dtype dt, int64_t T, int H, int B, Shape& s) {
    const int64_t rows = B > 0 ? T * (H / c.heads) / B : 0;   // of an average sample and key head
    const bool tc = dt == GDPA_BF16 && (c.d == 64 || c.d == 128);
    // Warp-level products up to 32 rows, tcgen05 above, whose tiles of 128 rows cost
    // much before the first event (32 users of 4 heads a key head, us, warp-level
    // and tcgen05: 32 rows on 300 events 19 and 24, on 4000 events 52 and 53; 64
    // rows 27 and 25, 89 and 55; 128 rows 42 and 29, 156 and 57).
    // On the CUDA cores: straight from the pages up to 4 rows, through shared memory
    // above (512 users, float32: one row 620 and 3199 us, 4 rows 416 and 875, 8 rows 413
    // and 460).
    s.kind = !tc ? rows <= 4 ? kFew : kSimt : rows <= 32 ? kMma : kTc;
    s.sms = cache_sms();
    if (s.sms == 0) return GDPA_ERR_CUDA;
    // What an item costs beside its events, in groups of 16 of them, and the fewest
    // that are worth a CTA (measured on the same; trees of 32 users on tcgen05: 75
    // us at 32 groups an item, 61 at 64, 71 at 160; windows of 1024 events of 128
    // users: 31 us at 12, 25 at 24, but 512 users' newest events 232 and 240).
    if (s.kind == kTc) {
        s.RT = 0;
        s.TM = rows <= 128 ? 128 : 256;
        s.grid = s.sms;
        s.min_share = 16;
        s.lead = 64;
    } else {
        // row tiles of 16 that a CTA holds: as many as an average sample fills
        s.RT = s.kind != kMma || rows <= 16 ? 1 : 2;
        s.TM = s.kind == kFew ? (rows <= 1 ? 1 : rows <= 2 ? 2 : 4) : s.kind == kMma && rows <= 8 ? 8 : 16 * s.RT;
        s.grid = s.sms * (s.kind == kFew ? cache_few_per_sm(c.store, s.TM) : s.kind == kMma && s.TM == 8 ? 3 : 2);   // resident
        s.lead = 20 / s.RT;
        s.min_share = 4 / s.RT;
    }
    if (s.grid > kMaxGrid) s.grid = kMaxGrid;
    s.bytes = (int64_t)s.grid * (sizeof(CacheDesc) + 2ll * cache_slot(s.TM, c.d) * 4);
    return GDPA_OK;
}

}  // namespace
}  // namespace gdpa

extern "C" {

gdpa_status gdpa_cache_workspace(const gdpa_cache* cache, gdpa_dtype dtype, int64_t T, int H, int B,
                                 int64_t* bytes) {
    gdpa::CacheView c;
    gdpa_status s;
    if (!gdpa::cache_view(cache, c, &s)) return s;
    if (!bytes || T < 0 || B < 0 || H < 1 || H % c.heads) return GDPA_ERR_INVALID_ARG;
    if (dtype != GDPA_BF16 && dtype != GDPA_F32) return GDPA_ERR_INVALID_ARG;
    if (!gdpa::sizes_fit(c, T, H)) return GDPA_ERR_UNSUPPORTED;
    gdpa::Shape p;
    s = gdpa::shape(c, dtype, T, H, B, p);
    if (s == GDPA_OK) *bytes = p.bytes;
    return s;
}

gdpa_status gdpa_cache_set_wait_test(int limit_us, int stall) {
    if (limit_us < 0 || stall < 0 || stall > 1) return GDPA_ERR_INVALID_ARG;
    gdpa::wait_limit_us.store((uint32_t)limit_us, std::memory_order_relaxed);
    gdpa::wait_stall.store(stall, std::memory_order_relaxed);
    return GDPA_OK;
}

gdpa_status gdpa_cache_fwd(const gdpa_cache* cache, gdpa_dtype dtype, int64_t T, int H,
                           const gdpa_cache_rows* q, void* o, float* lse, const gdpa_cache_where* where,
                           const gdpa_cache_attn* attn, void* workspace, int64_t workspace_bytes, void* stream) {
    using namespace gdpa;
    AttnArgs a;
    memset(&a, 0, sizeof(a));
    gdpa_status s;
    if (!cache_view(cache, a.c, &s)) return s;
    if (dtype != GDPA_BF16 && dtype != GDPA_F32) return GDPA_ERR_INVALID_ARG;
    if ((a.c.store == GDPA_STORE_BF16 && dtype != GDPA_BF16) || (a.c.store == GDPA_STORE_F32 && dtype != GDPA_F32))
        return GDPA_ERR_INVALID_ARG;
    if (T < 0 || H < 1 || H % a.c.heads || !q || !attn) return GDPA_ERR_INVALID_ARG;
    s = cache_where(where, T, a.c, a.w);
    if (s != GDPA_OK) return s;
    if (attn->mask < GDPA_CACHE_CAUSAL || attn->mask > GDPA_CACHE_TREE || attn->window < 0 || attn->sinks < 0)
        return GDPA_ERR_INVALID_ARG;
    if (attn->sinks > 0 && attn->window == 0) return GDPA_ERR_INVALID_ARG;
    if (attn->act < GDPA_ACT_GELU_ERF || attn->act > GDPA_ACT_SOFTMAX) return GDPA_ERR_INVALID_ARG;
    if (!(attn->alpha - attn->alpha == 0.0f)) return GDPA_ERR_INVALID_ARG;   // infinite or NaN
    if (lse && (attn->act != GDPA_ACT_SOFTMAX || (uintptr_t)lse % 4)) return GDPA_ERR_INVALID_ARG;
    const bool tree = attn->mask == GDPA_CACHE_TREE;
    if (T > 0 && tree && (!attn->parents || (uintptr_t)attn->parents % 4)) return GDPA_ERR_INVALID_ARG;
    a.G = H / a.c.heads;
    if (!sizes_fit(a.c, T, H)) return GDPA_ERR_UNSUPPORTED;
    if (T == 0 || a.w.B == 0) return GDPA_OK;
    const size_t es = dtype == GDPA_BF16 ? 2 : 4;
    if (!q->x || (uintptr_t)q->x % es || !o || (uintptr_t)o % 16) return GDPA_ERR_INVALID_ARG;
    Shape p;
    s = shape(a.c, dtype, T, H, a.w.B, p);
    if (s != GDPA_OK) return s;
    if (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < p.bytes) return GDPA_ERR_INVALID_ARG;
    a.q = q->x;
    a.qt = T > 1 ? q->token : 0;
    a.qh = H > 1 ? q->head : 0;
    a.q_wide = (uintptr_t)q->x % 16 == 0 && a.qt * (int64_t)es % 16 == 0 && a.qh * (int64_t)es % 16 == 0;
    a.o = o;
    a.lse = lse;
    a.parents = tree ? attn->parents : nullptr;
    a.H = H;
    a.mask = attn->mask;
    a.window = attn->window;
    a.sinks = attn->sinks;
    a.act = attn->act;
    a.TM = p.TM;
    a.RT = p.RT;
    a.min_share = p.min_share;
    a.lead = p.lead;
    a.wait_ns = tc::wait_limit_ns(wait_limit_us.load(std::memory_order_relaxed));
    a.stall = wait_stall.load(std::memory_order_relaxed);
    a.desc = (CacheDesc*)workspace;
    a.part = (float*)(a.desc + p.grid);
    const bool sm = a.act == kSoftmax;
    // the warp-level kernel's scores are in powers of two
    a.alpha = p.kind == kMma && sm ? attn->alpha * kLog2e : attn->alpha;
    cudaStream_t st = (cudaStream_t)stream;
    s = p.kind == kFew ? launch_cache_few(a, dtype, p.grid, st)
        : p.kind == kSimt ? launch_cache_simt(a, dtype, p.grid, st)
        : p.kind == kMma ? launch_cache_mma(a, p.grid, st)
        : a.c.store == GDPA_STORE_E4M3 ? launch_cache_tc_e4m3(a, p.grid, st) : launch_cache_tc_bf16(a, p.grid, st);
    if (s != GDPA_OK) return s;
    if (dtype == GDPA_BF16)
        return sm ? launch_join<__nv_bfloat16, true>(a, p.grid, p.sms, st) : launch_join<__nv_bfloat16, false>(a, p.grid, p.sms, st);
    return sm ? launch_join<float, true>(a, p.grid, p.sms, st) : launch_join<float, false>(a, p.grid, p.sms, st);
}

}  // extern "C"
