// Attention over the history cache for bf16 rows with d = 64 or 128, on
// warp-level tensor-core products (m16n8k16).
//
// With a handful of query rows a key head (one new event, or a small tree, times
// the heads that share it) every cached byte is used for a few products only, so
// what bounds the kernel is reading the cache once.  Each warp therefore streams
// its own events: groups of 16 come in by bulk copies through a ring in shared
// memory, several groups ahead, and are used from there as operands without any
// rearrangement (the cache lies in the order that needs none): a thread's 16
// bytes of a key row are the B operand of S = Q K^T for 2 (8-bit: 4) steps of
// the contraction, whose order over d is free as long as Q has the same; two
// value rows' bytes interleaved are the B operand of O += P V, each thread's
// columns of O being a run of d.  A CTA's four warps take turns over the groups
// (KS = 4 / RT of them, the others hold further 16-row tiles of the same events)
// and join their sums in shared memory.
//
// 8-bit codes become f16 (exactly) and their products are f16 ones: S =
// 2^(e_k + e_q) q' . c, where q' is the row scaled by a power of two to below 2,
// in f16 (bf16's 8 bits fit; elements below 2^-14 of the largest lose bits, at
// most 2^-25 of it).  (Products of E4M3 operands, m16n8k32, are converted to f16
// ones by the compiler, and Q needs two of them: 217 us, not 197, for 256 users'
// 8-bit histories.)  The value rows' powers of two go
// into the weights, w 2^e_v F, rounded to f16 (2^-11 of each); F is a power of two
// that brings the largest w 2^e_v of the 32 events that are taken together to
// [2^7, 2^15], moved (and O with it) when they leave that range.  f16 has its 11 bits
// down to 2^-14, so weights down to 2^-21 of the largest of those 32 have them,
// whatever went before: a long flat tail of events keeps its share behind one event
// far above it.  (Weights more than 2^-94 below all that O holds may be lost.)  bf16
// caches use bf16 products, weights rounded to bf16 (2^-8 of each).
// Scores, maxima, sums and O are float32.
//
// Newest events of 512 users (1.5 GB of bf16 rows) 240 us, 6.2 TB/s; 256 users'
// 8-bit histories, 4 heads a key head (1.1 GB) 198 us, 5.8 TB/s.
//
// A group that some row does not see is masked bit by bit.  A hidden event's
// weight is 0, and 0 times an infinity or a NaN would be NaN: a masked group's
// values enter the product without those, which are then added one by one to the
// rows that see them.
#include <type_traits>

#include "cache_mma_rows.cuh"

namespace gdpa {
namespace {

using namespace tc;
using namespace cache_mma;

template <int D, bool FP8, bool SM, bool R8>
__global__ void __launch_bounds__(kThreads, Cfg<D, FP8, R8>::kPerSm)
cache_mma_kernel(const __grid_constant__ AttnArgs a) {
    using C = Cfg<D, FP8, R8>;
    using Rows = std::conditional_t<R8, Rows8<D, FP8, SM>, Rows16<D, FP8, SM>>;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ uint64_t full[C::kRing], empty[C::kRing];
    __shared__ int64_t scan_tmp[kThreads / 32 + 2];
    __shared__ uint8_t gone[C::kRing];              // groups of a stage whose page lies outside the cache
    __shared__ float2 ml[4][16];
    __shared__ int abort_flag;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gq = lane >> 2, t = lane & 3;
    const int RT = a.RT, KS = 4 / RT;
    const int rt = warp % RT, ks = warp / RT;
    const int NS = C::kRing / 4 * RT, ring0 = ks * NS;   // this warp's ring: stages ring0 .. ring0 + NS
    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < C::kRing; ++i) {
            mbar_init(&full[i], a.stall ? 2 : 1);   // (an arrival that never comes)
            mbar_init(&empty[i], RT);
        }
        fence_mbar_init();
    }
    const Abort ab{&abort_flag, a.c.err, a.wait_ns};
    asm volatile("griddepcontrol.launch_dependents;");
    if (tid == 0) a.desc[blockIdx.x].parts = 0;
    Share sh = find_share<kThreads>(a, scan_tmp);   // (synchronises the CTA)
    // places in this warp's ring, and the parity of their use: of the next group
    // to load (the wait for it to be empty) and to use; groups on their way
    int st_in = ring0, st_out = ring0, on_way = 0;
    uint32_t ph_in = 1, ph_out = 0;
    const auto next_place = [&](int& st, uint32_t& ph) {
        if (++st == ring0 + NS) {
            st = ring0;
            ph ^= 1;
        }
    };
    while (sh.more()) {
        const Segment g = next_segment(a, sh);
        if (g.rows == 0) break;
        constexpr int GN = C::kTake;
        const int stages = (g.n + GN - 1) / GN;
        const int mine = stages > ks ? (stages - ks + KS - 1) / KS : 0;   // this ring's: ks, ks + KS, ...
        // ---- loads: the ring's first warp; pages looked up 32 groups at a time, a
        // lane a copy: K and V of each group by columns of the layout, and the scales
        constexpr uint32_t kPiece = C::kKeys / C::kCols;
        constexpr int kCopies = 2 * C::kCols + (FP8 ? 2 : 0);   // of a group
        const int cu = lane / kCopies, cc = lane % kCopies;     // group of the stage, copy
        const bool is_v = cc & 1, is_scale = cc >= 2 * C::kCols;
        int64_t my_block = -1;
        const auto issue = [&](int i) {             // whole warp, stage i of this ring's
            if ((i & (32 / GN - 1)) == 0) {
                const int j = (ks + KS * (i + lane / GN)) * GN + lane % GN;
                my_block = j < g.n ? cache_block(a.c, a.w, g.b, (int64_t)segment_group(g, j) * kCacheGroup, g.h) : -1;
            }
            const int at0 = (i & (32 / GN - 1)) * GN;
            const int64_t blk = __shfl_sync(0xffffffffu, my_block, at0 + min(cu, GN - 1));
            const uint32_t there = __ballot_sync(0xffffffffu, my_block >= 0) >> at0 & ((1u << GN) - 1);
            if (!__all_sync(0xffffffffu, mbar_wait(&empty[st_in], ph_in, ab, 1))) return false;
            if (lane == 0) {
                gone[st_in] = (uint8_t)~there;
                mbar_arrive_expect_tx(&full[st_in], __popc(there) * (2 * C::kKeys + C::kScales));
            }
            __syncwarp();
            if (cu < GN && blk >= 0) {
                const int e0 = (segment_group(g, (ks + KS * i) * GN + cu) * kCacheGroup) & ((1 << a.c.page_log) - 1);
                if (is_scale) {
                    bulk_load(&full[st_in], smem + C::kMain + (st_in * GN + cu) * C::kScales + 16 * is_v,
                              (is_v ? a.c.vs : a.c.ks) + (blk << a.c.page_log) + e0, 16);
                } else {
                    const int col = cc >> 1;
                    const int at = C::kRow >= 128 ? ((col << a.c.page_log) + e0) * 128 : e0 * C::kRow;
                    bulk_load(&full[st_in], smem + st_in * C::kStage + cu * 2 * C::kKeys + is_v * C::kKeys + col * kPiece,
                              (is_v ? a.c.v : a.c.k) + blk * a.c.block + at, kPiece);
                }
            }
            ++on_way;
            next_place(st_in, ph_in);
            return true;
        };
        int ahead = 0;
        bool ok = true;
        if (rt == 0)
            for (; ahead < mine && ahead < NS && ok; ++ahead) ok = issue(ahead);

        // ---- the warp's rows
        const bool active = 16 * rt < g.rows;
        Rows rows;
        rows.start(a, g, 16 * rt, gq, t);

        // ---- the ring's stages
        for (int i = 0; i < mine && ok; ++i) {
            const int st = st_out;
            if (!__all_sync(0xffffffffu, mbar_wait(&full[st], ph_out, ab, 2))) {
                ok = false;
                break;
            }
            next_place(st_out, ph_out);
            const uint8_t* stage = smem + st * C::kStage;
            const uint32_t missing = gone[st] & ((1u << GN) - 1);   // (also groups behind the last)
            int e0[GN];
#pragma unroll
            for (int u = 0; u < GN; ++u) e0[u] = segment_group(g, (ks + KS * i) * GN + u) * kCacheGroup;
            if (active && e0[0] < rows.hi_max)
                rows.stage(a, g, e0, missing, stage, smem + C::kMain + st * GN * C::kScales, lane);
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
            --on_way;
            if (rt == 0 && ahead < mine) {
                ok = issue(ahead);
                ++ahead;
            }
        }
        // ---- the warps' sums, through the rings' memory
        if (!ok) {
            // gave up: copies still on their way land before the memory is given back
            if (rt == 0)
                for (; on_way > 0; --on_way) {
                    mbar_wait_teardown(&full[st_out], ph_out);
                    next_place(st_out, ph_out);
                }
        }
        __syncthreads();
        if (abort_flag) return;
        float* sums = reinterpret_cast<float*>(smem);
        rows.finish(g, 16 * rt, gq, t, sums + warp * C::kRows * C::kRowLen, ml[warp]);
        __syncthreads();
        finish_segment<__nv_bfloat16, SM, kThreads>(
            a, g, KS,
            [&](int w, int r, int c) { return reinterpret_cast<const float4*>(sums + w * C::kRows * C::kRowLen + C::sum_at(r, c)); },
            [&](int w, int r) { return ml[w][r]; });
        fence_proxy_async_smem();   // the next segment's copies write where these sums were
        __syncthreads();
    }
}

template <int D, bool FP8, bool SM, bool R8>
gdpa_status launch(const AttnArgs& a, int grid, cudaStream_t st) {
    using C = Cfg<D, FP8, R8>;
    static std::atomic<uint64_t> done{0};
    if (!cache_smem((const void*)cache_mma_kernel<D, FP8, SM, R8>, C::kBytes, done)) return GDPA_ERR_CUDA;
    cache_mma_kernel<D, FP8, SM, R8><<<grid, kThreads, C::kBytes, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? GDPA_OK : GDPA_ERR_CUDA;
}

template <int D, bool FP8>
gdpa_status launch_rows(const AttnArgs& a, int grid, cudaStream_t st) {
    const bool sm = a.act == kSoftmax;
    if (a.TM == 8) return sm ? launch<D, FP8, true, true>(a, grid, st) : launch<D, FP8, false, true>(a, grid, st);
    return sm ? launch<D, FP8, true, false>(a, grid, st) : launch<D, FP8, false, false>(a, grid, st);
}

}  // namespace

gdpa_status launch_cache_mma(const AttnArgs& a, int grid, cudaStream_t st) {
    const bool fp8 = a.c.store == GDPA_STORE_E4M3;
    if (a.c.d == 128) return fp8 ? launch_rows<128, true>(a, grid, st) : launch_rows<128, false>(a, grid, st);
    return fp8 ? launch_rows<64, true>(a, grid, st) : launch_rows<64, false>(a, grid, st);
}

}  // namespace gdpa
