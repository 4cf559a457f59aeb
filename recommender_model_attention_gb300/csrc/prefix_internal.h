// Internal declarations of shared-prefix attention (gdpa_prefix_*): the plan
// the host makes, the records its kernels walk, and the launchers.
//
// Rows.  The query rows of a key head hk are its r = H / Hkv query heads of
// every token, packed token by token: row t * r + j is head hk * r + j of
// token t.  A row tile is tpt = 128 / r whole tokens (at most 128 rows).
//
// Parts.  Attention over a union of key ranges is taken range by range: each
// piece of work gives, for the rows of one tile, unnormalised sums over its
// keys (and, for softmax, the reference maximum and the weights' sum), in a
// part of the plan's workspace; the merge joins the parts of every row.  A
// part of n rows starts at a row offset of the workspace and holds float4
// columns [d / 4][n] (so that a thread per row writes and reads whole lines)
// and float2 (maximum in base 2, sum) [n].
//
// Own keys of few rows and keys ("small": the rule is in prefix_plan.cpp) are
// taken by warp-level kernels in the tensor-core family; the CUDA-core family
// walks their pieces like any other.
#pragma once

#include <atomic>
#include <mutex>
#include <utility>
#include <vector>

#include "gdpa_internal.h"

namespace gdpa {

constexpr int kPieceOwn = 1;    // keys of the samples' own, not of the prefix
constexpr int kUnitPart = 256;
constexpr int kPieceDual = 2;   // one row tile: the slots take alternate key blocks

// One piece of forward work: keys [k0, k0 + nk) against one row tile of
// tokens [tok, tok + nA), or two tiles, [tok, tok + nA) and the nB tokens
// behind.  i0 / j0: positions of token `tok` and of key k0 in their sample
// (own keys).  part0/1: row offset of slot 0/1's sums (-1: unused).
struct PrefixPiece {
    int32_t tok, nA, nB, hk;
    int32_t k0, nk, flags, i0;
    int32_t j0, part0, part1, pad;
};
static_assert(sizeof(PrefixPiece) == 48, "PrefixPiece layout");

// 4 warp_rows rows of a piece's slot: rows from 4 warp_rows * (sub >> 1) on of
// slot sub & 1.
struct RowBlock {
    int32_t piece, sub;
};

// Backward unit: keys [k0, k0 + nk) (nk <= 128) of head hk against tokens
// [tok, tok + ntok), token `tok` at position i0 of its sample, key k0 at j0
// (own keys).  flags as a piece's; kUnitPart * (i + 1): one of several ranges of
// the tokens, whose dV and dK go to part i of the workspace, [128 keys][d]
// floats each.  In the list of joins: parts [tok, tok + ntok).
struct PrefixUnit {
    int32_t k0, nk, tok, ntok;
    int32_t hk, flags, i0, j0;
};
static_assert(sizeof(PrefixUnit) == 32, "PrefixUnit layout");

// One (row tile of a group, key head) for the merge: tokens [tok, tok + n),
// prefix parts at row offsets part + i * n * r, i < layers.
struct PrefixTile {
    int32_t tok, n, hk, part;
    int32_t layers, pad[3];
};
static_assert(sizeof(PrefixTile) == 32, "PrefixTile layout");

// Per token, its own keys: head hk's parts are at part + (hk * layers + i) *
// rows, the token's rows there from row0 on; layers = 0 without own keys.
struct PrefixOwn {
    int32_t part, row0, layers, rows;
};
static_assert(sizeof(PrefixOwn) == 16, "PrefixOwn layout");

struct PrefixPlan {
    int device = 0;
    bool host_only = false;
    int B = 0, G = 0, H = 0, Hkv = 0, r = 1, d = 0, mask = 0, window = 0, S = 0;
    int tpt = 128;               // tokens of a row tile
    int kernel = GDPA_KERNEL_AUTO;
    uint32_t wait_limit_us = 0;  // test hook (gdpa_prefix_set_wait_test)
    int stall = 0;
    int64_t Tq = 0, Tkv = 0, Tp = 0;
    int64_t n_part_rows = 0;
    std::vector<RowBlock> blocks;   // of the CUDA-core kernels, 4 warp_rows rows each
    int warp_rows = 8;
    int max_layers = 0;          // most prefix parts of a row tile
    std::vector<PrefixPiece> pieces; // the tensor-core family's, then the small own ones
    std::vector<int32_t> seg;        // [S + 1] first piece of each CTA
    std::vector<PrefixTile> tiles;
    std::vector<PrefixOwn> own;      // [Tq]
    std::vector<PrefixUnit> units;   // the tensor-core family's, then the small own ones
    std::vector<int32_t> useg;       // [S + 1] first unit of each CTA
    std::vector<PrefixUnit> joins;   // units in ranges, for the sum over them
    int64_t n_unit_parts = 0;
    // small own keys: one unit per sample and key head, those of at most 8
    // packed rows first; and the same cut into 8 rows each (j0: the first)
    std::vector<PrefixUnit> smalls, eights;
    int64_t n_small8 = 0;
    // device copies, one allocation (offsets below), and workspaces
    uint8_t* d_tables = nullptr;
    size_t off_seg = 0, off_tiles = 0, off_own = 0, off_units = 0, off_useg = 0, off_smalls = 0, off_eights = 0, off_joins = 0, off_blocks = 0, off_err = 0;
    float* d_parts = nullptr;        // [n_part_rows] x d floats
    float* d_ml = nullptr;           // [n_part_rows] float2
    float* d_grad = nullptr;         // backward: the parts of split units, then delta [Tq][H]
    size_t grad_bytes = 0;
    int32_t last_err[4] = {0, 0, 0, 0};
    int64_t launches = 0;
    int chain = 0;                   // kernels of the current call that a next one may start beside
    cudaEvent_t ready = nullptr;     // the upload, on the creation stream
    cudaEvent_t last = nullptr;      // the plan's latest work
    // its latest work in each of the captures that it was in last
    struct InCapture { unsigned long long id; cudaEvent_t event; };
    std::vector<InCapture> captures;
    bool has_work = false, is_ready = false;   // is_ready: the upload is known to be over
    std::mutex lock;                 // host state above

    const PrefixPiece* dev_pieces() const { return (const PrefixPiece*)d_tables; }
    const int32_t* dev_seg() const { return (const int32_t*)(d_tables + off_seg); }
    const PrefixTile* dev_tiles() const { return (const PrefixTile*)(d_tables + off_tiles); }
    const PrefixOwn* dev_own() const { return (const PrefixOwn*)(d_tables + off_own); }
    const PrefixUnit* dev_units() const { return (const PrefixUnit*)(d_tables + off_units); }
    const RowBlock* dev_blocks() const { return (const RowBlock*)(d_tables + off_blocks); }
    const PrefixUnit* dev_joins() const { return (const PrefixUnit*)(d_tables + off_joins); }
    const int32_t* dev_useg() const { return (const int32_t*)(d_tables + off_useg); }
    const PrefixUnit* dev_smalls() const { return (const PrefixUnit*)(d_tables + off_smalls); }
    const PrefixUnit* dev_eights() const { return (const PrefixUnit*)(d_tables + off_eights); }
    int32_t* dev_err() const { return (int32_t*)(d_tables + off_err); }
};

// The tensors of one call (device pointers, checked).
struct PrefixIO {
    const void *q, *kp, *vp, *k, *v;
    void* o = nullptr;               // forward out; backward: the forward's O (softmax)
    float* lse = nullptr;
    const void* d_o = nullptr;
    void *dq = nullptr, *dkp = nullptr, *dvp = nullptr, *dk = nullptr, *dv = nullptr;
    float alpha = 1.0f;
    int act = 0;
};

// Raise a kernel's dynamic shared-memory limit, once per device (`done`: one
// bit each, a static of the caller's).
template <typename K>
bool allow_smem(K kern, int bytes, int device, std::atomic<uint64_t>& done) {
    const uint64_t bit = device < 64 ? 1ull << device : 0;
    if (done.load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

// Launch a kernel; `early`: it may start once every block of the kernel before
// it on the stream has called grid_let_next (or ended), and must itself call
// grid_wait_previous before it ends, or before it reads what that kernel
// wrote: its own end then also says that the kernel before it has ended.
template <typename... P, typename... A>
bool launch_kernel(void (*kern)(P...), dim3 grid, int threads, int smem, cudaStream_t st, bool early,
                   A&&... args) {
    cudaLaunchConfig_t c = {};
    c.gridDim = grid;
    c.blockDim = dim3((unsigned)threads);
    c.dynamicSmemBytes = (size_t)smem;
    c.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = at;
    c.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&c, kern, std::forward<A>(args)...) == cudaSuccess;
}

#ifdef __CUDACC__
__device__ __forceinline__ void grid_let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A part's maximum, for the merge, which passes over parts whose maximum is
// -inf (nothing visible): one whose only scores are NaN must count.
__device__ __forceinline__ float counted(float m, float l) { return l != l && m == -INFINITY ? 0.0f : m; }

// 32 bytes of a row: as one store, a whole sector, where the row is aligned to
// it.  (Halves of sectors stored one after the other cost the gradients of the
// own keys 54 us, not 47, in a training batch of 32 users.)
__device__ __forceinline__ void store_sector(void* to, const uint32_t (&v)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]), "r"(v[1]),
                     "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(to)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4*>(to)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}
#endif

// Host planner (prefix_plan.cpp): INVALID_ARG for bad offsets.
gdpa_status build_prefix_plan(PrefixPlan& p, const int32_t* q_off, const int32_t* kv_off,
                              const int32_t* group_off, const int32_t* prefix_off);

// CUDA-core kernels (prefix_simt.cu), float32 arithmetic, any head dim.
gdpa_status launch_prefix_simt_fwd(PrefixPlan& p, gdpa_dtype dt, const PrefixIO& io, cudaStream_t st);
gdpa_status launch_prefix_simt_bwd(PrefixPlan& p, gdpa_dtype dt, const PrefixIO& io,
                                   const float* delta, cudaStream_t st);
// Tensor-core forward (prefix_tc_fwd.cu; bf16, d = 64 or 128): the parts.
gdpa_status launch_prefix_tc_fwd(PrefixPlan& p, const PrefixIO& io, cudaStream_t st);
// The parts of the small own keys (prefix_own.cu).
gdpa_status launch_prefix_own_fwd(PrefixPlan& p, const PrefixIO& io, cudaStream_t st);
// Tensor-core backward (prefix_tc_bwd.cu): dK, dV, and the parts of dQ, of all
// but the small own keys, whose are prefix_own.cu's (units of at most 8 rows)
// and prefix_own_bwd.cu's.
gdpa_status launch_prefix_tc_bwd(PrefixPlan& p, const PrefixIO& io, const float* delta, cudaStream_t st);
gdpa_status launch_prefix_own_bwd8(PrefixPlan& p, const PrefixIO& io, const float* delta, cudaStream_t st);
gdpa_status launch_prefix_own_bwd(PrefixPlan& p, const PrefixIO& io, const float* delta, cudaStream_t st);
// Join the parts of every row: into O and lse (io.o, io.lse; normalised when
// `softmax`), of element type dt.
gdpa_status launch_prefix_merge(PrefixPlan& p, gdpa_dtype dt, void* out, float* lse, bool softmax,
                                cudaStream_t st);
// Sum the parts of split backward units: into dkp, dvp, dk, dv.
gdpa_status launch_prefix_join(PrefixPlan& p, gdpa_dtype dt, const PrefixIO& io, cudaStream_t st);
// delta[t][h] = dO . O (softmax backward)
gdpa_status launch_prefix_delta(PrefixPlan& p, gdpa_dtype dt, const PrefixIO& io, float* delta,
                                cudaStream_t st);

}  // namespace gdpa
