// C entry points of shared-prefix attention: argument checks, plan ownership,
// workspaces, ordering of a plan's work, dispatch.
#include <string.h>

#include <algorithm>
#include <new>

#include "prefix_internal.h"

using gdpa::PrefixIO;
using gdpa::PrefixPlan;

namespace {

constexpr size_t kCaptures = 16;   // captures under way at once on one plan

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

void free_prefix(PrefixPlan* p) {
    if (!p) return;
    if (!p->host_only) {
        int cur = -1;
        if (cudaGetDevice(&cur) == cudaSuccess && cur != p->device) cudaSetDevice(p->device);
        // the buffers go back on a stream that has waited for the plan's
        // work; the host waits only if that stream cannot be made
        cudaStream_t fs = nullptr;
        if (cudaStreamCreateWithFlags(&fs, cudaStreamNonBlocking) != cudaSuccess) {
            fs = nullptr;
            if (p->ready) cudaEventSynchronize(p->ready);
            if (p->has_work) cudaEventSynchronize(p->last);
        } else {
            if (p->ready) cudaStreamWaitEvent(fs, p->ready, 0);
            if (p->has_work) cudaStreamWaitEvent(fs, p->last, 0);
        }
        void* bufs[] = {p->d_tables, p->d_parts, p->d_ml, p->d_grad};
        for (void* b : bufs)
            if (b) cudaFreeAsync(b, fs);
        if (p->last) cudaEventDestroy(p->last);
        for (const PrefixPlan::InCapture& e : p->captures) cudaEventDestroy(e.event);
        if (p->ready) cudaEventDestroy(p->ready);
        if (fs) cudaStreamDestroy(fs);
        if (cur >= 0 && cur != p->device) cudaSetDevice(cur);
    }
    delete p;
}

gdpa_status check_device(const PrefixPlan& p) {
    int cur = -1;
    if (cudaGetDevice(&cur) != cudaSuccess) return GDPA_ERR_CUDA;
    return cur == p.device ? GDPA_OK : GDPA_ERR_INVALID_ARG;
}

// A call's stream, and the capture that it is in (0: none).
struct Call {
    cudaStream_t st;
    unsigned long long capture = 0;
    explicit Call(cudaStream_t s) : st(s) {
        cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
        if (cudaStreamGetCaptureInfo(s, &status, &capture) != cudaSuccess ||
            status == cudaStreamCaptureStatusNone)
            capture = 0;
    }
};

// Order work on the call's stream after the plan's upload and, the workspace
// being one, after the plan's work so far.  That is waited for whatever the
// handle: equal ones need not be the same stream (the per-thread default stream
// is another one in every thread, a new stream may get a destroyed one's
// handle).  A captured launch cannot depend on events from outside its graph:
// the host makes sure that they have happened.  It follows the plan's last call
// of the same capture, which may be on another stream of it.
gdpa_status begin_work(PrefixPlan& p, const Call& c) {
    p.chain = 0;
    if (c.capture) {
        cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
        if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return GDPA_ERR_CUDA;
        const bool ok = cudaEventSynchronize(p.ready) == cudaSuccess &&
                        (!p.has_work || cudaEventSynchronize(p.last) == cudaSuccess);
        cudaThreadExchangeStreamCaptureMode(&mode);
        if (!ok) return GDPA_ERR_CUDA;
        for (const PrefixPlan::InCapture& e : p.captures)
            if (e.id == c.capture && cudaStreamWaitEvent(c.st, e.event, 0) != cudaSuccess) return GDPA_ERR_CUDA;
        return GDPA_OK;
    }
    if (!p.is_ready) {
        if (cudaStreamWaitEvent(c.st, p.ready, 0) != cudaSuccess) return GDPA_ERR_CUDA;
        // (a query could spoil a capture that another thread has under way)
        cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
        if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return GDPA_ERR_CUDA;
        p.is_ready = cudaEventQuery(p.ready) == cudaSuccess;
        cudaThreadExchangeStreamCaptureMode(&mode);
        if (!p.is_ready) cudaGetLastError();   // not ready is not an error
    }
    if (p.has_work && cudaStreamWaitEvent(c.st, p.last, 0) != cudaSuccess) return GDPA_ERR_CUDA;
    return GDPA_OK;
}

gdpa_status end_work(PrefixPlan& p, const Call& c) {
    if (c.capture) {   // (the graph's replays are the caller's to order)
        // captures may be under way side by side; the place of the one that the
        // plan was not in for longest is taken by a new one
        auto& all = p.captures;
        size_t i = 0;
        while (i < all.size() && all[i].id != c.capture) ++i;
        if (i == all.size()) {
            if (all.size() < kCaptures) {
                PrefixPlan::InCapture e{0, nullptr};
                if (cudaEventCreateWithFlags(&e.event, cudaEventDisableTiming) != cudaSuccess) return GDPA_ERR_CUDA;
                all.push_back(e);
            } else {
                i = 0;
            }
        }
        std::rotate(all.begin() + i, all.begin() + i + 1, all.end());
        all.back().id = 0;
        if (cudaEventRecord(all.back().event, c.st) != cudaSuccess) return GDPA_ERR_CUDA;
        all.back().id = c.capture;
        return GDPA_OK;
    }
    if (cudaEventRecord(p.last, c.st) != cudaSuccess) return GDPA_ERR_CUDA;
    p.has_work = true;
    return GDPA_OK;
}

gdpa_status create(const int32_t* q_off, const int32_t* kv_off, int B, const int32_t* group_off,
                   const int32_t* prefix_off, int G, int H, int Hkv, int d, gdpa_mask mask,
                   int window, int num_sms, bool host_only, cudaStream_t st, gdpa_prefix_plan* out) {
    if (!out) return GDPA_ERR_INVALID_ARG;
    *out = nullptr;
    if (!q_off || !group_off || !prefix_off || B < 0 || G < 0 || H < 1 || Hkv < 1 || d < 1 ||
        num_sms < 0 || (host_only && num_sms == 0))
        return GDPA_ERR_INVALID_ARG;
    if (H % Hkv) return GDPA_ERR_INVALID_ARG;
    if (mask != GDPA_MASK_NONE && mask != GDPA_MASK_CAUSAL_WINDOW) return GDPA_ERR_INVALID_ARG;
    if (mask == GDPA_MASK_CAUSAL_WINDOW && window < 1) return GDPA_ERR_INVALID_ARG;
    if (d > 128 || d % 4 != 0 || H / Hkv > gdpa::kBM) return GDPA_ERR_UNSUPPORTED;
    if ((int64_t)H * d > (1 << 20) || num_sms > 65536) return GDPA_ERR_UNSUPPORTED;
    if (!host_only && Call(st).capture) return GDPA_ERR_ALLOC;   // a graph must not own the buffers
    PrefixPlan* p = nullptr;
    gdpa_status s = GDPA_OK;
    try {   // the planner's tables grow with the batch
        p = new PrefixPlan();
        p->host_only = host_only;
        p->B = B;
        p->G = G;
        p->H = H;
        p->Hkv = Hkv;
        p->r = H / Hkv;
        p->tpt = gdpa::kBM / p->r;
        p->d = d;
        p->mask = mask;
        p->window = mask == GDPA_MASK_CAUSAL_WINDOW ? window : 0;
        if (!host_only) {
            if (cudaGetDevice(&p->device) != cudaSuccess ||
                (num_sms == 0 && cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount,
                                                        p->device) != cudaSuccess)) {
                delete p;
                return GDPA_ERR_CUDA;
            }
        }
        p->S = num_sms;
        p->captures.reserve(kCaptures);
        std::vector<int32_t> none;
        if (!kv_off) {
            none.assign((size_t)B + 1, 0);
            kv_off = none.data();
        }
        s = gdpa::build_prefix_plan(*p, q_off, kv_off, group_off, prefix_off);
    } catch (const std::bad_alloc&) {
        s = GDPA_ERR_ALLOC;
    }
    if (s == GDPA_OK && !host_only) {
        // one table upload: all lists, then the error word
        struct { const void* src; size_t bytes; size_t* off; } t[] = {
            {p->pieces.data(), p->pieces.size() * sizeof(gdpa::PrefixPiece), nullptr},
            {p->seg.data(), p->seg.size() * 4, &p->off_seg},
            {p->tiles.data(), p->tiles.size() * sizeof(gdpa::PrefixTile), &p->off_tiles},
            {p->own.data(), p->own.size() * sizeof(gdpa::PrefixOwn), &p->off_own},
            {p->units.data(), p->units.size() * sizeof(gdpa::PrefixUnit), &p->off_units},
            {p->useg.data(), p->useg.size() * 4, &p->off_useg},
            {p->smalls.data(), p->smalls.size() * sizeof(gdpa::PrefixUnit), &p->off_smalls},
            {p->eights.data(), p->eights.size() * sizeof(gdpa::PrefixUnit), &p->off_eights},
            {p->blocks.data(), p->blocks.size() * sizeof(gdpa::RowBlock), &p->off_blocks},
            {p->joins.data(), p->joins.size() * sizeof(gdpa::PrefixUnit), &p->off_joins},
        };
        size_t at = 0;
        for (auto& e : t) {
            if (e.off) *e.off = at;
            at += up256(e.bytes);
        }
        p->off_err = at;
        at += 256;
        const size_t rows = (size_t)p->n_part_rows;
        auto take = [&](void** dst, size_t bytes) {
            if (s != GDPA_OK || bytes == 0) return;
            if (cudaMallocAsync(dst, bytes, st) != cudaSuccess) {
                *dst = nullptr;
                s = GDPA_ERR_ALLOC;
            }
        };
        take((void**)&p->d_tables, at);
        take((void**)&p->d_parts, rows * d * sizeof(float));
        take((void**)&p->d_ml, rows * 2 * sizeof(float));
        if (s == GDPA_ERR_ALLOC) cudaGetLastError();
        // pageable sources: the copies have read them when the calls return
        size_t pos = 0;
        for (auto& e : t) {
            if (s == GDPA_OK && e.bytes &&
                cudaMemcpyAsync(p->d_tables + pos, e.src, e.bytes, cudaMemcpyHostToDevice, st) != cudaSuccess)
                s = GDPA_ERR_CUDA;
            pos += up256(e.bytes);
        }
        if (s == GDPA_OK &&
            (cudaMemsetAsync(p->dev_err(), 0, 16, st) != cudaSuccess ||
             cudaEventCreateWithFlags(&p->ready, cudaEventDisableTiming) != cudaSuccess ||
             cudaEventCreateWithFlags(&p->last, cudaEventDisableTiming) != cudaSuccess ||
             cudaEventRecord(p->ready, st) != cudaSuccess))
            s = GDPA_ERR_CUDA;
        if (s != GDPA_OK) cudaStreamSynchronize(st);
    }
    if (s != GDPA_OK) {
        free_prefix(p);
        return s;
    }
    *out = (gdpa_prefix_plan)p;
    return GDPA_OK;
}

bool valid_act(int a) { return a >= GDPA_ACT_GELU_ERF && a <= GDPA_ACT_SOFTMAX; }

gdpa_status check_inputs(const PrefixPlan& p, gdpa_dtype dtype, const PrefixIO& io) {
    if (dtype != GDPA_BF16 && dtype != GDPA_F32) return GDPA_ERR_INVALID_ARG;
    if (!valid_act(io.act)) return GDPA_ERR_INVALID_ARG;
    if ((p.Tq > 0 && !io.q) || (p.Tp > 0 && (!io.kp || !io.vp)) || (p.Tkv > 0 && (!io.k || !io.v)))
        return GDPA_ERR_INVALID_ARG;
    const void* in[] = {io.q, io.kp, io.vp, io.k, io.v};
    for (const void* x : in)
        if (!aligned16(x)) return GDPA_ERR_INVALID_ARG;
    return GDPA_OK;
}

// Gradients of a backward that would be written where something is still read,
// or written twice: dq is stored last, after everything has been read, the key
// gradients are not.
bool gradients_clash(const PrefixPlan& p, gdpa_dtype dt, const PrefixIO& io) {
    struct Range { uintptr_t at; size_t n; };
    const size_t e = dt == GDPA_BF16 ? 2 : 4, row = (size_t)p.d * e;
    const size_t nq = (size_t)p.Tq * p.H * row, np = (size_t)p.Tp * p.Hkv * row, nk = (size_t)p.Tkv * p.Hkv * row;
    const bool sm = io.act == GDPA_ACT_SOFTMAX;
    const Range out[] = {{(uintptr_t)io.dkp, np}, {(uintptr_t)io.dvp, np}, {(uintptr_t)io.dk, nk},
                         {(uintptr_t)io.dv, nk}, {(uintptr_t)io.dq, nq}};
    const Range in[] = {{(uintptr_t)io.q, nq}, {(uintptr_t)io.kp, np}, {(uintptr_t)io.vp, np}, {(uintptr_t)io.k, nk},
                        {(uintptr_t)io.v, nk}, {(uintptr_t)io.d_o, nq}, {(uintptr_t)io.o, sm ? nq : 0},
                        {(uintptr_t)io.lse, sm ? (size_t)p.Tq * p.H * 4 : 0}};
    auto meet = [](const Range& a, const Range& b) { return a.at < b.at + b.n && b.at < a.at + a.n && a.n && b.n; };
    for (int i = 0; i < 4; ++i) {
        for (const Range& x : in)
            if (meet(out[i], x)) return true;
        for (int j = i + 1; j < 5; ++j)
            if (meet(out[i], out[j])) return true;
    }
    return false;
}

// true when this plan and type run on the tensor-core kernels
bool use_tc(const PrefixPlan& p, gdpa_dtype dt) {
    return dt == GDPA_BF16 && p.kernel != GDPA_KERNEL_SIMT && (p.d == 64 || p.d == 128);
}

gdpa_status fwd(gdpa_prefix_plan plan, gdpa_dtype dtype, const PrefixIO& io, void* stream) {
    if (!plan || ((PrefixPlan*)plan)->host_only) return GDPA_ERR_INVALID_ARG;
    PrefixPlan& p = *(PrefixPlan*)plan;
    if (gdpa_status s = check_inputs(p, dtype, io)) return s;
    const bool sm = io.act == GDPA_ACT_SOFTMAX;
    if (p.Tq > 0 && (!io.o || !aligned16(io.o) || (uintptr_t)io.lse % 4)) return GDPA_ERR_INVALID_ARG;
    if (p.kernel == GDPA_KERNEL_TCGEN05 && !use_tc(p, dtype)) return GDPA_ERR_UNSUPPORTED;
    if (gdpa_status s = check_device(p)) return s;
    if (p.Tq == 0) return GDPA_OK;
    cudaStream_t st = (cudaStream_t)stream;
    std::lock_guard<std::mutex> hold(p.lock);
    const Call call(st);
    if (gdpa_status s = begin_work(p, call)) return s;
    gdpa_status s;
    if (use_tc(p, dtype)) {
        s = gdpa::launch_prefix_own_fwd(p, io, st);
        if (s == GDPA_OK) s = gdpa::launch_prefix_tc_fwd(p, io, st);
    } else {
        s = gdpa::launch_prefix_simt_fwd(p, dtype, io, st);
    }
    if (s == GDPA_OK) s = gdpa::launch_prefix_merge(p, dtype, io.o, sm ? io.lse : nullptr, sm, st);
    const gdpa_status e = end_work(p, call);
    return s != GDPA_OK ? s : e;
}

gdpa_status bwd(gdpa_prefix_plan plan, gdpa_dtype dtype, const PrefixIO& io, void* stream) {
    if (!plan || ((PrefixPlan*)plan)->host_only) return GDPA_ERR_INVALID_ARG;
    PrefixPlan& p = *(PrefixPlan*)plan;
    if (gdpa_status s = check_inputs(p, dtype, io)) return s;
    const bool sm = io.act == GDPA_ACT_SOFTMAX;
    if (p.Tq > 0 && (!io.d_o || !io.dq || (sm && (!io.o || !io.lse)))) return GDPA_ERR_INVALID_ARG;
    if ((p.Tp > 0 && (!io.dkp || !io.dvp)) || (p.Tkv > 0 && (!io.dk || !io.dv)))
        return GDPA_ERR_INVALID_ARG;
    const void* out[] = {io.d_o, io.dq, io.dkp, io.dvp, io.dk, io.dv, sm ? io.o : nullptr};
    for (const void* x : out)
        if (!aligned16(x)) return GDPA_ERR_INVALID_ARG;
    if ((uintptr_t)io.lse % 4 || gradients_clash(p, dtype, io)) return GDPA_ERR_INVALID_ARG;
    if (p.kernel == GDPA_KERNEL_TCGEN05 && !use_tc(p, dtype)) return GDPA_ERR_UNSUPPORTED;
    if (gdpa_status s = check_device(p)) return s;
    cudaStream_t st = (cudaStream_t)stream;
    std::lock_guard<std::mutex> hold(p.lock);
    const Call call(st);
    const size_t unit_parts = (size_t)p.n_unit_parts * 2 * gdpa::kBN * p.d;   // floats
    const size_t need = (unit_parts + (size_t)p.Tq * p.H) * sizeof(float);
    if (p.grad_bytes < need && call.capture) return GDPA_ERR_ALLOC;   // a graph must not own the workspace
    if (gdpa_status s = begin_work(p, call)) return s;
    if (p.grad_bytes < need) {
        if (cudaMallocAsync((void**)&p.d_grad, need, st) != cudaSuccess) {
            p.d_grad = nullptr;
            cudaGetLastError();
            return GDPA_ERR_ALLOC;
        }
        p.grad_bytes = need;
    }
    gdpa_status s = GDPA_OK;
    float* delta = p.d_grad + unit_parts;
    if (sm) s = gdpa::launch_prefix_delta(p, dtype, io, delta, st);
    if (use_tc(p, dtype)) {
        if (s == GDPA_OK) s = gdpa::launch_prefix_own_bwd8(p, io, delta, st);
        if (s == GDPA_OK) s = gdpa::launch_prefix_own_bwd(p, io, delta, st);
        if (s == GDPA_OK) s = gdpa::launch_prefix_tc_bwd(p, io, delta, st);
    } else if (s == GDPA_OK) {
        s = gdpa::launch_prefix_simt_bwd(p, dtype, io, delta, st);
    }
    if (s == GDPA_OK) s = gdpa::launch_prefix_join(p, dtype, io, st);
    if (s == GDPA_OK) s = gdpa::launch_prefix_merge(p, dtype, io.dq, nullptr, false, st);
    const gdpa_status e = end_work(p, call);
    return s != GDPA_OK ? s : e;
}

}  // namespace

extern "C" {

gdpa_status gdpa_prefix_create(const int32_t* q_off, const int32_t* kv_off, int B,
                               const int32_t* group_off, const int32_t* prefix_off, int G, int H,
                               int Hkv, int d, gdpa_mask mask, int window, int num_sms, void* stream,
                               gdpa_prefix_plan* out) {
    return create(q_off, kv_off, B, group_off, prefix_off, G, H, Hkv, d, mask, window, num_sms, false,
                  (cudaStream_t)stream, out);
}

gdpa_status gdpa_prefix_create_host(const int32_t* q_off, const int32_t* kv_off, int B,
                                    const int32_t* group_off, const int32_t* prefix_off, int G, int H,
                                    int Hkv, int d, gdpa_mask mask, int window, int num_sms,
                                    gdpa_prefix_plan* out) {
    return create(q_off, kv_off, B, group_off, prefix_off, G, H, Hkv, d, mask, window, num_sms, true,
                  nullptr, out);
}

gdpa_status gdpa_prefix_export(gdpa_prefix_plan plan, int32_t* pieces, int64_t cap, int64_t* n,
                               int32_t* seg) {
    if (!plan) return GDPA_ERR_INVALID_ARG;
    const PrefixPlan& p = *(PrefixPlan*)plan;
    if (n) *n = (int64_t)p.pieces.size();
    if (seg) memcpy(seg, p.seg.data(), p.seg.size() * 4);
    if (cap < (int64_t)p.pieces.size() || (!p.pieces.empty() && !pieces)) return GDPA_ERR_INVALID_ARG;
    if (!p.pieces.empty()) memcpy(pieces, p.pieces.data(), p.pieces.size() * sizeof(gdpa::PrefixPiece));
    return GDPA_OK;
}

gdpa_status gdpa_prefix_export_list(gdpa_prefix_plan plan, gdpa_prefix_list which, int32_t* rows,
                                    int64_t cap, int64_t* n) {
    if (!plan) return GDPA_ERR_INVALID_ARG;
    const PrefixPlan& p = *(PrefixPlan*)plan;
    const int32_t counts[4] = {(int32_t)p.n_part_rows, (int32_t)p.n_unit_parts, (int32_t)p.n_small8, p.warp_rows};
    const void* src = nullptr;
    size_t count = 0, bytes = 0;
    auto list = [&](const auto& v) {
        src = v.data();
        count = v.size();
        bytes = sizeof(v[0]);
    };
    switch (which) {
    case GDPA_PREFIX_UNITS: list(p.units); break;
    case GDPA_PREFIX_UNIT_SEG: list(p.useg); break;
    case GDPA_PREFIX_JOINS: list(p.joins); break;
    case GDPA_PREFIX_SMALLS: list(p.smalls); break;
    case GDPA_PREFIX_EIGHTS: list(p.eights); break;
    case GDPA_PREFIX_BLOCKS: list(p.blocks); break;
    case GDPA_PREFIX_TILES: list(p.tiles); break;
    case GDPA_PREFIX_OWN: list(p.own); break;
    case GDPA_PREFIX_COUNTS: src = counts, count = 1, bytes = sizeof(counts); break;
    default: return GDPA_ERR_INVALID_ARG;
    }
    if (n) *n = (int64_t)count;
    if (cap < (int64_t)count || (count && !rows)) return GDPA_ERR_INVALID_ARG;
    if (count) memcpy(rows, src, count * bytes);
    return GDPA_OK;
}

gdpa_status gdpa_prefix_set_kernel(gdpa_prefix_plan plan, gdpa_kernel kernel) {
    if (!plan || kernel < GDPA_KERNEL_AUTO || kernel > GDPA_KERNEL_SIMT) return GDPA_ERR_INVALID_ARG;
    ((PrefixPlan*)plan)->kernel = kernel;
    return GDPA_OK;
}

gdpa_status gdpa_prefix_set_wait_test(gdpa_prefix_plan plan, int limit_us, int stall) {
    if (!plan || limit_us < 0 || stall < 0 || stall > 2) return GDPA_ERR_INVALID_ARG;
    PrefixPlan& p = *(PrefixPlan*)plan;
    p.wait_limit_us = (uint32_t)limit_us;
    p.stall = stall;
    return GDPA_OK;
}

gdpa_status gdpa_prefix_fwd(gdpa_prefix_plan plan, gdpa_dtype dtype, const void* q, const void* kp,
                            const void* vp, const void* k, const void* v, void* o, float* lse,
                            float alpha, gdpa_act act, void* stream) {
    PrefixIO io{q, kp, vp, k, v};
    io.o = o;
    io.lse = lse;
    io.alpha = alpha;
    io.act = act;
    return fwd(plan, dtype, io, stream);
}

gdpa_status gdpa_prefix_bwd(gdpa_prefix_plan plan, gdpa_dtype dtype, const void* q, const void* kp,
                            const void* vp, const void* k, const void* v, const void* o,
                            const void* d_o, const float* lse, void* dq, void* dkp, void* dvp,
                            void* dk, void* dv, float alpha, gdpa_act act, void* stream) {
    PrefixIO io{q, kp, vp, k, v};
    io.o = const_cast<void*>(o);
    io.lse = const_cast<float*>(lse);
    io.d_o = d_o;
    io.dq = dq;
    io.dkp = dkp;
    io.dvp = dvp;
    io.dk = dk;
    io.dv = dv;
    io.alpha = alpha;
    io.act = act;
    return bwd(plan, dtype, io, stream);
}

gdpa_status gdpa_prefix_check(gdpa_prefix_plan plan, void* stream) {
    if (!plan || ((PrefixPlan*)plan)->host_only) return GDPA_ERR_INVALID_ARG;
    PrefixPlan& p = *(PrefixPlan*)plan;
    if (gdpa_status s = check_device(p)) return s;
    std::lock_guard<std::mutex> hold(p.lock);
    cudaStream_t st = (cudaStream_t)stream;
    if ((p.has_work && cudaEventSynchronize(p.last) != cudaSuccess) ||
        cudaEventSynchronize(p.ready) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess)
        return GDPA_ERR_CUDA;
    int32_t err[4];
    if (cudaMemcpyAsync(err, p.dev_err(), sizeof(err), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return GDPA_ERR_CUDA;
    if (err[0] == gdpa::kDevOk) return GDPA_OK;
    memcpy(p.last_err, err, sizeof(err));
    if (cudaMemsetAsync(p.dev_err(), 0, sizeof(err), st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return GDPA_ERR_CUDA;
    return err[0] == gdpa::kDevTimeout ? GDPA_ERR_TIMEOUT : GDPA_ERR_DEVICE;
}

gdpa_status gdpa_prefix_error_detail(gdpa_prefix_plan plan, int32_t* detail) {
    if (!plan || !detail) return GDPA_ERR_INVALID_ARG;
    memcpy(detail, ((PrefixPlan*)plan)->last_err, 16);
    return GDPA_OK;
}

int64_t gdpa_prefix_launches(gdpa_prefix_plan plan) {
    return plan ? ((PrefixPlan*)plan)->launches : -1;
}

void gdpa_prefix_destroy(gdpa_prefix_plan plan) { free_prefix((PrefixPlan*)plan); }

}  // extern "C"
