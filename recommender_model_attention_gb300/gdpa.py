"""Thin ctypes binding of the GDPA C ABI (``include/gdpa.h``).

Argument marshalling only: every step of planning and of the forward and
backward passes runs in the C++/CUDA library.  There is no fallback: if the
library has not been built, every call raises.

``stream=`` (default: the current stream): the call only enqueues work there.
Its inputs must be ready on that stream; outputs that it allocates are the
stream's, to be waited for before other streams read them.
"""

from __future__ import annotations

import ctypes
import os
import struct
from typing import NamedTuple

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgdpa_gb300.so")

ACT = {"gelu_erf": 0, "gelu_tanh": 1, "silu": 2, "gelu_taylor6": 3, "identity": 4,
       "softmax": 5}
MASK = {"none": 0, "causal_window": 1}
SCHED = {"zigzag": 0, "round_robin": 1, "zigzag_timed": 2}
KERNEL = {"auto": 0, "tcgen05": 1, "simt": 2}
ROPE_LAYOUT = {"half": 0, "interleaved": 1}
ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}
# lists of a shared-prefix plan: (index, columns)
PREFIX_LIST = {"units": (0, 8), "unit_seg": (1, 1), "joins": (2, 8), "smalls": (3, 8), "eights": (4, 8),
               "blocks": (5, 2), "tiles": (6, 8), "own": (7, 4), "counts": (8, 4)}
KV_SPLIT_AUTO = -1   # max_kv_blocks_per_tile: the planner chooses
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported configuration", 3: "CUDA error",
          4: "allocation failed", 5: "kernel barrier wait timed out",
          6: "kernel reported an internal error",
          7: "batch exceeds the static scratch of gdpa_fwd_noalloc"}
BLOCK_M = 128
BLOCK_N = 128

_lib = None


class _RopeSpec(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("turns", ctypes.c_uint64 * 64)]


class GdpaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__("%s: %s (status %d)" % (what, STATUS.get(status, "?"), status))
        self.status = status


def lib():
    """The loaded shared library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("GDPA CUDA library missing (%s); build it with "
                               "recommender_model_attention_gb300.build()" % LIB_PATH)
        try:
            _torch_names()   # (importing torch loads the CUDA runtime the library links)
        except ImportError:
            pass
        L = ctypes.CDLL(LIB_PATH)
        i32p = ctypes.POINTER(ctypes.c_int32)
        i64p = ctypes.POINTER(ctypes.c_int64)
        vp = ctypes.c_void_p
        st = ctypes.c_int
        sig = {
            "gdpa_plan_create": [i32p, i32p, st, st, st, st, st, st, st, st, vp, ctypes.POINTER(vp)],
            "gdpa_plan_create_host": [i32p, i32p, st, st, st, st, st, st, st, st, ctypes.POINTER(vp)],
            "gdpa_plan_sizes": [vp, i64p, i64p, ctypes.POINTER(ctypes.c_int)],
            "gdpa_plan_export": [vp, i32p, ctypes.c_int64, i64p, i32p],
            "gdpa_plan_export_bwd": [vp, i32p, ctypes.c_int64, i64p, i32p, ctypes.POINTER(ctypes.c_int)],
            "gdpa_plan_set_kernel": [vp, st],
            "gdpa_plan_set_timing": [vp, st],
            "gdpa_plan_set_shared_q": [vp, st],
            "gdpa_plan_set_wait_test": [vp, st, st],
            "gdpa_plan_set_qk_norm": [vp, ctypes.c_float, ctypes.c_float],
            "gdpa_fwd": [vp, st, vp, vp, vp, vp, ctypes.c_float, st, vp],
            "gdpa_bwd": [vp, st, vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, st, vp],
            "gdpa_check": [vp, vp],
            "gdpa_error_detail": [vp, i32p],
            "gdpa_sm_times": [vp, st, ctypes.POINTER(ctypes.c_uint64), i32p],
            "gdpa_fwd_noalloc": [i32p, i32p, st, st, st, st, st, vp, vp, vp, vp, ctypes.c_float,
                                 st, vp],
            "gdpa_act_eval": [st, st, vp, vp, vp, ctypes.c_int64, vp],
            "gdpa_shard_batch": [i32p, i32p, st, st, st, st, st, i32p, i64p],
            "gdpa_softmax_fwd": [vp, st, vp, vp, vp, vp, vp, ctypes.c_float, vp],
            "gdpa_softmax_bwd": [vp, st, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, vp],
            "gdpa_mx_quantise": [vp, ctypes.c_int64, vp, vp, vp],
            "gdpa_mx_dequantise": [vp, vp, ctypes.c_int64, vp, vp],
            "gdpa_fwd_mx": [vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, st, vp],
            "gdpa_bwd_mx": [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, st, vp],
            "gdpa_rope_init": [ctypes.POINTER(_RopeSpec), st, st, ctypes.c_double, st, ctypes.c_double,
                               ctypes.c_double, ctypes.c_double, ctypes.c_double, ctypes.c_float],
            "gdpa_rope_init_freqs": [ctypes.POINTER(_RopeSpec), st, st,
                                     ctypes.POINTER(ctypes.c_double), ctypes.c_float],
            "gdpa_rope_apply": [ctypes.POINTER(_RopeSpec), st, st, ctypes.c_int64, st,
                                vp, st, vp, st, vp, vp, st, vp],
            "gdpa_prefix_create": [i32p, i32p, st, i32p, i32p, st, st, st, st, st, st, st, vp,
                                   ctypes.POINTER(vp)],
            "gdpa_prefix_create_host": [i32p, i32p, st, i32p, i32p, st, st, st, st, st, st, st,
                                        ctypes.POINTER(vp)],
            "gdpa_prefix_export": [vp, i32p, ctypes.c_int64, i64p, i32p],
            "gdpa_prefix_export_list": [vp, st, i32p, ctypes.c_int64, i64p],
            "gdpa_prefix_set_kernel": [vp, st],
            "gdpa_prefix_set_wait_test": [vp, st, st],
            "gdpa_prefix_fwd": [vp, st] + [vp] * 7 + [ctypes.c_float, st, vp],
            "gdpa_prefix_bwd": [vp, st] + [vp] * 13 + [ctypes.c_float, st, vp],
            "gdpa_prefix_check": [vp, vp],
            "gdpa_prefix_error_detail": [vp, i32p],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        L.gdpa_plan_launches.argtypes = [vp]
        L.gdpa_plan_launches.restype = ctypes.c_int64
        L.gdpa_plan_destroy.argtypes = [vp]
        L.gdpa_plan_destroy.restype = None
        L.gdpa_prefix_launches.argtypes = [vp]
        L.gdpa_prefix_launches.restype = ctypes.c_int64
        L.gdpa_prefix_destroy.argtypes = [vp]
        L.gdpa_prefix_destroy.restype = None
        L.gdpa_status_str.argtypes = [ctypes.c_int]
        L.gdpa_status_str.restype = ctypes.c_char_p
        _lib = L
    return _lib


# What the calls need of torch, looked up once by lib(): these entry points are
# also used for a handful of rows, where marshalling is most of the time.
_DTYPE_ID = _POSITION_BITS = _empty = _raw_stream = _current_device = _on_device = _f32 = None


def _torch_names():
    global _DTYPE_ID, _POSITION_BITS, _empty, _raw_stream, _current_device, _on_device, _f32
    import torch
    _f32 = torch.float32
    _DTYPE_ID = {torch.bfloat16: 0, torch.float32: 1}
    _POSITION_BITS = {torch.int32: 32, torch.int64: 64}
    _empty = torch.empty
    _current_device, _on_device = torch.cuda.current_device, torch.cuda.device
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if _raw_stream is None:
        def _raw_stream(index):
            return torch.cuda.current_stream(index).cuda_stream


def _ok(status: int, what: str):
    if status != 0:
        raise GdpaError(status, what)


def _i32(a):
    a = np.ascontiguousarray(np.asarray(a, dtype=np.int32))
    return a, a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))


def _stream_ptr(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


class Plan:
    """A GDPA tile plan (forward tiles and backward units dealt to SMs).

    max_kv_blocks: 0 = one forward tile per query tile; k > 0 = key ranges
    cut into chunks of at most k 128-row key blocks; "auto" = the planner's
    choice (2-block chunks when some query tile reaches 8 key blocks).
    """

    def __init__(self, q_off, kv_off, H: int, d: int, mask: str = "none", window: int = 0,
                 sched: str = "zigzag", num_sms: int = 0, max_kv_blocks: int = 0,
                 stream=None, host_only: bool = False):
        L = lib()
        qo, qp = _i32(q_off)
        ko, kp = _i32(kv_off)
        if len(qo) != len(ko) or len(qo) < 1:
            raise ValueError("offset arrays must both have B + 1 entries")
        self.B, self.H, self.d = len(qo) - 1, int(H), int(d)
        self.mask, self.window = mask, int(window)
        self.Tq, self.Tkv = int(qo[-1]), int(ko[-1])
        self.q_off, self.kv_off = qo.copy(), ko.copy()
        self.shared_q = 0
        self.q_rows = self.Tq   # rows of q and dq (the seeds in shared-query mode)
        mkb = KV_SPLIT_AUTO if max_kv_blocks == "auto" else int(max_kv_blocks)
        h = ctypes.c_void_p()
        if host_only:
            _ok(L.gdpa_plan_create_host(qp, kp, self.B, self.H, self.d, MASK[mask], int(window),
                                        SCHED[sched], int(num_sms), mkb,
                                        ctypes.byref(h)), "gdpa_plan_create_host")
        else:
            _ok(L.gdpa_plan_create(qp, kp, self.B, self.H, self.d, MASK[mask], int(window),
                                   SCHED[sched], int(num_sms), mkb,
                                   _stream_ptr(stream), ctypes.byref(h)), "gdpa_plan_create")
        self._h = h

    @property
    def handle(self):
        if self._h is None:
            raise RuntimeError("plan destroyed")
        return self._h

    def sizes(self):
        nf, nb, s = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int()
        _ok(lib().gdpa_plan_sizes(self.handle, ctypes.byref(nf), ctypes.byref(nb), ctypes.byref(s)),
            "gdpa_plan_sizes")
        return nf.value, nb.value, s.value

    @property
    def num_sms(self) -> int:
        return self.sizes()[2]

    def export(self):
        """(tiles int32 [n, 6] = b, h, m, kb0, kb1, sm;  seg int32 [S + 1])."""
        nf, _, S = self.sizes()
        tiles = np.zeros((max(nf, 1), 6), dtype=np.int32)
        seg = np.zeros(S + 1, dtype=np.int32)
        n = ctypes.c_int64()
        _ok(lib().gdpa_plan_export(self.handle, tiles.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                   nf, ctypes.byref(n),
                                   seg.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))), "gdpa_plan_export")
        return tiles[:n.value], seg

    def export_bwd(self):
        """(units int32 [n, 7] = b, h, j, m0, m1, flags, sm;  seg [S + 1];  zero_dq)."""
        _, nb, S = self.sizes()
        units = np.zeros((max(nb, 1), 7), dtype=np.int32)
        seg = np.zeros(S + 1, dtype=np.int32)
        n, z = ctypes.c_int64(), ctypes.c_int()
        _ok(lib().gdpa_plan_export_bwd(self.handle, units.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                       nb, ctypes.byref(n),
                                       seg.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                       ctypes.byref(z)), "gdpa_plan_export_bwd")
        return units[:n.value], seg, bool(z.value)

    def set_kernel(self, kernel: str):
        _ok(lib().gdpa_plan_set_kernel(self.handle, KERNEL[kernel]), "gdpa_plan_set_kernel")

    def set_shared_q(self, n_seeds: int):
        """Shared-query mode: q (and the backward's dq) hold n_seeds seed rows
        shared by every sample, sample b's queries being seeds 0 .. Lq_b - 1;
        0 restores per-token queries."""
        _ok(lib().gdpa_plan_set_shared_q(self.handle, int(n_seeds)), "gdpa_plan_set_shared_q")
        self.shared_q = int(n_seeds)
        self.q_rows = self.shared_q if self.shared_q > 0 else self.Tq

    def set_timing(self, enable: bool):
        _ok(lib().gdpa_plan_set_timing(self.handle, 1 if enable else 0), "gdpa_plan_set_timing")

    def set_qk_norm(self, gain: float = 1.0, eps: float = 1e-6):
        """Fused RMSNorm of the Q and K rows inside the kernels (gain > 0);
        gain = 0 turns it off."""
        _ok(lib().gdpa_plan_set_qk_norm(self.handle, ctypes.c_float(gain), ctypes.c_float(eps)),
            "gdpa_plan_set_qk_norm")

    def set_wait_test(self, limit_us: int = 0, stall: bool = False):
        """Failure-path test hook: bounded-wait limit (microseconds, 0 = the
        default) and whether CTA 0's loader skips its first query-tile load on
        the next tensor-core launches, so that a wait expires."""
        _ok(lib().gdpa_plan_set_wait_test(self.handle, int(limit_us), 1 if stall else 0),
            "gdpa_plan_set_wait_test")

    def sm_times(self, which: str = "fwd"):
        """(start_end uint64 [S, 2] in ns, smid int32 [S]) of the last timed launch."""
        S = self.num_sms
        se = np.zeros((S, 2), dtype=np.uint64)
        sm = np.zeros(S, dtype=np.int32)
        _ok(lib().gdpa_sm_times(self.handle, 0 if which == "fwd" else 1,
                                se.ctypes.data_as(ctypes.POINTER(ctypes.c_uint64)),
                                sm.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))), "gdpa_sm_times")
        return se, sm

    def check(self, stream=None):
        status = lib().gdpa_check(self.handle, _stream_ptr(stream))
        if status != 0:
            code, site, cta, word = self.error_detail()
            raise GdpaError(status, "gdpa_check (device code %d, wait site %d, CTA %d, %d)"
                            % (code, site, cta, word))

    def error_detail(self):
        """(device code, wait site, CTA, word) of the last failure that
        check() reported for this plan; zeros if none."""
        d = (ctypes.c_int32 * 4)()
        _ok(lib().gdpa_error_detail(self.handle, d), "gdpa_error_detail")
        return tuple(int(v) for v in d)

    @property
    def launches(self) -> int:
        return int(lib().gdpa_plan_launches(self.handle))

    def destroy(self):
        if getattr(self, "_h", None) is not None:
            lib().gdpa_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def _dtype_id(t):
    import torch
    if t.dtype == torch.bfloat16:
        return 0
    if t.dtype == torch.float32:
        return 1
    raise TypeError("GDPA takes bfloat16 or float32 tensors, got %s" % t.dtype)


def _check(t, rows, plan, name, dtype=None):
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if tuple(t.shape) != (rows, plan.H, plan.d):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), (rows, plan.H, plan.d)))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s" % (name, dtype))


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t.numel() else ctypes.c_void_p(0)


def _new(shape, dtype, device, stream):
    """An output tensor for work on ``stream`` (None: the current one).  Memory
    belongs to the stream it is allocated on: there it is free to be written,
    and it is not given out again before the current stream's uses are over."""
    if _empty is None:
        _torch_names()
    if stream is None:
        return _empty(shape, dtype=dtype, device=device)
    import torch
    with torch.cuda.stream(stream):
        t = _empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def gdpa_fwd(plan: Plan, q, k, v, o=None, alpha=None, act: str = "gelu_erf", stream=None):
    """O = act(alpha Q K^T) V per sample and head; returns O ([Tq, H, d], dtype of q)."""
    import torch
    _check(q, plan.q_rows, plan, "q")
    _check(k, plan.Tkv, plan, "k", q.dtype)
    _check(v, plan.Tkv, plan, "v", q.dtype)
    if o is None:
        o = _new((plan.Tq, plan.H, plan.d), q.dtype, q.device, stream)
    _check(o, plan.Tq, plan, "o", q.dtype)
    alpha = plan.d ** -0.5 if alpha is None else float(alpha)
    _ok(lib().gdpa_fwd(plan.handle, _dtype_id(q), _ptr(q), _ptr(k), _ptr(v), _ptr(o),
                       ctypes.c_float(alpha), ACT[act], _stream_ptr(stream)), "gdpa_fwd")
    return o


def gdpa_bwd(plan: Plan, q, k, v, do, dq=None, dk=None, dv=None, alpha=None,
             act: str = "gelu_erf", stream=None):
    """(dQ, dK, dV) as float32 tensors given the upstream gradient dO (dQ per
    seed row, summed over the samples, in shared-query mode)."""
    import torch
    _check(q, plan.q_rows, plan, "q")
    _check(k, plan.Tkv, plan, "k", q.dtype)
    _check(v, plan.Tkv, plan, "v", q.dtype)
    _check(do, plan.Tq, plan, "do", q.dtype)
    f32 = torch.float32
    dq = _new(q.shape, f32, q.device, stream) if dq is None else dq
    dk = _new(k.shape, f32, k.device, stream) if dk is None else dk
    dv = _new(v.shape, f32, v.device, stream) if dv is None else dv
    _check(dq, plan.q_rows, plan, "dq", f32)
    _check(dk, plan.Tkv, plan, "dk", f32)
    _check(dv, plan.Tkv, plan, "dv", f32)
    alpha = plan.d ** -0.5 if alpha is None else float(alpha)
    _ok(lib().gdpa_bwd(plan.handle, _dtype_id(q), _ptr(q), _ptr(k), _ptr(v), _ptr(do), _ptr(dq),
                       _ptr(dk), _ptr(dv), ctypes.c_float(alpha), ACT[act], _stream_ptr(stream)),
        "gdpa_bwd")
    return dq, dk, dv


class MX(NamedTuple):
    """An MXFP8 tensor: E4M3 codes (uint8, the values' shape) and one E8M0
    scale byte (exponent + 127) per 32 values along the last axis."""
    elements: "object"
    scales: "object"


def mx_quantise(x, stream=None) -> MX:
    """bf16 CUDA tensor (last axis a multiple of 32) -> its MXFP8 encoding."""
    import torch
    if not x.is_cuda or not x.is_contiguous() or x.dtype != torch.bfloat16:
        raise ValueError("mx_quantise takes a contiguous bfloat16 CUDA tensor")
    if x.shape[-1] % 32:
        raise ValueError("the last axis must be a multiple of 32")
    el = _new(x.shape, torch.uint8, x.device, stream)
    sc = _new(x.shape[:-1] + (x.shape[-1] // 32,), torch.uint8, x.device, stream)
    _ok(lib().gdpa_mx_quantise(_ptr(x), x.numel(), _ptr(el), _ptr(sc), _stream_ptr(stream)),
        "gdpa_mx_quantise")
    return MX(el, sc)


def mx_dequantise(m: MX, stream=None):
    """The bf16 values an MXFP8 tensor stands for."""
    import torch
    el, sc = m
    _mx_check(el, sc, 0, None, "x")
    x = _new(el.shape, torch.bfloat16, el.device, stream)
    _ok(lib().gdpa_mx_dequantise(_ptr(el), _ptr(sc), el.numel(), _ptr(x), _stream_ptr(stream)),
        "gdpa_mx_dequantise")
    return x


def _mx_check(el, sc, rows, plan, name):
    import torch
    for t, what in ((el, "elements"), (sc, "scales")):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != torch.uint8:
            raise ValueError("%s %s must be a contiguous uint8 CUDA tensor" % (name, what))
    if tuple(sc.shape) != tuple(el.shape[:-1]) + (el.shape[-1] // 32,) or el.shape[-1] % 32:
        raise ValueError("%s: scales must have one byte per 32 elements" % name)
    if plan is not None and tuple(el.shape) != (rows, plan.H, plan.d):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(el.shape),
                                                           (rows, plan.H, plan.d)))


def gdpa_fwd_mx(plan: Plan, q: MX, k: MX, v, o=None, alpha=None, act: str = "gelu_erf",
                stream=None):
    """gdpa_fwd with Q and K in MXFP8 (``mx_quantise``); V and O bf16."""
    import torch
    _mx_check(q.elements, q.scales, plan.q_rows, plan, "q")
    _mx_check(k.elements, k.scales, plan.Tkv, plan, "k")
    _check(v, plan.Tkv, plan, "v", torch.bfloat16)
    if o is None:
        o = _new((plan.Tq, plan.H, plan.d), torch.bfloat16, v.device, stream)
    _check(o, plan.Tq, plan, "o", torch.bfloat16)
    alpha = plan.d ** -0.5 if alpha is None else float(alpha)
    _ok(lib().gdpa_fwd_mx(plan.handle, _ptr(q.elements), _ptr(q.scales), _ptr(k.elements),
                          _ptr(k.scales), _ptr(v), _ptr(o), ctypes.c_float(alpha), ACT[act],
                          _stream_ptr(stream)), "gdpa_fwd_mx")
    return o


def gdpa_bwd_mx(plan: Plan, q, k, v, do, dq=None, dk=None, dv=None, alpha=None,
                act: str = "gelu_erf", stream=None):
    """gdpa_bwd with Q and K in MXFP8: float32 (dQ, dK, dV) with respect to the
    values the MXFP8 tensors stand for.  q = k = None reuses the bf16
    expansion of the plan's previous MXFP8 call (the forward's)."""
    import torch
    reuse = q is None and k is None
    if not reuse:
        _mx_check(q.elements, q.scales, plan.q_rows, plan, "q")
        _mx_check(k.elements, k.scales, plan.Tkv, plan, "k")
        ptrs = [_ptr(q.elements), _ptr(q.scales), _ptr(k.elements), _ptr(k.scales)]
    else:
        ptrs = [ctypes.c_void_p(0)] * 4
    _check(v, plan.Tkv, plan, "v", torch.bfloat16)
    _check(do, plan.Tq, plan, "do", torch.bfloat16)
    f32 = torch.float32
    dq = _new((plan.q_rows, plan.H, plan.d), f32, v.device, stream) if dq is None else dq
    dk = _new(v.shape, f32, v.device, stream) if dk is None else dk
    dv = _new(v.shape, f32, v.device, stream) if dv is None else dv
    _check(dq, plan.q_rows, plan, "dq", f32)
    _check(dk, plan.Tkv, plan, "dk", f32)
    _check(dv, plan.Tkv, plan, "dv", f32)
    alpha = plan.d ** -0.5 if alpha is None else float(alpha)
    _ok(lib().gdpa_bwd_mx(plan.handle, *ptrs, _ptr(v), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv),
                          ctypes.c_float(alpha), ACT[act], _stream_ptr(stream)), "gdpa_bwd_mx")
    return dq, dk, dv


def shard_batch(q_off, kv_off, H: int, num_ranks: int, mask: str = "none", window: int = 0):
    """(rank of each sample int32 [B], work of each rank int64 [R]): the
    samples of one batch dealt to ranks by work in zigzag order
    (gdpa_shard_batch)."""
    qo, qp = _i32(q_off)
    ko, kp = _i32(kv_off)
    if len(qo) != len(ko) or len(qo) < 1:
        raise ValueError("offset arrays must both have B + 1 entries")
    B = len(qo) - 1
    rank = np.zeros(max(B, 1), dtype=np.int32)
    work = np.zeros(int(num_ranks), dtype=np.int64)
    _ok(lib().gdpa_shard_batch(qp, kp, B, int(H), MASK[mask], int(window), int(num_ranks),
                               rank.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                               work.ctypes.data_as(ctypes.POINTER(ctypes.c_int64))),
        "gdpa_shard_batch")
    return rank[:B], work


def shard_rows(q_off, kv_off, rank_of_sample, rank: int):
    """The local batch of one rank: (local q_off, local kv_off, query row
    indices, key row indices, sample indices) of the samples dealt to
    ``rank``, in their batch order; the index arrays gather the rank's rows
    from (or scatter its results to) the whole batch's token-major tensors."""
    q_off = np.asarray(q_off, dtype=np.int64)
    kv_off = np.asarray(kv_off, dtype=np.int64)
    mine = np.nonzero(np.asarray(rank_of_sample) == rank)[0]
    lq = q_off[mine + 1] - q_off[mine]
    lkv = kv_off[mine + 1] - kv_off[mine]
    qi = np.concatenate([np.arange(q_off[b], q_off[b + 1]) for b in mine] or [np.zeros(0, np.int64)])
    ki = np.concatenate([np.arange(kv_off[b], kv_off[b + 1]) for b in mine] or [np.zeros(0, np.int64)])
    lo = np.concatenate([[0], np.cumsum(lq)]).astype(np.int32)
    lk = np.concatenate([[0], np.cumsum(lkv)]).astype(np.int32)
    return lo, lk, qi.astype(np.int64), ki.astype(np.int64), mine


def allreduce_seed_grad(dq, group=None):
    """Shared-query mode over several ranks, each with its own samples: each
    rank's ``dq`` ([n_seeds, H, d] float32 from gdpa_bwd) holds its samples'
    share of the seeds' gradient, and the sum over ranks, one all-reduce of
    that small tensor, is the gradient of the whole batch (the only exchange
    the sharded path has).  In place; returns ``dq``."""
    import torch.distributed as dist
    dist.all_reduce(dq, op=dist.ReduceOp.SUM, group=group)
    return dq


def gdpa_fwd_noalloc(q_off, kv_off, q, k, v, o, alpha=None, act: str = "gelu_erf",
                     mask: str = "none", window: int = 0, stream=None):
    """Forward into a caller-provided ``o`` with no allocation by the library.

    For callers that cannot allocate device memory themselves (see
    ``gdpa_fwd_noalloc`` in include/gdpa.h): bf16, d in {64, 128}, at most
    GDPA_NOALLOC_MAX_TILES (32768) forward tiles.
    """
    qo, qp = _i32(q_off)
    ko, kp = _i32(kv_off)
    B = len(qo) - 1
    H, d = int(q.shape[1]), int(q.shape[2])
    alpha = d ** -0.5 if alpha is None else float(alpha)
    _ok(lib().gdpa_fwd_noalloc(qp, kp, B, H, d, MASK[mask], int(window), _ptr(q), _ptr(k), _ptr(v),
                               _ptr(o), ctypes.c_float(alpha), ACT[act], _stream_ptr(stream)),
        "gdpa_fwd_noalloc")
    return o


def act_eval(x, act: str = "gelu_erf", fast=True, stream=None):
    """(act(x), act'(x)) element-wise with the kernels' device functions
    (``fast``: the tensor-core flavour, one element at a time; ``fast=2``:
    the same in the f32x2 pair form those kernels evaluate it in; false: the
    float32 CUDA-core one).  ``x``: a contiguous float32 CUDA tensor."""
    import torch
    if x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 CUDA tensor")
    y = _new(x.shape, x.dtype, x.device, stream)
    dy = _new(x.shape, x.dtype, x.device, stream)
    mode = 2 if fast == 2 else (1 if fast else 0)
    _ok(lib().gdpa_act_eval(ACT[act], mode, _ptr(x), _ptr(y), _ptr(dy),
                            ctypes.c_int64(x.numel()), _stream_ptr(stream)), "gdpa_act_eval")
    return y, dy


def gdpa_softmax_fwd(plan: Plan, q, k, v, o=None, lse=None, alpha=None, stream=None):
    """Softmax variant (Jagged Flash Attention): (O, lse), lse the row
    log-sum-exp [Tq, H] float32 the backward needs."""
    import torch
    _check(q, plan.q_rows, plan, "q")
    _check(k, plan.Tkv, plan, "k", q.dtype)
    _check(v, plan.Tkv, plan, "v", q.dtype)
    if o is None:
        o = _new((plan.Tq, plan.H, plan.d), q.dtype, q.device, stream)
    _check(o, plan.Tq, plan, "o", q.dtype)
    if lse is None:
        lse = _new((plan.Tq, plan.H), torch.float32, q.device, stream)
    if lse.dtype != torch.float32 or tuple(lse.shape) != (plan.Tq, plan.H) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [Tq, H] tensor")
    alpha = plan.d ** -0.5 if alpha is None else float(alpha)
    _ok(lib().gdpa_softmax_fwd(plan.handle, _dtype_id(q), _ptr(q), _ptr(k), _ptr(v), _ptr(o),
                               _ptr(lse), ctypes.c_float(alpha), _stream_ptr(stream)),
        "gdpa_softmax_fwd")
    return o, lse


def gdpa_softmax_bwd(plan: Plan, q, k, v, o, do, lse, dq=None, dk=None, dv=None, alpha=None,
                     stream=None):
    """(dQ, dK, dV) of the softmax variant from its forward's O and lse."""
    import torch
    f32 = torch.float32
    _check(q, plan.q_rows, plan, "q")
    _check(k, plan.Tkv, plan, "k", q.dtype)
    _check(v, plan.Tkv, plan, "v", q.dtype)
    _check(o, plan.Tq, plan, "o", q.dtype)
    _check(do, plan.Tq, plan, "do", q.dtype)
    if lse.dtype != f32 or tuple(lse.shape) != (plan.Tq, plan.H) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [Tq, H] tensor")
    dq = _new(q.shape, f32, q.device, stream) if dq is None else dq
    dk = _new(k.shape, f32, k.device, stream) if dk is None else dk
    dv = _new(v.shape, f32, v.device, stream) if dv is None else dv
    for t, n, rows in ((dq, "dq", plan.q_rows), (dk, "dk", plan.Tkv), (dv, "dv", plan.Tkv)):
        _check(t, rows, plan, n, f32)
    alpha = plan.d ** -0.5 if alpha is None else float(alpha)
    _ok(lib().gdpa_softmax_bwd(plan.handle, _dtype_id(q), _ptr(q), _ptr(k), _ptr(v), _ptr(o),
                               _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
                               ctypes.c_float(alpha), _stream_ptr(stream)), "gdpa_softmax_bwd")
    return dq, dk, dv


class Rope:
    """Rotary positions: which columns turn, how fast, and by what amplitude.

    rot_dim: the first columns of every head row that turn (even, <= d).
    layout: pairs (i, i + rot_dim / 2) "half" or (2 i, 2 i + 1) "interleaved".
    scaling: "none", "linear" (positions over ``factor``), "ntk" (the base
    stretched by ``factor``) or "by_parts" (pairs that turn less than ``lo``
    times over ``orig_len`` positions slowed by ``factor``, those over ``hi``
    left as they are, a ramp between).  scale: amplitude of the turned columns.
    freqs: radians per position of each pair instead of base and scaling.

    Host data only: one object serves every device, stream and thread.
    """

    def __init__(self, rot_dim: int, layout: str = "half", base: float = 10000.0,
                 scaling: str = "none", factor: float = 1.0, orig_len: float = 0.0, lo: float = 1.0,
                 hi: float = 32.0, scale: float = 1.0, freqs=None):
        self.rot_dim, self.layout = int(rot_dim), layout
        self.spec = _RopeSpec()
        self._ref = ctypes.byref(self.spec)
        if freqs is not None:
            f = np.ascontiguousarray(np.asarray(freqs, dtype=np.float64))
            if f.shape != (self.rot_dim // 2,):
                raise ValueError("freqs must have rot_dim / 2 entries")
            _ok(lib().gdpa_rope_init_freqs(ctypes.byref(self.spec), self.rot_dim,
                                           ROPE_LAYOUT[layout],
                                           f.ctypes.data_as(ctypes.POINTER(ctypes.c_double)), scale),
                "gdpa_rope_init_freqs")
        else:
            _ok(lib().gdpa_rope_init(ctypes.byref(self.spec), self.rot_dim, ROPE_LAYOUT[layout], base,
                                     ROPE_SCALING[scaling], factor, orig_len, lo, hi, scale),
                "gdpa_rope_init")


# gdpa_rope_tensor: x, y, heads, then the four strides
_rope_tensor = struct.Struct("=QQi4xqqqq").pack


def _rope_rows(x, y, T, d, dtype, dev, name, stream):
    """One tensor of a rope call: checks; its output, and its packed record."""
    shape, xs = x.shape, x.stride()
    if len(shape) != 3 or shape[0] != T or shape[2] != d or x.device != dev:
        raise ValueError("%s must be a [%d, heads, %d] tensor on %s, got %s on %s"
                         % (name, T, d, dev, tuple(shape), x.device))
    if x.dtype != dtype:
        raise TypeError("%s must be %s" % (name, dtype))
    heads = shape[1]
    if y is None:
        y = _new(shape, dtype, dev, stream)
        ys = (heads * d, d, 1)
    else:
        if y.shape != shape or y.dtype != dtype or y.device != dev:
            raise ValueError("%s output must have its input's shape, dtype and device" % name)
        ys = y.stride()
        if (T > 1 and ys[0] == 0) or (heads > 1 and ys[1] == 0):
            raise ValueError("%s output must not be an expanded tensor" % name)
    if d > 1 and (xs[2] != 1 or ys[2] != 1):
        raise ValueError("%s: the columns of a row must be contiguous" % name)
    return y, _rope_tensor(x.data_ptr(), y.data_ptr(), heads, xs[0], xs[1], ys[0], ys[1])


def _rope(rope, inverse, q, k, positions, offsets, starts, q_out, k_out, stream):
    shape = q.shape
    if len(shape) != 3 or not q.is_cuda:
        raise ValueError("q must be a [T, heads, d] CUDA tensor")
    T, d, dev, dtype = shape[0], shape[2], q.device, q.dtype
    kind = _DTYPE_ID.get(dtype)
    if kind is None:
        raise TypeError("GDPA takes bfloat16 or float32 tensors, got %s" % dtype)
    if (positions is None) == (offsets is None):
        raise ValueError("give either positions or offsets")
    if starts is not None and offsets is None:
        raise ValueError("starts belong to offsets")
    q_out, rows = _rope_rows(q, q_out, T, d, dtype, dev, "q", stream)
    n = 1
    if k is not None:
        k_out, more = _rope_rows(k, k_out, T, d, dtype, dev, "k", stream)
        rows += more
        n = 2
    elif k_out is not None:
        raise ValueError("k_out without k")
    bits, B, pos, off, start = 0, 0, None, None, None
    if positions is not None:
        bits = _POSITION_BITS.get(positions.dtype)
        if bits is None or positions.shape != (T,) or not positions.is_contiguous() or positions.device != dev:
            raise ValueError("positions must be a contiguous int32 or int64 [T] tensor on q's device")
        pos = positions.data_ptr()
    else:
        for t, what in ((offsets, "offsets"), (starts, "starts")):
            if t is not None and (_POSITION_BITS.get(t.dtype) != 32 or t.dim() != 1
                                  or not t.is_contiguous() or t.device != dev):
                raise ValueError("%s must be a contiguous int32 tensor on q's device" % what)
        B = offsets.shape[0] - 1
        if B < 0 or (starts is not None and starts.shape[0] != B):
            raise ValueError("offsets must have B + 1 entries and starts B")
        off = offsets.data_ptr()
        start = starts.data_ptr() if starts is not None and B else None
    if T:
        index = dev.index
        args = (rope._ref, inverse, kind, T, d, rows, n, pos, bits, off, start, B,
                _raw_stream(index) if stream is None else stream.cuda_stream)
        if index == _current_device():
            _ok(lib().gdpa_rope_apply(*args), "gdpa_rope_apply")
        else:
            with _on_device(index):
                _ok(lib().gdpa_rope_apply(*args), "gdpa_rope_apply")
    return q_out if k is None else (q_out, k_out)


def gdpa_rope_fwd(rope: Rope, q, k=None, positions=None, offsets=None, starts=None, q_out=None,
                  k_out=None, stream=None):
    """Q (and K of the same tokens) with rotary positions, in one launch.

    q, k: bf16 or float32 [T, heads, d] CUDA tensors, of any token and head
    strides (the Q and K parts of a packed projection).  positions: int32 or
    int64 [T]; or offsets (int32 [B + 1] CUDA tensor) with the optional int32
    [B] ``starts``: row t of sample b is at starts[b] + t - offsets[b], and
    rows behind the last offset are not written.  q_out, k_out: outputs (q and
    k themselves to work in place).  Returns q_out, or (q_out, k_out)."""
    return _rope(rope, 0, q, k, positions, offsets, starts, q_out, k_out, stream)


def gdpa_rope_bwd(rope: Rope, dq, dk=None, positions=None, offsets=None, starts=None, dq_out=None,
                  dk_out=None, stream=None):
    """Gradients with respect to gdpa_rope_fwd's inputs, given those of its
    outputs (the inverse turn, the amplitude included); arguments alike."""
    return _rope(rope, 1, dq, dk, positions, offsets, starts, dq_out, dk_out, stream)


class PrefixPlan:
    """Plan of shared-prefix attention: samples in groups that share keys.

    q_off, kv_off: int32 [B + 1] offsets of each sample's query rows and own
    keys (kv_off None: no own keys).  group_off: int32 [G + 1], group g holds
    samples group_off[g] .. group_off[g + 1].  prefix_off: int32 [G + 1], its
    prefix is rows prefix_off[g] .. prefix_off[g + 1] of kp and vp.  H query
    heads, ``kv_heads`` key heads (H unless given; a divisor of H).  mask,
    window: over a sample's own keys, as Plan's; the prefix is always seen.

    Belongs to the device that is current when it is made.
    """

    def __init__(self, q_off, kv_off, group_off, prefix_off, H: int, d: int, kv_heads=None,
                 mask: str = "none", window: int = 0, num_sms: int = 0, stream=None,
                 host_only: bool = False):
        L = lib()
        self._h = None
        qo, qp = _i32(q_off)
        ko, kp = _i32(np.zeros_like(qo) if kv_off is None else kv_off)
        go, gp = _i32(group_off)
        po, pp = _i32(prefix_off)
        if qo.ndim != 1 or qo.shape != ko.shape or len(qo) < 1:
            raise ValueError("q_off and kv_off must both have B + 1 entries")
        if go.ndim != 1 or go.shape != po.shape or len(go) < 1:
            raise ValueError("group_off and prefix_off must both have G + 1 entries")
        self.B, self.G = len(qo) - 1, len(go) - 1
        self.H, self.d = int(H), int(d)
        self.Hkv = self.H if kv_heads is None else int(kv_heads)
        self.Tq, self.Tkv, self.Tp = int(qo[-1]), int(ko[-1]), int(po[-1])
        self.num_sms = int(num_sms)
        self._rows, self._lse = (self.Tq, self.H, self.d), (self.Tq, self.H)
        self._prefix, self._keys = (self.Tp, self.Hkv, self.d), (self.Tkv, self.Hkv, self.d)
        h = ctypes.c_void_p()
        args = (qp, kp, self.B, gp, pp, self.G, self.H, self.Hkv, self.d, MASK[mask], int(window),
                int(num_sms))
        self.device = None
        if host_only:
            _ok(L.gdpa_prefix_create_host(*args, ctypes.byref(h)), "gdpa_prefix_create_host")
        else:
            import torch
            self.device = torch.device("cuda", torch.cuda.current_device())
            _ok(L.gdpa_prefix_create(*args, _stream_ptr(stream), ctypes.byref(h)),
                "gdpa_prefix_create")
        self._h = h

    @property
    def handle(self):
        if self._h is None:
            raise RuntimeError("plan destroyed")
        return self._h

    def export(self):
        """(pieces int32 [n, 12], seg int32 [num_sms + 1]) of a plan made with
        an explicit num_sms; columns as gdpa_prefix_export."""
        n = ctypes.c_int64()
        i32p = ctypes.POINTER(ctypes.c_int32)
        seg = np.zeros(self.num_sms + 1, dtype=np.int32) if self.num_sms else None
        lib().gdpa_prefix_export(self.handle, None, 0, ctypes.byref(n), None)
        pieces = np.zeros((max(1, n.value), 12), dtype=np.int32)
        _ok(lib().gdpa_prefix_export(self.handle, pieces.ctypes.data_as(i32p), n.value,
                                     ctypes.byref(n),
                                     None if seg is None else seg.ctypes.data_as(i32p)),
            "gdpa_prefix_export")
        return pieces[:n.value], seg

    def export_list(self, name: str):
        """int32 [n, columns]: a list of the plan (PREFIX_LIST), as
        gdpa_prefix_export_list."""
        which, width = PREFIX_LIST[name]
        n = ctypes.c_int64()
        lib().gdpa_prefix_export_list(self.handle, which, None, 0, ctypes.byref(n))
        rows = np.zeros((max(1, n.value), width), dtype=np.int32)
        _ok(lib().gdpa_prefix_export_list(self.handle, which, rows.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                          n.value, ctypes.byref(n)), "gdpa_prefix_export_list")
        return rows[:n.value]

    def set_kernel(self, kernel: str):
        _ok(lib().gdpa_prefix_set_kernel(self.handle, KERNEL[kernel]), "gdpa_prefix_set_kernel")

    def set_wait_test(self, limit_us: int = 0, stall: int = 0):
        """Failure-path test hook: bounded-wait limit (microseconds, 0 = the
        default), and whether CTA 0's first query load is skipped, so that a
        wait expires: 1 in the forward and the dK, dV kernel, 2 in the dQ one."""
        _ok(lib().gdpa_prefix_set_wait_test(self.handle, int(limit_us), int(stall)),
            "gdpa_prefix_set_wait_test")

    def error_detail(self):
        """As Plan.error_detail."""
        d = (ctypes.c_int32 * 4)()
        _ok(lib().gdpa_prefix_error_detail(self.handle, d), "gdpa_prefix_error_detail")
        return tuple(int(v) for v in d)

    def check(self, stream=None):
        """Wait for the plan's work; raise if a kernel reported a failure."""
        status = lib().gdpa_prefix_check(self.handle, _stream_ptr(stream))
        if status != 0:
            raise GdpaError(status, "gdpa_prefix_check (device code %d, wait site %d, CTA %d, %d)"
                            % self.error_detail())

    @property
    def launches(self) -> int:
        return int(lib().gdpa_prefix_launches(self.handle))

    def destroy(self):
        if getattr(self, "_h", None) is not None:
            lib().gdpa_prefix_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def _prefix_tensor(t, shape, plan, name, dtype):
    """Address of a checked tensor of that shape (None for no rows)."""
    if t is None and shape[0] == 0:
        return None
    if t is None or t.shape != shape:
        raise ValueError("%s has shape %s, expected %s"
                         % (name, None if t is None else tuple(t.shape), shape))
    if t.device != plan.device:
        raise ValueError("%s must be on the plan's device %s" % (name, plan.device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s" % (name, dtype))
    return t.data_ptr() if shape[0] else None


def _prefix_lse(lse, plan):
    if (lse.dtype != _f32 or lse.shape != plan._lse or not lse.is_contiguous()
            or lse.device != plan.device):
        raise ValueError("lse must be a contiguous float32 [Tq, H] tensor on the plan's device")
    return lse.data_ptr() if plan.Tq else None


def _prefix_inputs(plan, q, kp, vp, k, v):
    if plan.device is None:
        raise ValueError("a host-only plan cannot launch")
    dt = q.dtype
    kind = _DTYPE_ID.get(dt)
    if kind is None:
        raise TypeError("GDPA takes bfloat16 or float32 tensors, got %s" % dt)
    return (kind, _prefix_tensor(q, plan._rows, plan, "q", dt),
            _prefix_tensor(kp, plan._prefix, plan, "kp", dt),
            _prefix_tensor(vp, plan._prefix, plan, "vp", dt),
            _prefix_tensor(k, plan._keys, plan, "k", dt), _prefix_tensor(v, plan._keys, plan, "v", dt))


def _prefix_call(f, what, plan, args, alpha, act, stream):
    index = plan.device.index
    args += (plan.d ** -0.5 if alpha is None else alpha, ACT[act],
             _raw_stream(index) if stream is None else stream.cuda_stream)
    if index == _current_device():
        _ok(f(plan.handle, *args), what)
    else:
        with _on_device(index):
            _ok(f(plan.handle, *args), what)


def _prefix_fwd(plan, q, kp, vp, k, v, o, lse_ptr, alpha, act, stream):
    args = _prefix_inputs(plan, q, kp, vp, k, v)
    if o is None:
        o = _new(plan._rows, q.dtype, plan.device, stream)
        out = o.data_ptr()
    else:
        out = _prefix_tensor(o, plan._rows, plan, "o", q.dtype)
    args += (out, lse_ptr)
    _prefix_call(lib().gdpa_prefix_fwd, "gdpa_prefix_fwd", plan, args, alpha, act, stream)
    return o


def gdpa_prefix_fwd(plan: PrefixPlan, q, kp, vp, k=None, v=None, o=None, alpha=None,
                    act: str = "gelu_erf", stream=None):
    """O ([Tq, H, d], dtype of q): every query attends to its group's prefix
    (kp, vp [Tp, kv_heads, d]) and its sample's own keys (k, v [Tkv, kv_heads,
    d]; None if there are none) with weights act(alpha q.k)."""
    return _prefix_fwd(plan, q, kp, vp, k, v, o, None, alpha, act, stream)


def gdpa_prefix_softmax_fwd(plan: PrefixPlan, q, kp, vp, k=None, v=None, o=None, lse=None,
                            alpha=None, stream=None):
    """The softmax variant over prefix and own keys together: (O, lse)."""
    if plan.device is None:
        raise ValueError("a host-only plan cannot launch")
    if lse is None:
        lse = _new(plan._lse, _f32, plan.device, stream)
        ptr = lse.data_ptr()
    else:
        ptr = _prefix_lse(lse, plan)
    return _prefix_fwd(plan, q, kp, vp, k, v, o, ptr, alpha, "softmax", stream), lse


def _prefix_bwd(plan, q, kp, vp, k, v, o, do, lse, grads, alpha, act, stream):
    dt = q.dtype
    args = _prefix_inputs(plan, q, kp, vp, k, v)
    args += (None if o is None else _prefix_tensor(o, plan._rows, plan, "o", dt),
             _prefix_tensor(do, plan._rows, plan, "do", dt), None if lse is None else _prefix_lse(lse, plan))
    out = []
    for g, shape, name in zip(grads, (plan._rows, plan._prefix, plan._prefix, plan._keys, plan._keys),
                              ("dq", "dkp", "dvp", "dk", "dv")):
        if g is None:
            g = _new(shape, dt, plan.device, stream)
            args += (g.data_ptr(),)
        else:
            args += (_prefix_tensor(g, shape, plan, name, dt),)
        out.append(g)
    _prefix_call(lib().gdpa_prefix_bwd, "gdpa_prefix_bwd", plan, args, alpha, act, stream)
    return tuple(out)


def gdpa_prefix_bwd(plan: PrefixPlan, q, kp, vp, k, v, do, dq=None, dkp=None, dvp=None, dk=None,
                    dv=None, alpha=None, act: str = "gelu_erf", stream=None):
    """(dQ, dKp, dVp, dK, dV) given dO, in the inputs' dtype: the prefix's
    summed over the group's samples, key gradients over the query heads that
    share a key head."""
    if act == "softmax":
        raise ValueError("the softmax variant's gradients come from gdpa_prefix_softmax_bwd")
    return _prefix_bwd(plan, q, kp, vp, k, v, None, do, None, (dq, dkp, dvp, dk, dv), alpha, act,
                       stream)


def gdpa_prefix_softmax_bwd(plan: PrefixPlan, q, kp, vp, k, v, o, do, lse, dq=None, dkp=None,
                            dvp=None, dk=None, dv=None, alpha=None, stream=None):
    """(dQ, dKp, dVp, dK, dV) of the softmax variant from its forward's O and lse."""
    return _prefix_bwd(plan, q, kp, vp, k, v, o, do, lse, (dq, dkp, dvp, dk, dv), alpha, "softmax",
                       stream)
