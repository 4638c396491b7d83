"""Thin Python binding of the C ABI in include/cake_gg.h (ctypes; marshalling only).

Every function here converts arguments (torch tensors -> device pointers, the
current torch CUDA stream -> cudaStream_t) and calls the library of the same
name; all computation runs in the library's CUDA kernels.  There is no CPU or
eager fallback: if ``libcake_gg.so`` is missing, every call raises.

PyTorch is used only for device memory and streams.
"""
from __future__ import annotations

import ctypes
import functools
import os
import typing

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcake_gg.so")

CAKE_GG_OK = 0
CAKE_GG_ERR_INVALID_ARG = 1
CAKE_GG_ERR_ALIGNMENT = 2
CAKE_GG_ERR_OVERFLOW = 3
CAKE_GG_ERR_UNSUPPORTED = 4
CAKE_GG_ERR_WORKSPACE = 5
CAKE_GG_ERR_CUDA = 6
CAKE_GG_ERR_BAD_OFFSETS = 7
CAKE_GG_ERR_TIMEOUT = 8
CAKE_GG_ERR_SCRATCH_LIMIT = 9
CAKE_GG_ERR_BAD_ROWS = 10
CAKE_GG_NOALLOC_SCRATCH_BYTES = 32 << 20

CAKE_GG_FWD, CAKE_GG_DGRAD, CAKE_GG_WGRAD = 0, 1, 2
CAKE_GG_BF16, CAKE_GG_FP32, CAKE_GG_INT8, CAKE_GG_MX4 = 0, 1, 2, 3
CAKE_GG_ACT_NONE, CAKE_GG_ACT_SILU_MUL = 0, 1
CAKE_GG_MX4_MMA, CAKE_GG_MX4_ROWS = 0, 1
CAKE_GG_DEBUG_DROP_FIRST_LOAD = 1
CAKE_GG_SCORE_SOFTMAX, CAKE_GG_SCORE_SIGMOID = 0, 1
CAKE_GG_GROUP_MAX, CAKE_GG_GROUP_TOP2 = 0, 1

PASSES = {"fwd": CAKE_GG_FWD, "dgrad": CAKE_GG_DGRAD, "wgrad": CAKE_GG_WGRAD}
DTYPES = {"bf16": CAKE_GG_BF16, "fp32": CAKE_GG_FP32}
I8_X_DTYPES = {**DTYPES, "int8": CAKE_GG_INT8}
MX4_X_DTYPES = {**DTYPES, "mx4": CAKE_GG_MX4}
SCORES = {"softmax": CAKE_GG_SCORE_SOFTMAX, "sigmoid": CAKE_GG_SCORE_SIGMOID}
GROUP_SCORES = {"max": CAKE_GG_GROUP_MAX, "top2": CAKE_GG_GROUP_TOP2}
I8_ACTS = {None: CAKE_GG_ACT_NONE, "silu_mul": CAKE_GG_ACT_SILU_MUL}

EXPORTED = ["cake_gg_plan", "cake_gg_fwd", "cake_gg_dgrad", "cake_gg_wgrad",
            "cake_gg_check_status", "cake_gg_strerror", "cake_gg_tile_walk", "cake_gg_corun_spinner",
            "cake_gg_router_plan", "cake_gg_router_fp32",
            "cake_gg_i8_plan", "cake_gg_i8_gemm", "cake_gg_i8_quant",
            "cake_gg_mx4_plan", "cake_gg_mx4_gemm", "cake_gg_mx4_quant",
            "cake_gg_route_plan", "cake_gg_route", "cake_gg_route_grad", "cake_gg_combine_rows", "cake_gg_combine_grad",
            "cake_gg_zero_unnamed_rows"]


class CakeGGPlan(ctypes.Structure):
    """Mirror of cake_gg_plan_t (same field order, same C layout)."""
    _fields_ = [
        ("abi_version", ctypes.c_int32),
        ("pass_", ctypes.c_int32),
        ("E", ctypes.c_int32),
        ("N", ctypes.c_int32),
        ("K", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("M_max", ctypes.c_int64),
        ("deterministic", ctypes.c_int32),
        ("max_sms", ctypes.c_int32),
        ("tile_m", ctypes.c_int32),
        ("tile_n", ctypes.c_int32),
        ("tile_k", ctypes.c_int32),
        ("stages", ctypes.c_int32),
        ("pair", ctypes.c_int32),
        ("swap_ab", ctypes.c_int32),
        ("split_chunk", ctypes.c_int32),
        ("debug_flags", ctypes.c_int32),
        ("timeout_ns", ctypes.c_uint64),
        ("workspace_bytes", ctypes.c_uint64),
        ("staging_bufs", ctypes.c_int32),
        ("cluster_splits", ctypes.c_int32),
        ("tail_units", ctypes.c_int32),
        ("tail_splits", ctypes.c_int32),
        ("streamk_kblocks", ctypes.c_int32),
        ("epi_groups", ctypes.c_int32),
        ("tail_nsplit", ctypes.c_int32),
        ("reserved", ctypes.c_int32 * 1),
    ]

    def as_dict(self):
        return {f[0]: getattr(self, f[0]) for f in self._fields_ if f[0] != "reserved"}


class CakeGGRouterPlan(ctypes.Structure):
    """Mirror of cake_gg_router_plan_t (same field order, same C layout)."""
    _fields_ = [
        ("abi_version", ctypes.c_int32),
        ("R", ctypes.c_int32),
        ("T", ctypes.c_int64),
        ("K", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("workspace_bytes", ctypes.c_uint64),
        ("gemm", CakeGGPlan),
    ]


class CakeGGI8Plan(ctypes.Structure):
    """Mirror of cake_gg_i8_plan_t (same field order, same C layout)."""
    _fields_ = [
        ("abi_version", ctypes.c_int32),
        ("E", ctypes.c_int32),
        ("M_max", ctypes.c_int64),
        ("T", ctypes.c_int64),
        ("N", ctypes.c_int32),
        ("K", ctypes.c_int32),
        ("x_dtype", ctypes.c_int32),
        ("act", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("max_sms", ctypes.c_int32),
        ("path", ctypes.c_int32),
        ("pair", ctypes.c_int32),
        ("tile_rows", ctypes.c_int32),
        ("slots", ctypes.c_int32),
        ("stages", ctypes.c_int32),
        ("splits", ctypes.c_int32),
        ("debug_flags", ctypes.c_int32),
        ("first_rows", ctypes.c_int32),
        ("timeout_ns", ctypes.c_uint64),
        ("workspace_bytes", ctypes.c_uint64),
    ]

    def as_dict(self):
        return {f[0]: getattr(self, f[0]) for f in self._fields_ if f[0] != "reserved"}


class CakeGGMx4Plan(ctypes.Structure):
    """Mirror of cake_gg_mx4_plan_t (same field order, same C layout)."""
    _fields_ = [
        ("abi_version", ctypes.c_int32),
        ("E", ctypes.c_int32),
        ("M_max", ctypes.c_int64),
        ("T", ctypes.c_int64),
        ("N", ctypes.c_int32),
        ("K", ctypes.c_int32),
        ("x_dtype", ctypes.c_int32),
        ("act", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("max_sms", ctypes.c_int32),
        ("pair", ctypes.c_int32),
        ("tile_rows", ctypes.c_int32),
        ("stages", ctypes.c_int32),
        ("splits", ctypes.c_int32),
        ("debug_flags", ctypes.c_int32),
        ("path", ctypes.c_int32),
        ("timeout_ns", ctypes.c_uint64),
        ("workspace_bytes", ctypes.c_uint64),
    ]

    def as_dict(self):
        return {f[0]: getattr(self, f[0]) for f in self._fields_}


class CakeGGRouteOptions(ctypes.Structure):
    """Mirror of cake_gg_route_options_t (same field order, same C layout)."""
    _fields_ = [
        ("score", ctypes.c_int32),
        ("groups", ctypes.c_int32),
        ("top_groups", ctypes.c_int32),
        ("group_score", ctypes.c_int32),
        ("renormalize", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


class CakeGGRoutePlan(ctypes.Structure):
    """Mirror of cake_gg_route_plan_t (same field order, same C layout)."""
    _fields_ = [
        ("abi_version", ctypes.c_int32),
        ("E", ctypes.c_int32),
        ("T", ctypes.c_int64),
        ("top_k", ctypes.c_int32),
        ("cluster", ctypes.c_int32),
        ("blocks", ctypes.c_int32),
        ("block_tokens", ctypes.c_int32),
        ("workspace_bytes", ctypes.c_uint64),
    ]

    def as_dict(self):
        return {f[0]: getattr(self, f[0]) for f in self._fields_}


class CakeGGError(RuntimeError):
    def __init__(self, code, where):
        super().__init__(f"{where}: {cake_gg_strerror(code)} (status {code})")
        self.code = code


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libcake_gg.so; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with moe_ragged_grouped_gb300.build.build() "
            "(there is no fallback implementation)")
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    plan_p = ctypes.POINTER(CakeGGPlan)
    lib.cake_gg_plan.argtypes = [plan_p, ctypes.c_int, i32, i64, i32, i32, ctypes.c_int, ctypes.c_int, i32]
    lib.cake_gg_plan.restype = ctypes.c_int
    for name in ("cake_gg_fwd", "cake_gg_dgrad", "cake_gg_wgrad"):
        f = getattr(lib, name)
        f.argtypes = [plan_p, vp, vp, vp, vp, ctypes.c_int, ctypes.c_int, vp, sz, vp]
        f.restype = ctypes.c_int
    lib.cake_gg_check_status.argtypes = [vp, vp]
    lib.cake_gg_corun_spinner.argtypes = [i32, ctypes.c_uint64, vp]
    lib.cake_gg_corun_spinner.restype = ctypes.c_int
    lib.cake_gg_check_status.restype = ctypes.c_int
    lib.cake_gg_strerror.argtypes = [ctypes.c_int]
    lib.cake_gg_strerror.restype = ctypes.c_char_p
    lib.cake_gg_tile_walk.argtypes = [plan_p, ctypes.POINTER(ctypes.c_int32), i64,
                                      ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int64)]
    lib.cake_gg_tile_walk.restype = ctypes.c_int
    lib.cake_gg_wgrad_noalloc.argtypes = [plan_p, vp, vp, vp, vp, ctypes.c_int, ctypes.c_int, vp]
    lib.cake_gg_wgrad_noalloc.restype = ctypes.c_int
    rplan_p = ctypes.POINTER(CakeGGRouterPlan)
    lib.cake_gg_router_plan.argtypes = [rplan_p, i64, i32, i32, i32]
    lib.cake_gg_router_plan.restype = ctypes.c_int
    lib.cake_gg_router_fp32.argtypes = [rplan_p, vp, vp, vp, vp, sz, vp]
    lib.cake_gg_router_fp32.restype = ctypes.c_int
    i8plan_p = ctypes.POINTER(CakeGGI8Plan)
    lib.cake_gg_i8_plan.argtypes = [i8plan_p, i32, i64, i64, i32, i32, ctypes.c_int, ctypes.c_int, ctypes.c_int, i32]
    lib.cake_gg_i8_plan.restype = ctypes.c_int
    lib.cake_gg_i8_gemm.argtypes = [i8plan_p, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.cake_gg_i8_gemm.restype = ctypes.c_int
    lib.cake_gg_i8_quant.argtypes = [vp, ctypes.c_int, ctypes.c_int, i64, i32, vp, vp, vp]
    lib.cake_gg_i8_quant.restype = ctypes.c_int
    mx4plan_p = ctypes.POINTER(CakeGGMx4Plan)
    lib.cake_gg_mx4_plan.argtypes = [mx4plan_p, i32, i64, i64, i32, i32, ctypes.c_int, ctypes.c_int, ctypes.c_int, i32]
    lib.cake_gg_mx4_plan.restype = ctypes.c_int
    lib.cake_gg_mx4_gemm.argtypes = [mx4plan_p, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.cake_gg_mx4_gemm.restype = ctypes.c_int
    lib.cake_gg_mx4_quant.argtypes = [vp, ctypes.c_int, ctypes.c_int, i32, i64, i32, vp, vp, vp]
    lib.cake_gg_mx4_quant.restype = ctypes.c_int
    route_p, options_p = ctypes.POINTER(CakeGGRoutePlan), ctypes.POINTER(CakeGGRouteOptions)
    lib.cake_gg_route_plan.argtypes = [route_p, i64, i32, i32]
    lib.cake_gg_route_plan.restype = ctypes.c_int
    lib.cake_gg_route.argtypes = [route_p, options_p, vp, ctypes.c_int, i64, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.cake_gg_route.restype = ctypes.c_int
    lib.cake_gg_route_grad.argtypes = [i64, i32, i32, ctypes.c_int, ctypes.c_int, ctypes.c_float, vp, ctypes.c_int, i64, vp,
                                       vp, vp, vp]
    lib.cake_gg_route_grad.restype = ctypes.c_int
    lib.cake_gg_combine_rows.argtypes = [i64, i64, i32, i32, vp, ctypes.c_int, vp, vp, vp, ctypes.c_int, vp]
    lib.cake_gg_combine_rows.restype = ctypes.c_int
    lib.cake_gg_combine_grad.argtypes = [i64, i64, i32, i32, vp, ctypes.c_int, vp, ctypes.c_int, vp, vp, vp, vp, vp]
    lib.cake_gg_combine_grad.restype = ctypes.c_int
    lib.cake_gg_zero_unnamed_rows.argtypes = [i64, i64, i32, i32, vp, vp, ctypes.c_int, vp, vp]
    lib.cake_gg_zero_unnamed_rows.restype = ctypes.c_int
    _lib = lib
    return lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _current_stream(index):
    """The current stream's handle on a device (a few times cheaper than through a Stream object, where torch allows).

    Gives its name to torch's own function on the first call, as _current_device() does: a short
    product's time is the host's.
    """
    global _current_stream
    import torch
    _current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda i: torch.cuda.current_stream(i).cuda_stream)
    return _current_stream(index)


def _stream(stream, *tensors):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    for t in tensors:
        if t is not None and not isinstance(t, int) and getattr(t, "is_cuda", False):
            import torch
            return torch.cuda.current_stream(t.device).cuda_stream
    return 0


def _dtype_code(d):
    return DTYPES[d] if isinstance(d, str) else int(d)


def _pass_code(p):
    return PASSES[p] if isinstance(p, str) else int(p)


# ---------------------------------------------------------------- C ABI, same names


def cake_gg_strerror(code: int) -> str:
    return load_library().cake_gg_strerror(int(code)).decode()


def cake_gg_plan(pass_, E, M_max, N, K, out_dtype, deterministic, max_sms=0) -> CakeGGPlan:
    """cake_gg_plan(): returns the filled plan; raises CakeGGError on a non-zero status."""
    plan = CakeGGPlan()
    rc = load_library().cake_gg_plan(ctypes.byref(plan), _pass_code(pass_), int(E), int(M_max), int(N),
                                     int(K), _dtype_code(out_dtype), int(bool(deterministic)), int(max_sms))
    if rc != CAKE_GG_OK:
        raise CakeGGError(rc, "cake_gg_plan")
    return plan


def _call(name, plan, a, b, out, offsets, out_dtype, deterministic, workspace, workspace_bytes, stream):
    lib = load_library()
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else (
            workspace.numel() * workspace.element_size() if not isinstance(workspace, int) else plan.workspace_bytes)
    s = _stream(stream, a, b, out)
    return getattr(lib, name)(ctypes.byref(plan), _ptr(a), _ptr(b), _ptr(out), _ptr(offsets),
                              _dtype_code(out_dtype), int(bool(deterministic)), _ptr(workspace),
                              int(workspace_bytes), s)


def cake_gg_fwd(plan, X, W, Y, offsets, out_dtype, deterministic, workspace, workspace_bytes=None,
                stream=None) -> int:
    """cake_gg_fwd(): Y = X W_e^T per expert; returns the status code."""
    return _call("cake_gg_fwd", plan, X, W, Y, offsets, out_dtype, deterministic, workspace,
                 workspace_bytes, stream)


def cake_gg_dgrad(plan, G, W, dX, offsets, out_dtype, deterministic, workspace, workspace_bytes=None,
                  stream=None) -> int:
    """cake_gg_dgrad(): dX = G W_e per expert; returns the status code."""
    return _call("cake_gg_dgrad", plan, G, W, dX, offsets, out_dtype, deterministic, workspace,
                 workspace_bytes, stream)


def cake_gg_wgrad(plan, G, X, dW, offsets, out_dtype, deterministic, workspace, workspace_bytes=None,
                  stream=None) -> int:
    """cake_gg_wgrad(): dW_e = G_e^T X_e per expert; returns the status code."""
    return _call("cake_gg_wgrad", plan, G, X, dW, offsets, out_dtype, deterministic, workspace,
                 workspace_bytes, stream)


def cake_gg_wgrad_noalloc(plan, G, X, dW, offsets, out_dtype, deterministic, stream=None) -> int:
    """cake_gg_wgrad_noalloc(): the weight gradient using the library's fixed scratch.

    For callers that cannot allocate device memory (no workspace argument, no
    allocation inside the call).  Returns the status code;
    CAKE_GG_ERR_SCRATCH_LIMIT when plan.workspace_bytes exceeds
    CAKE_GG_NOALLOC_SCRATCH_BYTES.
    """
    s = _stream(stream, G, X, dW)
    return load_library().cake_gg_wgrad_noalloc(ctypes.byref(plan), _ptr(G), _ptr(X), _ptr(dW), _ptr(offsets),
                                                _dtype_code(out_dtype), int(bool(deterministic)), s)


def cake_gg_check_status(workspace, stream=None) -> int:
    """cake_gg_check_status(): synchronises the stream and returns the device status word."""
    return load_library().cake_gg_check_status(_ptr(workspace), _stream(stream, workspace))


def cake_gg_corun_spinner(ctas, ns, stream) -> int:
    """cake_gg_corun_spinner(): hold `ctas` SMs for `ns` nanoseconds on `stream` (a cudaStream_t value)."""
    return load_library().cake_gg_corun_spinner(int(ctas), int(ns), ctypes.c_void_p(int(stream)))


def cake_gg_tile_walk(plan, offsets) -> np.ndarray:
    """cake_gg_tile_walk(): the kernel's tile list for host offsets, as an int32 [count, 10] array."""
    lib = load_library()
    off = np.ascontiguousarray(offsets, dtype=np.int32)
    count = ctypes.c_int64(0)
    rc = lib.cake_gg_tile_walk(ctypes.byref(plan), off.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), 0,
                               None, ctypes.byref(count))
    if rc != CAKE_GG_OK:
        raise CakeGGError(rc, "cake_gg_tile_walk")
    out = np.zeros((count.value, 10), dtype=np.int32)
    rc = lib.cake_gg_tile_walk(ctypes.byref(plan), off.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                               count.value, out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                               ctypes.byref(count))
    if rc != CAKE_GG_OK:
        raise CakeGGError(rc, "cake_gg_tile_walk")
    return out


def cake_gg_router_plan(T, R, K, max_sms=0) -> CakeGGRouterPlan:
    """cake_gg_router_plan(): plan of the FP32 router GEMM (BF16x3 emulation); raises on error."""
    rp = CakeGGRouterPlan()
    rc = load_library().cake_gg_router_plan(ctypes.byref(rp), int(T), int(R), int(K), int(max_sms))
    if rc != CAKE_GG_OK:
        raise CakeGGError(rc, "cake_gg_router_plan")
    return rp


def cake_gg_router_fp32(rp, X, W, Y, workspace, workspace_bytes=None, stream=None) -> int:
    """cake_gg_router_fp32(): Y = X W^T by BF16x3 emulation on float32 torch tensors; returns the status."""
    s = _stream(stream, X, W, Y)
    nb = int(workspace.numel() * workspace.element_size()) if workspace_bytes is None else int(workspace_bytes)
    return load_library().cake_gg_router_fp32(ctypes.byref(rp), _ptr(X), _ptr(W), _ptr(Y), _ptr(workspace), nb, s)


def _i8_x_code(d):
    return I8_X_DTYPES[d] if isinstance(d, str) else int(d)


def _act_code(a):
    return I8_ACTS[a] if a is None or isinstance(a, str) else int(a)


def cake_gg_i8_plan(E, M_max, T, N, K, x_dtype="bf16", act=None, out_dtype="bf16", max_sms=0) -> CakeGGI8Plan:
    """cake_gg_i8_plan(): plan of an 8-bit product of M_max rows from T tokens; raises on error."""
    plan = CakeGGI8Plan()
    # the problem as int8_gemm compares it (a changed field is the library's to refuse)
    plan.problem = (int(E), int(M_max), int(T), int(N), int(K), _i8_x_code(x_dtype), _act_code(act),
                    _dtype_code(out_dtype))
    rc = load_library().cake_gg_i8_plan(ctypes.byref(plan), int(E), int(M_max), int(T), int(N), int(K),
                                        _i8_x_code(x_dtype), _act_code(act), _dtype_code(out_dtype), int(max_sms))
    if rc != CAKE_GG_OK:
        raise CakeGGError(rc, "cake_gg_i8_plan")
    return plan


def cake_gg_i8_gemm(plan, X, xs, rows, W, ws, Y, offsets, workspace, workspace_bytes=None, stream=None) -> int:
    """cake_gg_i8_gemm(): the 8-bit product; returns the status code."""
    nb = int(workspace.numel() * workspace.element_size()) if workspace_bytes is None else int(workspace_bytes)
    return load_library().cake_gg_i8_gemm(ctypes.byref(plan), _ptr(X), _ptr(xs), _ptr(rows), _ptr(W), _ptr(ws), _ptr(Y),
                                          _ptr(offsets), _ptr(workspace), nb, _stream(stream, W))


def cake_gg_i8_quant(X, x_dtype, act, T, K, Xq, xs, stream=None) -> int:
    """cake_gg_i8_quant(): rows of X to 8-bit rows and scales; returns the status code."""
    return load_library().cake_gg_i8_quant(_ptr(X), _i8_x_code(x_dtype), _act_code(act), int(T), int(K), _ptr(Xq),
                                           _ptr(xs), _stream(stream, X))


def _mx4_x_code(d):
    return MX4_X_DTYPES[d] if isinstance(d, str) else int(d)


def cake_gg_mx4_plan(E, M_max, T, N, K, x_dtype="bf16", act=None, out_dtype="bf16", max_sms=0) -> CakeGGMx4Plan:
    """cake_gg_mx4_plan(): plan of a 4-bit product of M_max rows from T tokens; raises on error."""
    plan = CakeGGMx4Plan()
    # the problem as mx4_gemm compares it (a changed field is the library's to refuse)
    plan.problem = (int(E), int(M_max), int(T), int(N), int(K), _mx4_x_code(x_dtype), _act_code(act),
                    _dtype_code(out_dtype))
    rc = load_library().cake_gg_mx4_plan(ctypes.byref(plan), int(E), int(M_max), int(T), int(N), int(K),
                                         _mx4_x_code(x_dtype), _act_code(act), _dtype_code(out_dtype), int(max_sms))
    if rc != CAKE_GG_OK:
        raise CakeGGError(rc, "cake_gg_mx4_plan")
    return plan


def cake_gg_mx4_gemm(plan, X, xs, rows, W, ws, Y, offsets, workspace, workspace_bytes=None, stream=None) -> int:
    """cake_gg_mx4_gemm(): the 4-bit product; returns the status code."""
    nb = int(workspace.numel() * workspace.element_size()) if workspace_bytes is None else int(workspace_bytes)
    return load_library().cake_gg_mx4_gemm(ctypes.byref(plan), _ptr(X), _ptr(xs), _ptr(rows), _ptr(W), _ptr(ws), _ptr(Y),
                                           _ptr(offsets), _ptr(workspace), nb, _stream(stream, W))


def cake_gg_mx4_quant(X, x_dtype, act, E, R, K, Xq, xs, stream=None) -> int:
    """cake_gg_mx4_quant(): E matrices of R rows to 4-bit codes and block scales; returns the status code."""
    return load_library().cake_gg_mx4_quant(_ptr(X), _mx4_x_code(x_dtype), _act_code(act), int(E), int(R), int(K),
                                            _ptr(Xq), _ptr(xs), _stream(stream, X))


def cake_gg_route_plan(T, E, top_k) -> CakeGGRoutePlan:
    """cake_gg_route_plan(): plan of routing T tokens to top_k of E experts each; raises on error."""
    plan = CakeGGRoutePlan()
    rc = load_library().cake_gg_route_plan(ctypes.byref(plan), int(T), int(E), int(top_k))
    if rc != CAKE_GG_OK:
        raise CakeGGError(rc, "cake_gg_route_plan")
    return plan


def cake_gg_route(plan, options, logits, logits_dtype, row_stride, bias, expert, weight, offsets, rows, position, workspace,
                  workspace_bytes=None, stream=None) -> int:
    """cake_gg_route(): experts, weights and rows of tokens by their router logits; returns the status code."""
    nb = int(workspace.numel() * workspace.element_size()) if workspace_bytes is None else int(workspace_bytes)
    return load_library().cake_gg_route(ctypes.byref(plan), ctypes.byref(options), _ptr(logits), _dtype_code(logits_dtype),
                                        int(row_stride), _ptr(bias), _ptr(expert), _ptr(weight), _ptr(offsets), _ptr(rows),
                                        _ptr(position), _ptr(workspace), nb, _stream(stream, logits))


def cake_gg_route_grad(T, E, top_k, score, renormalize, scale, logits, logits_dtype, row_stride, expert, d_weight, d_logits,
                       stream=None) -> int:
    """cake_gg_route_grad(): the logits' gradient from the weights'; returns the status code."""
    return load_library().cake_gg_route_grad(int(T), int(E), int(top_k), SCORES.get(score, score), int(bool(renormalize)),
                                             float(scale), _ptr(logits), _dtype_code(logits_dtype), int(row_stride),
                                             _ptr(expert), _ptr(d_weight), _ptr(d_logits), _stream(stream, logits))


def cake_gg_combine_rows(T, M, top_k, K, rows, rows_dtype, position, weight, out, out_dtype, stream=None) -> int:
    """cake_gg_combine_rows(): tokens as weighted sums of their rows; returns the status code."""
    return load_library().cake_gg_combine_rows(int(T), int(M), int(top_k), int(K), _ptr(rows), _dtype_code(rows_dtype),
                                               _ptr(position), _ptr(weight), _ptr(out), _dtype_code(out_dtype),
                                               _stream(stream, rows))


def cake_gg_combine_grad(T, M, top_k, K, d_out, out_dtype, rows, rows_dtype, position, weight, d_rows, d_weight,
                         stream=None) -> int:
    """cake_gg_combine_grad(): the gradients of rows and weights; returns the status code."""
    return load_library().cake_gg_combine_grad(int(T), int(M), int(top_k), int(K), _ptr(d_out), _dtype_code(out_dtype),
                                               _ptr(rows), _dtype_code(rows_dtype), _ptr(position), _ptr(weight), _ptr(d_rows),
                                               _ptr(d_weight), _stream(stream, d_out))


def cake_gg_zero_unnamed_rows(T, M, top_k, K, position, rows, rows_dtype, named, stream=None) -> int:
    """cake_gg_zero_unnamed_rows(): zeros in the rows that position does not name; returns the status code."""
    return load_library().cake_gg_zero_unnamed_rows(int(T), int(M), int(top_k), int(K), _ptr(position), _ptr(rows),
                                                    _dtype_code(rows_dtype), _ptr(named), _stream(stream, rows))


# ---------------------------------------------------------------- tensor-level helpers


def _torch_out_dtype(out_dtype):
    import torch
    return torch.float32 if _dtype_code(out_dtype) == CAKE_GG_FP32 else torch.bfloat16


def _for_stream(stream, device, make, result=False):
    """make()'s tensor as memory of `stream` (None: the current one).

    What a call on another stream than the current one writes has to come from
    that stream's memory and be filled in its order: filled on the current
    stream, a workspace could be cleared under the running product, and its
    memory would go back to a pool that does not wait for the product.  The
    caller reads a result on the current stream, so its memory waits for both.
    """
    if stream is None or device.type != "cuda":
        return make()
    handle = stream if isinstance(stream, int) else stream.cuda_stream
    if handle == _current_stream(device.index):
        return make()
    import torch
    current = torch.cuda.current_stream(device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        tensor = make()
    if result:
        tensor.record_stream(current)
    return tensor


def _result(shape, dtype, device, stream):
    """An output of a call on `stream`."""
    import torch
    return _for_stream(stream, device, lambda: torch.empty(shape, dtype=dtype, device=device), result=True)


def _scratch(plan, device, stream):
    """A workspace for one call on `stream`."""
    return _for_stream(stream, device, lambda: make_workspace(plan, device))


def make_workspace(plan, device):
    """A zero-filled workspace of plan.workspace_bytes (the library expects zeros before first use)."""
    import torch
    n = max(int(plan.workspace_bytes), 256)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def grouped_gemm(pass_, a, b, offsets, out_dtype="bf16", deterministic=True, max_sms=0, out=None,
                 plan=None, workspace=None, stream=None, check=True):
    """Run one pass on torch CUDA tensors, allocating the output and workspace through torch (for `stream`).

    fwd:   a = X [M, K], b = W [E, N, K] -> Y [M, N]
    dgrad: a = G [M, N], b = W [E, N, K] -> dX [M, K]
    wgrad: a = G [M, N], b = X [M, K], E from offsets -> dW [E, N, K]
    Rows >= offsets[E] of Y / dX are left as allocated (uninitialised).
    """
    p = _pass_code(pass_)
    E = int(offsets.numel()) - 1
    M = int(a.shape[0])
    if p == CAKE_GG_FWD:
        N, K = int(b.shape[1]), int(b.shape[2])
        shape = (M, N)
    elif p == CAKE_GG_DGRAD:
        N, K = int(b.shape[1]), int(b.shape[2])
        shape = (M, K)
    else:
        N, K = int(a.shape[1]), int(b.shape[1])
        shape = (E, N, K)
    if plan is None:
        plan = cake_gg_plan(p, E, M, N, K, out_dtype, deterministic, max_sms)
    if out is None:
        out = _result(shape, _torch_out_dtype(out_dtype), a.device, stream)
    if workspace is None:
        workspace = _scratch(plan, a.device, stream)
    fn = {CAKE_GG_FWD: cake_gg_fwd, CAKE_GG_DGRAD: cake_gg_dgrad, CAKE_GG_WGRAD: cake_gg_wgrad}[p]
    rc = fn(plan, a, b, out, offsets, out_dtype, deterministic, workspace, stream=stream)
    if rc != CAKE_GG_OK:
        raise CakeGGError(rc, f"cake_gg pass {pass_}")
    if check:
        st = cake_gg_check_status(workspace, stream)
        if st != CAKE_GG_OK:
            raise CakeGGError(st, f"cake_gg pass {pass_} (device status)")
    return out


def router_gemm(X, W, max_sms=0, out=None, plan=None, workspace=None, stream=None, check=True):
    """FP32 router logits Y [T, R] = X [T, K] W [R, K]^T by BF16x3 emulation (float32 torch tensors).

    Allocates the output and the workspace through torch (for `stream`) when not given.
    """
    import torch
    T, K = int(X.shape[0]), int(X.shape[1])
    R = int(W.shape[0])
    if plan is None:
        plan = cake_gg_router_plan(T, R, K, max_sms)
    if out is None:
        out = _result((T, R), torch.float32, X.device, stream)
    if workspace is None:
        workspace = _scratch(plan, X.device, stream)
    rc = cake_gg_router_fp32(plan, X, W, out, workspace, stream=stream)
    if rc != CAKE_GG_OK:
        raise CakeGGError(rc, "cake_gg_router_fp32")
    if check:
        st = cake_gg_check_status(workspace, stream)
        if st != CAKE_GG_OK:
            raise CakeGGError(st, "cake_gg_router_fp32 (device status)")
    return out


_i8_types = None


def _i8_torch():
    """Names of the X types, torch's int8, float32 and int32, and its output types by whether they are FP32."""
    global _i8_types
    if _i8_types is None:
        import torch
        _i8_types = ({torch.bfloat16: "bf16", torch.float32: "fp32", torch.int8: "int8"},
                     torch.int8, torch.float32, torch.int32, (torch.bfloat16, torch.float32))
    return _i8_types


def _i8_x_name(X):
    name = _i8_torch()[0].get(X.dtype)
    if name is None:
        raise TypeError(f"X is {X.dtype}: int8, bfloat16 or float32 are taken")
    return name


def _current_device():
    """The current CUDA device's index (asked only with a CUDA tensor in hand)."""
    global _current_device
    import torch
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    return _current_device()


def _refuse_device(tensor):
    """Raises: the kernels launch on the current CUDA device and take its addresses only."""
    if tensor.get_device() < 0:
        raise ValueError(f"the tensors are on {tensor.device}: CUDA tensors are needed")
    raise ValueError(f"the tensors are on {tensor.device}, the current CUDA device is {_current_device()}")


def _need(tensor, name, dtype, shape, device):
    """A dense tensor of this type and shape on `device`."""
    if tensor.dtype != dtype:
        raise TypeError(f"{name} is {tensor.dtype}: {dtype} is needed")
    if tuple(tensor.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(tensor.shape)}: {tuple(shape)} is needed")
    if tensor.device != device:
        raise ValueError(f"{name} is on {tensor.device}, not on {device}")
    if not tensor.is_contiguous():
        raise ValueError(f"{name} is not contiguous")


def quantize_rows(X, act=None, out=None, scale=None, stream=None):
    """Rows of X [T, K] (bf16 or fp32) as 8-bit integers [T, K] and FP32 scales [T].

    ``act="silu_mul"`` takes X [T, 2 K] = [g | u] and quantises silu(g) * u.
    The scale of a row is its largest magnitude / 127; integers are rounded to
    nearest, ties to even.  A row that holds a NaN or an infinity gets the scale
    NaN and zeros, one whose values are all below 2^-120 the scale 0 and zeros.
    Quantising W.reshape(E * N, K) gives int8_gemm's weights.  All tensors are on
    the current CUDA device (others are refused); stream as in int8_gemm.
    """
    import torch
    name = _i8_x_name(X)
    if act not in I8_ACTS:
        raise ValueError(f"act is None or 'silu_mul', got {act!r}")
    if X.dim() != 2 or (act is not None and X.shape[1] % 2 != 0):
        raise ValueError("X is [T, K], or [T, 2 K] with an activation")
    T, K = int(X.shape[0]), int(X.shape[1]) // (1 if act is None else 2)
    _need(X, "X", X.dtype, tuple(X.shape), X.device)
    if out is not None:
        _need(out, "out", torch.int8, (T, K), X.device)
    if scale is not None:
        _need(scale, "scale", torch.float32, (T,), X.device)
    if X.get_device() < 0 or X.get_device() != _current_device():
        _refuse_device(X)
    if out is None:
        out = _result((T, K), torch.int8, X.device, stream)
    if scale is None:
        scale = _result((T,), torch.float32, X.device, stream)
    rc = cake_gg_i8_quant(X, name, act, T, K, out, scale, stream)
    if rc != CAKE_GG_OK:
        raise CakeGGError(rc, "cake_gg_i8_quant")
    return out, scale


def int8_gemm(X, W, ws, xs=None, offsets=None, rows=None, act=None, out_dtype="bf16", max_sms=0, out=None,
              plan=None, workspace=None, stream=None, check=True):
    """Product of 8-bit rows and weights with a scale per token and per channel.

        Y[m, n] = (sum_k q[r, k] W[e, n, k]) * ws[e, n] * xs[r]

    W [E, N, K] int8 and ws [E, N] fp32 (dense: [N, K] and [N]); expert e owns
    the rows [offsets[e], offsets[e+1]) of Y (int32 [E + 1]; none for dense);
    r = rows[m] (int32 [M], the token that row m was routed from) or m itself.
    X is the tokens: int8 [T, K] with their scales xs [T], or bf16 / fp32
    [T, K] quantised on the way ([T, 2 K] with act="silu_mul", see
    quantize_rows).  Rows >= offsets[E] of Y are left as allocated.  Output and
    workspace are allocated through torch when not given, as memory of `stream`.
    All tensors are on the current CUDA device (others are refused).

    stream (a torch stream or a cudaStream_t value; none: the current stream)
    is where the kernels go.  On another stream than the current one the caller
    orders them after what wrote the inputs, and whatever reads the output, or
    writes or frees the inputs, after them.
    """
    names, i8, f32, i32, out_types = _i8_types or _i8_torch()
    name = names.get(X.dtype) or _i8_x_name(X)
    if act not in I8_ACTS:
        raise ValueError(f"act is None or 'silu_mul', got {act!r}")
    x_shape, w_shape = X.shape, W.shape
    if len(w_shape) not in (2, 3) or len(x_shape) != 2:
        raise ValueError("X is [T, K] and W [N, K] or [E, N, K]")
    E = w_shape[0] if len(w_shape) == 3 else 1
    N, K = w_shape[-2], w_shape[-1]
    T = x_shape[0]
    M = T if rows is None else rows.shape[0]
    if (xs is None) == (name == "int8"):
        raise ValueError("xs comes with int8 X, and only with it")
    if offsets is None and E != 1:
        raise ValueError("W of several experts comes with offsets")
    # the common case in few calls; what fails here is named below
    on = W.get_device()
    if not (W.dtype is i8 and W.is_contiguous() and ws.dtype is f32 and ws.shape == w_shape[:-1] and ws.is_contiguous()
            and x_shape[1] == (K if act is None else 2 * K) and X.is_contiguous() and on == X.get_device() == ws.get_device()
            and (xs is None or (xs.dtype is f32 and xs.shape == x_shape[:1] and xs.is_contiguous() and xs.get_device() == on))
            and (offsets is None or (offsets.dtype is i32 and offsets.shape == (E + 1,) and offsets.is_contiguous()
                                     and offsets.get_device() == on))
            and (rows is None or (rows.dtype is i32 and rows.dim() == 1 and rows.is_contiguous() and rows.get_device() == on))):
        device = W.device
        _need(W, "W", i8, w_shape, device)
        _need(X, "X", X.dtype, (T, K if act is None else 2 * K), device)
        _need(ws, "ws", f32, w_shape[:-1], device)
        if xs is not None:
            _need(xs, "xs", f32, (T,), device)
        if offsets is not None:
            _need(offsets, "offsets", i32, (E + 1,), device)
        if rows is not None:
            _need(rows, "rows", i32, (M,), device)
    out_code = DTYPES[out_dtype] if out_dtype.__class__ is str else int(out_dtype)
    out_type = out_types[out_code == CAKE_GG_FP32]
    if plan is None:
        plan = cake_gg_i8_plan(E, M, T, N, K, name, act, out_dtype, max_sms)
    elif getattr(plan, "problem", None) != (E, M, T, N, K, I8_X_DTYPES[name], I8_ACTS[act], out_code):
        raise ValueError("the plan is another problem's")
    if out is not None and not (out.dtype is out_type and out.shape == (M, N) and out.is_contiguous()
                                and out.get_device() == on):
        _need(out, "out", out_type, (M, N), W.device)
    if on < 0 or on != _current_device():
        _refuse_device(W)
    if out is None:
        out = _result((M, N), out_type, W.device, stream)
    if workspace is None:
        workspace = _scratch(plan, W.device, stream)
    elif workspace.get_device() != on:
        raise ValueError(f"workspace is on {workspace.device}, not on {W.device}")
    if stream is None:
        stream = _current_stream(on)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    # (the call of cake_gg_i8_gemm() above, without its conversions: a short product's
    # time is the host's)
    rc = (_lib or load_library()).cake_gg_i8_gemm(
        ctypes.byref(plan), X.data_ptr(), None if xs is None else xs.data_ptr(),
        None if rows is None else rows.data_ptr(), W.data_ptr(), ws.data_ptr(), out.data_ptr(),
        None if offsets is None else offsets.data_ptr(), workspace.data_ptr(), workspace.nbytes, stream)
    if rc != CAKE_GG_OK:
        raise CakeGGError(rc, "cake_gg_i8_gemm")
    if check:
        st = cake_gg_check_status(workspace, stream)
        if st != CAKE_GG_OK:
            raise CakeGGError(st, "cake_gg_i8_gemm (device status)")
    return out


def _mx4_tiles(R, K):
    """Shape of the scale tiles of a matrix of R rows of K values."""
    return (-(-R // 128), -(-K // 128), 32, 4, 4)


def quantize_mx4(X, act=None, out=None, scale=None, stream=None):
    """X [T, K] or [E, R, K] (bf16 or fp32) as 4-bit codes [.., K / 2] and block scales (both uint8).

    A block of 32 values along K shares a power of two; the codes are E2M1,
    two to a byte, the even one low, and the scales E8M0 in tiles of 128 rows x 4 blocks:
    [ceil(T / 128), ceil(K / 128), 32, 4, 4], or [E, ceil(R / 128), ..] with a
    tile grid for each of E matrices, which are mx4_gemm's tokens and weights
    (mx4_values() says what they stand for).  ``act="silu_mul"`` takes rows
    [g | u] of 2 K values and quantises silu(g) * u.  A block that holds a NaN or
    an infinity becomes NaN.  K is a multiple of 32.  In a `scale` that is given,
    rows past the last of a tile stay as they were.  All tensors are on the
    current CUDA device (others are refused); stream as in int8_gemm.
    """
    import torch
    name = {torch.bfloat16: "bf16", torch.float32: "fp32"}.get(X.dtype)
    if name is None:
        raise TypeError(f"X is {X.dtype}: bfloat16 or float32 are taken")
    if act not in I8_ACTS:
        raise ValueError(f"act is None or 'silu_mul', got {act!r}")
    if X.dim() not in (2, 3) or (act is not None and X.shape[-1] % 2 != 0):
        raise ValueError("X is [T, K] or [E, R, K], or twice as wide with an activation")
    E = int(X.shape[0]) if X.dim() == 3 else 1
    R, K = int(X.shape[-2]), int(X.shape[-1]) // (1 if act is None else 2)
    lead = (E,) if X.dim() == 3 else ()
    _need(X, "X", X.dtype, tuple(X.shape), X.device)
    if out is not None:
        _need(out, "out", torch.uint8, lead + (R, K // 2), X.device)
    if scale is not None:
        _need(scale, "scale", torch.uint8, lead + _mx4_tiles(R, K), X.device)
    if X.get_device() < 0 or X.get_device() != _current_device():
        _refuse_device(X)
    if out is None:
        out = _result(lead + (R, K // 2), torch.uint8, X.device, stream)
    if scale is None:
        scale = _for_stream(stream, X.device, lambda: torch.zeros(lead + _mx4_tiles(R, K), dtype=torch.uint8, device=X.device),
                            result=True)
    rc = cake_gg_mx4_quant(X, name, act, E, R, K, out, scale, stream)
    if rc != CAKE_GG_OK:
        raise CakeGGError(rc, "cake_gg_mx4_quant")
    return out, scale


def mx4_values(q, scale):
    """The FP32 numbers [.., K] that 4-bit codes [.., K / 2] and their scale tiles stand for (torch operations, any device)."""
    import torch
    R, K = int(q.shape[-2]), 2 * int(q.shape[-1])
    sizes = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
    codes = torch.stack([q & 15, q >> 4], dim=-1).reshape(*q.shape[:-1], K).long()
    v = torch.where(codes < 8, sizes[codes & 7], -sizes[codes & 7])
    s = scale.transpose(-4, -2)                         # [.., tile, r % 128 / 32, r % 32, K / 128, block]
    s = s.reshape(*scale.shape[:-5], scale.shape[-5] * 128, scale.shape[-4] * 4)[..., :R, :K // 32].to(torch.int32)
    # the power of two by its bits: 2^-127 is below the normal range
    power = torch.where(s == 0, torch.full_like(s, 1 << 22), s << 23).view(torch.float32)
    power = torch.where(s == 255, torch.full_like(power, float("nan")), power)
    return v * power.repeat_interleave(32, dim=-1)


_mx4_types = None


def _mx4_torch():
    """Names of the X types, torch's uint8 and int32, and its output types by whether they are FP32."""
    global _mx4_types
    if _mx4_types is None:
        import torch
        _mx4_types = ({torch.bfloat16: "bf16", torch.float32: "fp32", torch.uint8: "mx4"}, torch.uint8, torch.int32,
                      (torch.bfloat16, torch.float32))
    return _mx4_types


def mx4_gemm(X, W, ws, xs=None, offsets=None, rows=None, act=None, out_dtype="bf16", max_sms=0, out=None,
             plan=None, workspace=None, stream=None, check=True):
    """Product of 4-bit rows and weights with a power of two for each block of 32 values.

        Y[m, n] = sum_k x[r, k] w[e, n, k]

    W [E, N, K / 2] uint8 and its scale tiles ws (dense: [N, K / 2]) are
    quantize_mx4's; expert e owns the rows [offsets[e], offsets[e+1]) of Y
    (int32 [E + 1]; none for dense); r = rows[m] (int32 [M], the token that row m
    was routed from) or m itself.  X is the tokens: uint8 [T, K / 2] with their
    scale tiles xs, or bf16 / fp32 [T, K] quantised on the way ([T, 2 K] with
    act="silu_mul", see quantize_mx4).  Rows >= offsets[E] of Y are left as
    allocated.  Output, workspace, devices, `stream` and `check` as in int8_gemm.
    """
    names, u8, i32, out_types = _mx4_types or _mx4_torch()
    name = names.get(X.dtype)
    if name is None:
        raise TypeError(f"X is {X.dtype}: uint8, bfloat16 or float32 are taken")
    if act not in I8_ACTS:
        raise ValueError(f"act is None or 'silu_mul', got {act!r}")
    x_shape, w_shape = X.shape, W.shape
    if len(w_shape) not in (2, 3) or len(x_shape) != 2:
        raise ValueError("X is [T, K] and W [N, K / 2] or [E, N, K / 2]")
    E = w_shape[0] if len(w_shape) == 3 else 1
    N, K = w_shape[-2], 2 * w_shape[-1]
    T = x_shape[0]
    M = T if rows is None else rows.shape[0]
    if (xs is None) == (name == "mx4"):
        raise ValueError("xs comes with 4-bit X, and only with it")
    if offsets is None and E != 1:
        raise ValueError("W of several experts comes with offsets")
    width = K // 2 if name == "mx4" else K if act is None else 2 * K
    tiles = w_shape[:-2] + _mx4_tiles(N, K)
    # the common case in few calls; what fails here is named below
    on = W.get_device()
    if not (W.dtype is u8 and W.is_contiguous() and ws.dtype is u8 and ws.shape == tiles and ws.is_contiguous()
            and x_shape[1] == width and X.is_contiguous() and on == X.get_device() == ws.get_device()
            and (xs is None or (xs.dtype is u8 and xs.shape == _mx4_tiles(T, K) and xs.is_contiguous() and xs.get_device() == on))
            and (offsets is None or (offsets.dtype is i32 and offsets.shape == (E + 1,) and offsets.is_contiguous()
                                     and offsets.get_device() == on))
            and (rows is None or (rows.dtype is i32 and rows.dim() == 1 and rows.is_contiguous() and rows.get_device() == on))):
        device = W.device
        _need(W, "W", u8, w_shape, device)
        _need(X, "X", X.dtype, (T, width), device)
        _need(ws, "ws", u8, tiles, device)
        if xs is not None:
            _need(xs, "xs", u8, _mx4_tiles(T, K), device)
        if offsets is not None:
            _need(offsets, "offsets", i32, (E + 1,), device)
        if rows is not None:
            _need(rows, "rows", i32, (M,), device)
    out_code = DTYPES[out_dtype] if out_dtype.__class__ is str else int(out_dtype)
    out_type = out_types[out_code == CAKE_GG_FP32]
    if plan is None:
        plan = cake_gg_mx4_plan(E, M, T, N, K, name, act, out_dtype, max_sms)
    elif getattr(plan, "problem", None) != (E, M, T, N, K, MX4_X_DTYPES[name], I8_ACTS[act], out_code):
        raise ValueError("the plan is another problem's")
    if out is not None and not (out.dtype is out_type and out.shape == (M, N) and out.is_contiguous()
                                and out.get_device() == on):
        _need(out, "out", out_type, (M, N), W.device)
    if on < 0 or on != _current_device():
        _refuse_device(W)
    if out is None:
        out = _result((M, N), out_type, W.device, stream)
    if workspace is None:
        workspace = _scratch(plan, W.device, stream)
    elif workspace.get_device() != on:
        raise ValueError(f"workspace is on {workspace.device}, not on {W.device}")
    if stream is None:
        stream = _current_stream(on)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    # (the call of cake_gg_mx4_gemm() above, without its conversions)
    rc = (_lib or load_library()).cake_gg_mx4_gemm(
        ctypes.byref(plan), X.data_ptr(), None if xs is None else xs.data_ptr(),
        None if rows is None else rows.data_ptr(), W.data_ptr(), ws.data_ptr(), out.data_ptr(),
        None if offsets is None else offsets.data_ptr(), workspace.data_ptr(), workspace.nbytes, stream)
    if rc != CAKE_GG_OK:
        raise CakeGGError(rc, "cake_gg_mx4_gemm")
    if check:
        st = cake_gg_check_status(workspace, stream)
        if st != CAKE_GG_OK:
            raise CakeGGError(st, "cake_gg_mx4_gemm (device status)")
    return out


class Routing(typing.NamedTuple):
    """Where T tokens go, each to top_k of E experts (what route() gives)."""
    expert: typing.Any      # int32 [T, top_k]: experts, the best first
    weight: typing.Any      # float32 [T, top_k]
    offsets: typing.Any     # int32 [E + 1]: expert e's rows are [offsets[e], offsets[e + 1])
    rows: typing.Any        # int32 [T * top_k]: the token of each row
    position: typing.Any    # int32 [T, top_k]: the row of each token's j-th expert


def empty_routing(T, E, top_k, device) -> Routing:
    """An uninitialised Routing, for route()'s `out`."""
    import torch
    def i32(*shape):
        return torch.empty(shape, dtype=torch.int32, device=device)
    return Routing(i32(T, top_k), torch.empty((T, top_k), dtype=torch.float32, device=device), i32(E + 1), i32(T * top_k),
                   i32(T, top_k))


_real_types = None


def _real_torch():
    """Names of the real types, torch's float32 and int32."""
    global _real_types
    if _real_types is None:
        import torch
        _real_types = {torch.bfloat16: "bf16", torch.float32: "fp32"}, torch.float32, torch.int32
    return _real_types


def _real_name(tensor, name):
    """ "bf16" or "fp32"."""
    kind = _real_torch()[0].get(tensor.dtype)
    if kind is None:
        raise TypeError(f"{name} is {tensor.dtype}: bfloat16 or float32 are taken")
    return kind


def _logits(logits):
    """The type of router logits [T, E] whose rows are dense (they may lie apart), T, E and how far apart."""
    kind = _real_name(logits, "logits")
    shape = logits.shape
    if len(shape) != 2:
        raise ValueError("logits are [T, E]")
    T, E = shape
    apart, step = logits.stride()
    if (E > 1 and step != 1) or (T > 1 and apart < E):
        raise ValueError("the rows of logits are not dense")
    return kind, T, E, apart if T > 1 else E


def _is(tensor, dtype, shape, on):
    """Whether this is a dense tensor of this type and shape on CUDA device `on` (_need() says what is not)."""
    return tensor.dtype is dtype and tensor.shape == shape and tensor.get_device() == on and tensor.is_contiguous()


def _here(tensor):
    """The index of a tensor's device, which has to be the current one."""
    on = tensor.get_device()
    if on < 0 or on != _current_device():
        _refuse_device(tensor)
    return on


def _handle(stream, on):
    """A stream's handle (none: the current one's)."""
    if stream is None:
        return _current_stream(on)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _score_code(score):
    if score not in SCORES:
        raise ValueError(f"score is 'softmax' or 'sigmoid', got {score!r}")
    return SCORES[score]


@functools.lru_cache(maxsize=64)
def _route_options(score, groups, top_groups, group_score, renormalize, scale):
    if group_score not in GROUP_SCORES:
        raise ValueError(f"group_score is 'max' or 'top2', got {group_score!r}")
    return CakeGGRouteOptions(_score_code(score), groups, groups if top_groups is None else top_groups,
                              GROUP_SCORES[group_score], int(renormalize), float.fromhex(scale))


def route(logits, top_k, score="softmax", bias=None, groups=1, top_groups=None, group_score="max", renormalize=True,
          scale=1.0, plan=None, workspace=None, out=None, stream=None) -> Routing:
    """Routes T tokens by their router logits [T, E] (bf16 or fp32; rows may lie apart, as in a slice of columns).

    Scores are the softmax of a token's logits or their sigmoid; its experts are
    the top_k largest by score + bias (float32 [E]; none: by the logits), ties to
    the lowest index, a NaN last; with groups > 1 only from the `top_groups` (none:
    all) of the E / groups neighbouring experts that have the largest group_score: "max", the
    largest of the group, or "top2", the sum of its two largest.  The choice is
    that of 64-bit scores.  Weights are the chosen experts' scores, without the
    bias, divided by their sum with `renormalize`, times `scale`.  Rows are numbered
    by expert, then by token: offsets and rows are what int8_gemm, mx4_gemm and
    grouped_gemm take, position leads back (combine_rows).  In a loop, make the plan
    (cake_gg_route_plan), the workspace and the outputs (empty_routing) once.  All
    tensors are on the current CUDA device; stream as in int8_gemm.
    """
    kind, T, E, apart = _logits(logits)
    # (plain values: a tensor's may change, and it is its identity that a cache sees, to which -0.0 is 0.0)
    options = _route_options(score, int(groups), None if top_groups is None else int(top_groups), group_score, bool(renormalize),
                             float(scale).hex())
    if plan is None:
        plan = cake_gg_route_plan(T, E, top_k)
    elif (plan.T, plan.E, plan.top_k) != (T, E, top_k):
        raise ValueError("the plan is another problem's")
    _, f32, i32 = _real_types
    on, many = logits.get_device(), (T, top_k)
    if bias is not None and not _is(bias, f32, (E,), on):
        _need(bias, "bias", f32, (E,), logits.device)
    if out is not None:
        expert, weight, offsets, rows, position = out
        if not (_is(expert, i32, many, on) and _is(weight, f32, many, on) and _is(offsets, i32, (E + 1,), on)
                and _is(rows, i32, (T * top_k,), on) and _is(position, i32, many, on)):
            for tensor, name, dtype, shape in zip(out, Routing._fields, (i32, f32, i32, i32, i32),
                                                  (many, many, (E + 1,), (T * top_k,), many)):
                _need(tensor, name, dtype, shape, logits.device)
    _here(logits)
    if out is None:
        out = Routing(*(_result(shape, dtype, logits.device, stream) for shape, dtype in
                        ((many, i32), (many, f32), ((E + 1,), i32), ((T * top_k,), i32), (many, i32))))
        expert, weight, offsets, rows, position = out
    if workspace is None:
        workspace = _scratch(plan, logits.device, stream)
    elif workspace.get_device() != on:
        raise ValueError(f"workspace is on {workspace.device}, not on {logits.device}")
    # (the call of cake_gg_route() above, without its conversions: a few tokens' time is the host's)
    rc = (_lib or load_library()).cake_gg_route(
        ctypes.byref(plan), ctypes.byref(options), logits.data_ptr(), DTYPES[kind], apart,
        None if bias is None else bias.data_ptr(), expert.data_ptr(), weight.data_ptr(), offsets.data_ptr(), rows.data_ptr(),
        position.data_ptr(), workspace.data_ptr(), workspace.nbytes, _handle(stream, on))
    if rc != CAKE_GG_OK:
        raise CakeGGError(rc, "cake_gg_route")
    return out


def route_grad(logits, expert, d_weight, score="softmax", renormalize=True, scale=1.0, out=None, stream=None):
    """The gradient [T, E] of route()'s logits, in their type, from that of its weights (float32 [T, top_k]).

    expert, score, renormalize and scale are route()'s.  The choice of experts and
    the bias have no gradient.  All tensors are on the current CUDA device.
    """
    kind, T, E, apart = _logits(logits)
    code = _score_code(score)
    if expert.dim() != 2:
        raise ValueError("expert is [T, top_k]")
    _, f32, i32 = _real_types
    on, top_k = logits.get_device(), expert.shape[1]
    if not (_is(expert, i32, (T, top_k), on) and _is(d_weight, f32, (T, top_k), on)):
        _need(expert, "expert", i32, (T, top_k), logits.device)
        _need(d_weight, "d_weight", f32, (T, top_k), logits.device)
    if out is not None and not _is(out, logits.dtype, (T, E), on):
        _need(out, "out", logits.dtype, (T, E), logits.device)
    _here(logits)
    if out is None:
        out = _result((T, E), logits.dtype, logits.device, stream)
    rc = (_lib or load_library()).cake_gg_route_grad(T, E, top_k, code, bool(renormalize), scale, logits.data_ptr(), DTYPES[kind],
                                                     apart, expert.data_ptr(), d_weight.data_ptr(), out.data_ptr(),
                                                     _handle(stream, on))
    if rc != CAKE_GG_OK:
        raise CakeGGError(rc, "cake_gg_route_grad")
    return out


def _need_position(position, weight, like, on):
    """T and top_k of int32 [T, top_k] positions and their float32 weights, on the device of `like`."""
    _, f32, i32 = _real_types
    shape = position.shape
    if len(shape) != 2:
        raise ValueError("position is [T, top_k]")
    if not (_is(position, i32, shape, on) and (weight is None or _is(weight, f32, shape, on))):
        _need(position, "position", i32, tuple(shape), like.device)
        if weight is not None:
            _need(weight, "weight", f32, tuple(shape), like.device)
    return shape


def combine_rows(rows, position, weight=None, out_dtype="bf16", out=None, stream=None):
    """Tokens [T, K] as sums of their rows: out[t] = sum_j weight[t, j] * rows[position[t, j]].

    rows [M, K] are bf16 or fp32, position int32 [T, top_k] (a Routing's; outside
    [0, M): no row), weight float32 [T, top_k] (none: ones); K is a multiple of 8.
    FP32 sums over j in order, rounded once.  All tensors are on the current CUDA device; stream as in
    int8_gemm.
    """
    kind = _real_name(rows, "rows")
    if rows.dim() != 2:
        raise ValueError("rows are [M, K]")
    (M, K), on = rows.shape, rows.get_device()
    if not rows.is_contiguous():
        raise ValueError("rows is not contiguous")
    T, top_k = _need_position(position, weight, rows, on)
    code = _dtype_code(out_dtype)
    out_type = (_i8_types or _i8_torch())[4][code == CAKE_GG_FP32]
    if out is not None and not _is(out, out_type, (T, K), on):
        _need(out, "out", out_type, (T, K), rows.device)
    _here(rows)
    if out is None:
        out = _result((T, K), out_type, rows.device, stream)
    rc = (_lib or load_library()).cake_gg_combine_rows(T, M, top_k, K, rows.data_ptr(), DTYPES[kind], position.data_ptr(),
                                                       None if weight is None else weight.data_ptr(), out.data_ptr(), code,
                                                       _handle(stream, on))
    if rc != CAKE_GG_OK:
        raise CakeGGError(rc, "cake_gg_combine_rows")
    return out


def _zero_rest(rows, position, stream):
    """Zeros in the rows that position does not name."""
    import torch
    (T, top_k), (M, K) = position.shape, rows.shape
    named = _result((M,), torch.uint8, rows.device, stream)
    rc = cake_gg_zero_unnamed_rows(T, M, top_k, K, position, rows, _real_name(rows, "rows"), named, stream)
    if rc != CAKE_GG_OK:
        raise CakeGGError(rc, "cake_gg_zero_unnamed_rows")


def combine_grad(d_out, rows, position, weight, out=None, stream=None, zero_rest=False):
    """Gradients of combine_rows: (d_rows [M, K] in the rows' type, d_weight float32 [T, top_k]), from d_out [T, K].

    position names each of the M = T * top_k rows once, as a Routing's does (rows
    of another number are refused; rows that it does not name keep what `out`, or
    fresh memory, holds, or with zero_rest become zeros).
    """
    kind, out_kind = _real_name(rows, "rows"), _real_name(d_out, "d_out")
    if rows.dim() != 2 or d_out.dim() != 2:
        raise ValueError("rows are [M, K], d_out is [T, K]")
    if weight is None:
        raise ValueError("without weights the rows' gradient is gather_rows(d_out, position)")
    (M, K), on = rows.shape, rows.get_device()
    if not rows.is_contiguous():
        raise ValueError("rows is not contiguous")
    T, top_k = _need_position(position, weight, rows, on)
    if not _is(d_out, d_out.dtype, (T, K), on):
        _need(d_out, "d_out", d_out.dtype, (T, K), rows.device)
    if M != T * top_k:
        raise ValueError(f"{M} rows for {T} x {top_k} positions")
    if out is not None and not _is(out, rows.dtype, (M, K), on):
        _need(out, "out", rows.dtype, (M, K), rows.device)
    _here(rows)
    if out is None:
        out = _result((M, K), rows.dtype, rows.device, stream)
    d_weight = _result((T, top_k), weight.dtype, rows.device, stream)
    rc = (_lib or load_library()).cake_gg_combine_grad(T, M, top_k, K, d_out.data_ptr(), DTYPES[out_kind], rows.data_ptr(),
                                                       DTYPES[kind], position.data_ptr(), weight.data_ptr(), out.data_ptr(),
                                                       d_weight.data_ptr(), _handle(stream, on))
    if rc != CAKE_GG_OK:
        raise CakeGGError(rc, "cake_gg_combine_grad")
    if zero_rest:
        _zero_rest(out, position, stream)
    return out, d_weight


def gather_rows(X, position, out=None, stream=None, weight=None, out_dtype=None, zero_rest=False):
    """Tokens X [T, K] (bf16 or fp32) as rows in expert order [T * top_k, K]: out[position[t, j]] = X[t].

    position names each row once, as a Routing's does (rows that it does not name keep what
    `out`, or fresh memory, holds, or with zero_rest become zeros); K is a multiple of 8.  With
    weight (float32 [T, top_k]) a row is weight[t, j] X[t], an FP32 product;
    out_dtype is "bf16" or "fp32" (none: X's type).  This is combine_grad's d_rows
    without the rows.
    """
    kind = _real_name(X, "X")
    if X.dim() != 2:
        raise ValueError("X is [T, K]")
    (tokens, K), on = X.shape, X.get_device()
    if not X.is_contiguous():
        raise ValueError("X is not contiguous")
    T, top_k = _need_position(position, weight, X, on)
    if tokens != T:
        raise ValueError(f"{tokens} tokens for {T} positions")
    M = T * top_k
    code = DTYPES[kind] if out_dtype is None else _dtype_code(out_dtype)
    out_type = (_i8_types or _i8_torch())[4][code == CAKE_GG_FP32]
    if out is not None and not _is(out, out_type, (M, K), on):
        _need(out, "out", out_type, (M, K), X.device)
    _here(X)
    if out is None:
        out = _result((M, K), out_type, X.device, stream)
    rc = (_lib or load_library()).cake_gg_combine_grad(T, M, top_k, K, X.data_ptr(), DTYPES[kind], None, code, position.data_ptr(),
                                                       None if weight is None else weight.data_ptr(), out.data_ptr(), None,
                                                       _handle(stream, on))
    if rc != CAKE_GG_OK:
        raise CakeGGError(rc, "cake_gg_combine_grad")
    if zero_rest:
        _zero_rest(out, position, stream)
    return out
