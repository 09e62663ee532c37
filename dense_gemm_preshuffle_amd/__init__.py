"""Python binding of the gfx950 preshuffle GEMM library (libgemm_preshuffle.so).

Argument marshalling only: every step of the GEMM runs in the library's HIP
kernels. PyTorch supplies device memory and the current stream. The entry
points have the names of the C ABI (include/gemm_preshuffle.h):

    gemm_preshuffle_b(b, dtype)                      -> preshuffled B (uint8, flat)
    gemm_a8w8(a, b_shuf, scale_a, scale_b, ...)      -> C int32 (INT8) or bf16 (FP8)
    gemm_bf16(a, b_shuf, ...)                        -> C bf16
    gemm_mxfp4(a, scale_a, b_shuf, scale_b, ...)     -> C bf16
    gemm_f16(a, b_shuf, ...)                         -> C fp16
    gemm_w4a8(a, b_shuf, scale_a, scale_b, ...)      -> C bf16 (int8 A, INT4 B)
    gemm_ex(dtype, a, b_shuf, ..., bias, act)        -> any type with the fused
                                                        bias / activation epilogue
    gemm_plan(dtype, M, N, K, opts)                  -> dict (host-only planner query)
    gemm_ex_ws(dtype, ..., workspace=ws)             -> gemm_ex with a device workspace, which
                                                        lets the planner split K across workgroups
    gemm_workspace_size(dtype, M, N, K, opts)        -> bytes gemm_ex_ws needs (0: none)
    gemm_plan_ws(dtype, M, N, K, opts)               -> dict, the plan of gemm_ex_ws
    workspace(dtype, M, N, K, opts)                  -> a zeroed device workspace of that size
    gemm_ex_noalloc(dtype, ...)                      -> gemm_ex_ws on the library's own static
                                                        device workspace (allocates nothing)
    gemm_gated_preshuffle(w, dtype)                  -> gate / up weights [2F, H] laid out for gemm_gated
    gemm_gated(dtype, x, w_shuf, act, save)          -> h = act(x Wg^T) * (x Wu^T) (and gate, up to keep)
    gemm_gated_backward(dtype, dh, gate, up, x, w)   -> dx, dw
    gemm_backward(dtype, dc, a, b)                   -> da, db of C = A B^T
    gated_workspace, gated_backward_workspace, backward_workspace
                                                     -> device workspaces of these
    gemm_w4a16_preshuffle(q, scales, zeros, group)   -> W4Weights, 4-bit weights laid out with their scales
    gemm_w4a16(x, weights, bias, act)                -> act(x W^T + bias) (BF16 / FP16 activations)
    gemm_w4a16_gated(x, weights, act)                -> act(x Wg^T) * (x Wu^T) on 4-bit weights
    w4a16_workspace(M, weights)                      -> a device workspace of these (None: none needed)
    gemm_gated_plan, gemm_w4a16_plan                 -> dict, the kernel they run (host-only)
    gemm_backward_plan                               -> two of them, or None (host-only)

Tensors: A is [M, K] (INT8 / FP8 as any 1-byte dtype, BF16 / FP16 as
bfloat16 / float16 or a 2-byte integer view, MXFP4 as uint8 [M, K/2]; W4A8:
int8 [M, K]); B before the shuffle is [N, K] the same way (W4A8: packed INT4
uint8 [N, K/2]). If the library has not been built the first call raises
GemmLibraryMissing: there is no fallback of any kind.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import re

__all__ = [
    "GemmError", "GemmLibraryMissing", "GemmOpts", "lib_path", "load_library",
    "gemm_preshuffle_b", "gemm_a8w8", "gemm_bf16", "gemm_mxfp4", "gemm_f16", "gemm_w4a8", "gemm_ex",
    "gemm_plan", "ACTS", "gemm_ex_ws", "gemm_ex_noalloc", "gemm_workspace_size", "gemm_plan_ws", "workspace",
    "gemm_gated_preshuffle", "gemm_gated", "gemm_gated_workspace_size", "gated_workspace", "gemm_gated_backward",
    "gemm_gated_backward_workspace_size", "gated_backward_workspace", "gemm_backward", "gemm_backward_workspace_size",
    "backward_workspace", "W4Weights", "gemm_w4a16_weights_size", "gemm_w4a16_preshuffle", "gemm_w4a16",
    "gemm_w4a16_gated", "gemm_w4a16_workspace_size", "w4a16_workspace", "gemm_gated_plan", "gemm_w4a16_plan",
    "gemm_backward_plan", "gemm_status_string", "source_hash", "DTYPES", "EPI_DIRECT", "EPI_CSHUFFLE", "KERNEL_TILE",
    "KERNEL_SPLITK", "KERNEL_WIDE", "KERNEL_ROWS", "KERNEL_PAIR",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libgemm_preshuffle.so"

# gp_dtype values of the C ABI
GP_I8, GP_FP8_E4M3, GP_BF16, GP_FP4_E2M1, GP_I32, GP_F16, GP_I4 = 0, 1, 2, 3, 4, 5, 6
DTYPES = {"int8": GP_I8, "fp8": GP_FP8_E4M3, "bf16": GP_BF16, "mxfp4": GP_FP4_E2M1,
          "fp16": GP_F16, "w4a8": GP_I4}
_ELEM_BITS = {GP_I8: 8, GP_FP8_E4M3: 8, GP_BF16: 16, GP_FP4_E2M1: 4, GP_F16: 16, GP_I4: 4}   # of B
_OUT = {GP_I8: GP_I32, GP_FP8_E4M3: GP_BF16, GP_BF16: GP_BF16, GP_FP4_E2M1: GP_BF16, GP_F16: GP_F16,
        GP_I4: GP_BF16}
# gp_status values of a HIP runtime or launch error, and of a missing / too small workspace
GP_EHIP = 5
GP_EDTYPE = 3
GP_EWORKSPACE = 6
# gp_act values of the C ABI
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}
EPI_AUTO, EPI_DIRECT, EPI_CSHUFFLE = 0, 1, 2
KERNEL_AUTO, KERNEL_TILE, KERNEL_SPLITK, KERNEL_WIDE, KERNEL_ROWS, KERNEL_PAIR = 0, 1, 2, 3, 4, 5


class GemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: status {status} ({gemm_status_string(status)})"
        if status == GP_EHIP and _lib is not None:
            msg += f" [{_lib.gemm_last_hip_error().decode()} from {_lib.gemm_last_hip_call().decode()}]"
        super().__init__(msg)


class GemmLibraryMissing(ImportError):
    pass


class GemmOpts(ctypes.Structure):
    _fields_ = [("tile_m", ctypes.c_int), ("tile_n", ctypes.c_int), ("tile_k", ctypes.c_int),
                ("epilogue", ctypes.c_int), ("kernel", ctypes.c_int), ("xcd_swizzle", ctypes.c_int),
                ("waves", ctypes.c_int), ("mfma", ctypes.c_int), ("pipeline", ctypes.c_int),
                ("ksplit", ctypes.c_int), ("scheduler", ctypes.c_int)]


class GemmPlanInfo(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("tile_m", ctypes.c_int), ("tile_n", ctypes.c_int),
                ("tile_k", ctypes.c_int), ("epilogue", ctypes.c_int), ("xcd_swizzle", ctypes.c_int),
                ("waves", ctypes.c_int), ("threads", ctypes.c_int), ("lds_bytes", ctypes.c_int),
                ("grid", ctypes.c_int64), ("k_tiles", ctypes.c_int64),
                ("mfma_per_wave_tile", ctypes.c_int64), ("mfma_total", ctypes.c_int64),
                ("mfma", ctypes.c_int), ("pipeline", ctypes.c_int), ("ksplit", ctypes.c_int),
                ("scheduler", ctypes.c_int), ("workspace_bytes", ctypes.c_int64)]


_lib = None


def lib_path() -> str:
    return os.environ.get("GEMM_PRESHUFFLE_LIB", os.path.join(_PKG, _LIB_NAME))


def load_library():
    """Load (once) and return the ctypes handle of the HIP library."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise GemmLibraryMissing(
            f"{path} is not built; run `python -m dense_gemm_preshuffle_amd.build` "
            "(or __graft_entry__.build()) first")
    # PyTorch ships its own HIP and HSA runtimes under the sonames of ROCm's
    # (libamdhip64.so.7, libhsa-runtime64.so.1). Loaded after torch, this
    # library binds to those copies: one runtime per process. Loaded before
    # torch, it would bind to /opt/rocm's copies and torch would then load
    # its own: two runtimes, and the second to start finds no device
    # (hipGetDevice: hipErrorNoDevice). So torch is imported first.
    import torch  # noqa: F401

    lib = ctypes.CDLL(path)
    vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.gemm_preshuffle_b.argtypes = [vp, vp, i64, i64, ci, vp]
    lib.gemm_a8w8.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ci, ci, ctypes.POINTER(GemmOpts), vp]
    lib.gemm_bf16.argtypes = [vp, vp, vp, i64, i64, i64, ctypes.POINTER(GemmOpts), vp]
    lib.gemm_mxfp4.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ctypes.POINTER(GemmOpts), vp]
    lib.gemm_f16.argtypes = [vp, vp, vp, i64, i64, i64, ctypes.POINTER(GemmOpts), vp]
    lib.gemm_w4a8.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, ctypes.POINTER(GemmOpts), vp]
    lib.gemm_ex.argtypes = [ci, ci, vp, vp, vp, vp, vp, ci, vp, i64, i64, i64, ctypes.POINTER(GemmOpts), vp]
    lib.gemm_plan.argtypes = [ci, i64, i64, i64, ctypes.POINTER(GemmOpts), ctypes.POINTER(GemmPlanInfo)]
    lib.gemm_plan_ws.argtypes = [ci, i64, i64, i64, ctypes.POINTER(GemmOpts), ctypes.POINTER(GemmPlanInfo)]
    lib.gemm_workspace_size.argtypes = [ci, i64, i64, i64, ctypes.POINTER(GemmOpts), ctypes.POINTER(ctypes.c_size_t)]
    lib.gemm_ex_ws.argtypes = [ci, ci, vp, vp, vp, vp, vp, ci, vp, i64, i64, i64, ctypes.POINTER(GemmOpts), vp,
                               ctypes.c_size_t, vp]
    lib.gemm_ex_noalloc.argtypes = [ci, ci, vp, vp, vp, vp, vp, ci, vp, i64, i64, i64, ctypes.POINTER(GemmOpts), vp]
    sz, psz = ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)
    lib.gemm_gated_preshuffle.argtypes = [vp, vp, i64, i64, ci, vp]
    lib.gemm_gated.argtypes = [ci, vp, vp, ci, vp, vp, vp, i64, i64, i64, vp, sz, vp]
    lib.gemm_gated_workspace_size.argtypes = [ci, i64, i64, i64, psz]
    lib.gemm_gated_backward.argtypes = [ci, vp, vp, vp, vp, vp, ci, vp, vp, i64, i64, i64, vp, sz, vp]
    lib.gemm_gated_backward_workspace_size.argtypes = [ci, i64, i64, i64, ci, ci, psz]
    lib.gemm_backward.argtypes = [ci, vp, vp, vp, vp, vp, i64, i64, i64, vp, sz, vp]
    lib.gemm_backward_workspace_size.argtypes = [ci, i64, i64, i64, ci, ci, psz]
    lib.gemm_w4a16_weights_size.argtypes = [i64, i64, ci, ci, ci, psz]
    lib.gemm_w4a16_preshuffle.argtypes = [ci, vp, vp, vp, vp, i64, i64, ci, ci, vp]
    lib.gemm_w4a16.argtypes = [ci, vp, vp, ci, vp, ci, vp, i64, i64, i64, ci, vp]
    lib.gemm_w4a16_gated.argtypes = [ci, vp, vp, ci, ci, vp, i64, i64, i64, ci, vp]
    lib.gemm_w4a16_workspace_size.argtypes = [i64, i64, i64, ci, ci, psz]
    lib.gemm_backward_plan.argtypes = [ci, i64, i64, i64, ci, ci, ci, ctypes.POINTER(GemmPlanInfo),
                                       ctypes.POINTER(GemmPlanInfo)]
    lib.gemm_gated_plan.argtypes = [ci, i64, i64, i64, ctypes.POINTER(GemmPlanInfo)]
    lib.gemm_w4a16_plan.argtypes = [i64, i64, i64, ci, ci, ci, ctypes.POINTER(GemmPlanInfo)]
    lib.gemm_w4a16_ws.argtypes = [ci, vp, vp, ci, vp, ci, vp, i64, i64, i64, ci, ci, vp, sz, vp]
    lib.gemm_status_string.argtypes = [ci]
    lib.gemm_status_string.restype = ctypes.c_char_p
    lib.gemm_last_hip_error.argtypes = []
    lib.gemm_last_hip_error.restype = ctypes.c_char_p
    lib.gemm_last_hip_call.argtypes = []
    lib.gemm_last_hip_call.restype = ctypes.c_char_p
    for f in ("gemm_preshuffle_b", "gemm_a8w8", "gemm_bf16", "gemm_mxfp4", "gemm_f16", "gemm_w4a8", "gemm_ex",
              "gemm_plan", "gemm_plan_ws", "gemm_workspace_size", "gemm_ex_ws", "gemm_ex_noalloc",
              "gemm_gated_preshuffle", "gemm_gated", "gemm_gated_workspace_size", "gemm_gated_backward",
              "gemm_gated_backward_workspace_size",
              "gemm_backward", "gemm_backward_workspace_size", "gemm_w4a16_weights_size", "gemm_w4a16_preshuffle",
              "gemm_w4a16", "gemm_w4a16_gated", "gemm_w4a16_workspace_size", "gemm_w4a16_ws", "gemm_gated_plan",
              "gemm_w4a16_plan", "gemm_backward_plan"):
        getattr(lib, f).restype = ci
    _lib = lib
    return lib


def source_hash() -> str:
    """SHA-256 over the HIP sources of the library (identifies a kernel build)."""
    import hashlib

    csrc = os.path.join(_PKG, "csrc")
    h = hashlib.sha256()
    for f in sorted(os.listdir(csrc)):
        if f.endswith((".hip", ".hpp", ".h")):
            h.update(f.encode())
            h.update(open(os.path.join(csrc, f), "rb").read())
    return h.hexdigest()


def header_functions() -> list:
    """Names of the functions the public header declares."""
    hdr = os.path.join(os.path.dirname(_PKG), "include", "gemm_preshuffle.h")
    txt = open(hdr).read()
    return re.findall(r"^(?:int|const char\*)\s+(\w+)\(", txt, flags=re.M)


def gemm_status_string(status: int) -> str:
    try:
        return load_library().gemm_status_string(int(status)).decode()
    except GemmLibraryMissing:
        return "library not built"


def _opts(opts):
    if opts is None:
        return None
    if isinstance(opts, GemmOpts):
        return ctypes.byref(opts)
    o = GemmOpts()
    for k, v in dict(opts).items():
        setattr(o, k, int(v))
    return ctypes.byref(o)


def _dt(x) -> int:
    return DTYPES[x] if isinstance(x, str) else int(x)


def _stream(stream):
    """The handle of a stream argument: None is torch's current stream, an int a handle, else a torch stream."""
    if stream is None:
        from torch import _C

        # the handle alone: making the Stream object of torch.cuda.current_stream()
        # took 2.6 us of the 9 us that a small product's call spent on the host
        return _C._cuda_getCurrentRawStream(_C._cuda_getDevice())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(status: int, where: str):
    if status != 0:
        raise GemmError(status, where)


def _row_bytes(t) -> int:
    return t.shape[-1] * t.element_size()


def gemm_plan(dtype, M: int, N: int, K: int, opts=None) -> dict:
    """Host-only: the plan a GEMM call with these sizes and options would launch."""
    info = GemmPlanInfo()
    _check(load_library().gemm_plan(_dt(dtype), M, N, K, _opts(opts), ctypes.byref(info)), "gemm_plan")
    return {name: getattr(info, name) for name, _ in GemmPlanInfo._fields_}


def gemm_plan_ws(dtype, M: int, N: int, K: int, opts=None) -> dict:
    """Host-only: the plan of gemm_ex_ws with these sizes and options (it may split K)."""
    info = GemmPlanInfo()
    _check(load_library().gemm_plan_ws(_dt(dtype), M, N, K, _opts(opts), ctypes.byref(info)), "gemm_plan_ws")
    return {name: getattr(info, name) for name, _ in GemmPlanInfo._fields_}


def gemm_workspace_size(dtype, M: int, N: int, K: int, opts=None) -> int:
    """Host-only: workspace bytes a gemm_ex_ws call with these arguments needs (0: none)."""
    n = ctypes.c_size_t()
    _check(load_library().gemm_workspace_size(_dt(dtype), M, N, K, _opts(opts), ctypes.byref(n)),
           "gemm_workspace_size")
    return int(n.value)


def workspace(dtype, M: int, N: int, K: int, opts=None, device="cuda"):
    """A zero-filled device workspace for gemm_ex_ws with these arguments (None when none is needed).
    Zero once here; every call leaves its counters zero again."""
    import torch

    n = gemm_workspace_size(dtype, M, N, K, opts)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


def gemm_preshuffle_b(b, dtype, out=None, stream=None):
    """B [N, K] (device tensor) -> preshuffled bytes (uint8, flat, N*Kb)."""
    import torch

    dt = _dt(dtype)
    N = b.shape[0]
    Kb = _row_bytes(b)
    K = Kb * 8 // _ELEM_BITS[dt]
    if out is None:
        out = torch.empty(N * Kb, dtype=torch.uint8, device=b.device)
    _check(load_library().gemm_preshuffle_b(_ptr(b), _ptr(out), N, K, dt, _stream(stream)),
           "gemm_preshuffle_b")
    return out


def gemm_a8w8(a, b_shuf, scale_a=None, scale_b=None, c=None, N=None, in_dtype="int8",
              opts=None, stream=None):
    """INT8 (-> int32, no scales) or FP8 E4M3 (-> bf16, fp32 scales) GEMM."""
    import torch

    dt = _dt(in_dtype)
    M, K = a.shape[0], _row_bytes(a)
    if N is None:
        N = b_shuf.numel() * b_shuf.element_size() // K
    out_dt = GP_I32 if dt == GP_I8 else GP_BF16
    if c is None:
        c = torch.empty(M, N, dtype=torch.int32 if out_dt == GP_I32 else torch.bfloat16, device=a.device)
    _check(load_library().gemm_a8w8(_ptr(a), _ptr(b_shuf), _ptr(scale_a), _ptr(scale_b), _ptr(c),
                                    M, N, K, dt, out_dt, _opts(opts), _stream(stream)), "gemm_a8w8")
    return c


def gemm_bf16(a, b_shuf, c=None, N=None, opts=None, stream=None):
    """BF16 GEMM, bf16 output."""
    import torch

    M, K = a.shape[0], a.shape[1]
    if N is None:
        N = b_shuf.numel() * b_shuf.element_size() // (2 * K)
    if c is None:
        c = torch.empty(M, N, dtype=torch.bfloat16, device=a.device)
    _check(load_library().gemm_bf16(_ptr(a), _ptr(b_shuf), _ptr(c), M, N, K, _opts(opts), _stream(stream)),
           "gemm_bf16")
    return c


def gemm_mxfp4(a, scale_a, b_shuf, scale_b, c=None, N=None, opts=None, stream=None):
    """MXFP4 GEMM: a uint8 [M, K/2], scale_a uint8 [M, K/32], bf16 output."""
    import torch

    M, K = a.shape[0], 2 * _row_bytes(a)
    if N is None:
        N = b_shuf.numel() * b_shuf.element_size() * 2 // K
    if c is None:
        c = torch.empty(M, N, dtype=torch.bfloat16, device=a.device)
    _check(load_library().gemm_mxfp4(_ptr(a), _ptr(scale_a), _ptr(b_shuf), _ptr(scale_b), _ptr(c),
                                     M, N, K, _opts(opts), _stream(stream)), "gemm_mxfp4")
    return c


def gemm_f16(a, b_shuf, c=None, N=None, opts=None, stream=None):
    """FP16 GEMM, fp16 output."""
    import torch

    M, K = a.shape[0], a.shape[1]
    if N is None:
        N = b_shuf.numel() * b_shuf.element_size() // (2 * K)
    if c is None:
        c = torch.empty(M, N, dtype=torch.float16, device=a.device)
    _check(load_library().gemm_f16(_ptr(a), _ptr(b_shuf), _ptr(c), M, N, K, _opts(opts), _stream(stream)),
           "gemm_f16")
    return c


def gemm_w4a8(a, b_shuf, scale_a, scale_b, c=None, N=None, opts=None, stream=None):
    """int8 A [M, K] x INT4 B (preshuffled as GP_I4), fp32 scales, bf16 output."""
    import torch

    M, K = a.shape[0], _row_bytes(a)
    if N is None:
        N = b_shuf.numel() * b_shuf.element_size() * 2 // K
    if c is None:
        c = torch.empty(M, N, dtype=torch.bfloat16, device=a.device)
    _check(load_library().gemm_w4a8(_ptr(a), _ptr(b_shuf), _ptr(scale_a), _ptr(scale_b), _ptr(c),
                                    M, N, K, _opts(opts), _stream(stream)), "gemm_w4a8")
    return c


def gemm_ex(dtype, a, b_shuf, scale_a=None, scale_b=None, bias=None, act="none", c=None, N=None,
            opts=None, stream=None):
    """Any input type with the fused epilogue: C = act(scaled accumulator + bias[n])."""
    import torch

    dt = _dt(dtype)
    out_dt = _OUT[dt]
    M = a.shape[0]
    K = _row_bytes(a) * 8 // (8 if dt == GP_I4 else _ELEM_BITS[dt])
    if N is None:
        N = b_shuf.numel() * b_shuf.element_size() * 8 // (K * _ELEM_BITS[dt])
    if c is None:
        tdt = {GP_I32: torch.int32, GP_BF16: torch.bfloat16, GP_F16: torch.float16}[out_dt]
        c = torch.empty(M, N, dtype=tdt, device=a.device)
    a_ = ACTS[act] if isinstance(act, str) else int(act)
    _check(load_library().gemm_ex(dt, out_dt, _ptr(a), _ptr(b_shuf), _ptr(scale_a), _ptr(scale_b), _ptr(bias),
                                  a_, _ptr(c), M, N, K, _opts(opts), _stream(stream)), "gemm_ex")
    return c


def gemm_ex_ws(dtype, a, b_shuf, scale_a=None, scale_b=None, bias=None, act="none", c=None, N=None,
               opts=None, workspace=None, stream=None):
    """gemm_ex with a device workspace (a uint8 tensor from `workspace()`), so
    that the planner may split K across workgroups."""
    import torch

    dt = _dt(dtype)
    out_dt = _OUT[dt]
    M = a.shape[0]
    K = _row_bytes(a) * 8 // (8 if dt == GP_I4 else _ELEM_BITS[dt])
    if N is None:
        N = b_shuf.numel() * b_shuf.element_size() * 8 // (K * _ELEM_BITS[dt])
    if c is None:
        tdt = {GP_I32: torch.int32, GP_BF16: torch.bfloat16, GP_F16: torch.float16}[out_dt]
        c = torch.empty(M, N, dtype=tdt, device=a.device)
    a_ = ACTS[act] if isinstance(act, str) else int(act)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load_library().gemm_ex_ws(dt, out_dt, _ptr(a), _ptr(b_shuf), _ptr(scale_a), _ptr(scale_b), _ptr(bias),
                                     a_, _ptr(c), M, N, K, _opts(opts), _ptr(workspace), nbytes, _stream(stream)),
           "gemm_ex_ws")
    return c


def gemm_ex_noalloc(dtype, a, b_shuf, c, scale_a=None, scale_b=None, bias=None, act="none", N=None, opts=None,
                    stream=None):
    """gemm_ex_ws on the library's own static device workspace: nothing is
    allocated, so the output tensor `c` must be given. Calls that overlap in
    time on one device share that workspace and must not be made."""
    dt = _dt(dtype)
    out_dt = _OUT[dt]
    M = a.shape[0]
    K = _row_bytes(a) * 8 // (8 if dt == GP_I4 else _ELEM_BITS[dt])
    if N is None:
        N = b_shuf.numel() * b_shuf.element_size() * 8 // (K * _ELEM_BITS[dt])
    a_ = ACTS[act] if isinstance(act, str) else int(act)
    _check(load_library().gemm_ex_noalloc(dt, out_dt, _ptr(a), _ptr(b_shuf), _ptr(scale_a), _ptr(scale_b),
                                          _ptr(bias), a_, _ptr(c), M, N, K, _opts(opts), _stream(stream)),
           "gemm_ex_noalloc")
    return c


# ---- gated feed-forward product, gradients ----

_HALF = {GP_BF16: "bfloat16", GP_F16: "float16"}


@functools.lru_cache(maxsize=None)
def _half(dtype):
    """(gp_dtype, torch dtype) of a BF16 / FP16 operator."""
    import torch

    dt = _dt(dtype)
    if dt not in _HALF:
        raise GemmError(GP_EDTYPE, "BF16 or FP16 operator")
    return dt, getattr(torch, _HALF[dt])


def _fits(t, shape, dtype, device) -> bool:
    """A contiguous tensor of this shape and type on this device."""
    return t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == device


def _want(where, t, shape, dtype, device=None):
    """A given tensor is a contiguous device tensor of this shape and type."""
    if t.is_cuda and _fits(t, shape, dtype, t.device if device is None else device):
        return
    if (not t.is_cuda or tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous()
            or (device is not None and t.device != device)):
        raise ValueError(f"{where}: expected a contiguous {dtype} tensor {tuple(shape)}"
                         f"{'' if device is None else f' on {device}'}, got {t.dtype} {tuple(t.shape)} "
                         f"on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")


def _act(act) -> int:
    return ACTS[act] if isinstance(act, str) else int(act)


_SAME = contextlib.nullcontext()


def _on(stream, device):
    """Context in which torch allocates for the stream that a call runs on:
    memory from torch's allocator belongs to the stream it was asked for on,
    so a buffer that only the call holds must come from the call's stream."""
    if stream is None:
        return _SAME
    import torch

    if isinstance(stream, int):
        return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device)) if stream else \
            torch.cuda.stream(torch.cuda.default_stream(device))
    return torch.cuda.stream(stream)


# workspace sizes depend on the arguments alone, so a decode loop asks the planner once
@functools.lru_cache(maxsize=1024)
def _size(fn, *args) -> int:
    n = ctypes.c_size_t()
    _check(getattr(load_library(), fn)(*args, ctypes.byref(n)), fn)
    return int(n.value)


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _workspace_bytes(where, t, device) -> int:
    """Bytes of a workspace tensor, which the call's device has to hold in one piece."""
    if t is None:
        return 0
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{where}: expected a contiguous workspace on {device}, got one on {t.device}"
                         f"{'' if t.is_contiguous() else ', not contiguous'}")
    return t.numel() * t.element_size()


def gemm_gated_preshuffle(w, dtype, out=None, stream=None):
    """w [2F, H] (F gate rows, then F up rows) -> layout of gemm_gated (uint8, flat)."""
    import torch

    dt, t = _half(dtype)
    F2, H = w.shape
    if F2 % 2:
        raise ValueError("gemm_gated_preshuffle: w holds F gate rows and F up rows")
    _want("gemm_gated_preshuffle: w", w, (F2, H), t)
    n = 2 * F2 * (-(-H // 64) * 64)    # K is filled up to whole 128-byte tiles
    with _on(stream, w.device):
        out = torch.empty(n, dtype=torch.uint8, device=w.device) if out is None else out
        _want("gemm_gated_preshuffle: out", out, (n,), torch.uint8, w.device)
        _check(load_library().gemm_gated_preshuffle(_ptr(w), _ptr(out), F2 // 2, H, dt, _stream(stream)),
               "gemm_gated_preshuffle")
    return out


def gemm_gated_workspace_size(dtype, M: int, F: int, H: int) -> int:
    """Host-only: workspace bytes of gemm_gated for these sizes (0: none)."""
    return _size("gemm_gated_workspace_size", _dt(dtype), M, F, H)


def gemm_gated_plan(dtype, M: int, F: int, H: int) -> dict:
    """Host-only: the kernel that gemm_gated runs for these sizes."""
    info = GemmPlanInfo()
    _check(load_library().gemm_gated_plan(_dt(dtype), M, F, H, ctypes.byref(info)), "gemm_gated_plan")
    return {name: getattr(info, name) for name, _ in GemmPlanInfo._fields_}


def _split_workspace(n: int, device):
    """n bytes with zero arrival counters (the first 64 KiB). The partial sums after them are written before
    they are read; clearing them too made gemm_gated without a workspace of the caller's 46.0 us instead of
    36.4 at 259 x 2192 x 6560 (28 MB)."""
    import torch

    if not n:
        return None
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:65536].zero_()
    return ws


def gated_workspace(dtype, M: int, F: int, H: int, device="cuda"):
    """A device workspace for gemm_gated, its counters zero (None when none is needed). Zero once here;
    every call leaves its counters zero again. Calls that may overlap need one each."""
    return _split_workspace(gemm_gated_workspace_size(dtype, M, F, H), device)


def gemm_gated(dtype, x, w_shuf, act="silu", save=False, h=None, gate=None, up=None, workspace=None, stream=None):
    """h = act(x Wg^T) * (x Wu^T), x [M, H], w_shuf from gemm_gated_preshuffle.
    Returns h, or (h, gate, up) with save=True. Without a workspace one is made
    for the call where the plan needs it."""
    import torch

    dt, t = _half(dtype)
    M, H = x.shape
    device = x.device
    Hp = -(-H // 64) * 64
    F = _nbytes(w_shuf) // (4 * Hp) if H else 0
    _want("gemm_gated: x", x, (M, H), t)
    _want("gemm_gated: w_shuf", w_shuf, (4 * F * Hp,), torch.uint8, device)
    if not save and (gate is not None or up is not None):
        raise ValueError("gemm_gated: gate and up are written with save=True")
    for name, v in (("h", h), ("gate", gate), ("up", up)):
        if v is not None and not _fits(v, (M, F), t, device):
            _want(f"gemm_gated: {name}", v, (M, F), t, device)
    with _on(stream, device):
        h = x.new_empty((M, F)) if h is None else h
        if save:
            gate = x.new_empty((M, F)) if gate is None else gate
            up = x.new_empty((M, F)) if up is None else up
        if workspace is None:
            workspace = gated_workspace(dt, M, F, H, device)
    _check(load_library().gemm_gated(dt, x.data_ptr(), w_shuf.data_ptr(), _act(act), h.data_ptr(), _ptr(gate), _ptr(up),
                                     M, F, H, _ptr(workspace), _workspace_bytes("gemm_gated", workspace, device),
                                     _stream(stream)), "gemm_gated")
    return (h, gate, up) if save else h


def gemm_gated_backward_workspace_size(dtype, M: int, F: int, H: int, want_dx=True, want_dw=True) -> int:
    """Host-only: workspace bytes of gemm_gated_backward."""
    return _size("gemm_gated_backward_workspace_size", _dt(dtype), M, F, H, int(want_dx), int(want_dw))


def gated_backward_workspace(dtype, M: int, F: int, H: int, want_dx=True, want_dw=True, device="cuda"):
    """A device workspace for gemm_gated_backward (its contents need not be set)."""
    import torch

    return torch.empty(gemm_gated_backward_workspace_size(dtype, M, F, H, want_dx, want_dw), dtype=torch.uint8,
                       device=device)


def gemm_gated_backward(dtype, dh, gate, up, x, w, act="silu", want_dx=True, want_dw=True, dx=None, dw=None,
                        workspace=None, stream=None):
    """(dx [M, H], dw [2F, H]) of gemm_gated from dh and the kept gate and up
    ([M, F]); w [2F, H] row-major. An output that is not wanted is None, and the
    operand that it alone needs (w for dx, x for dw) may be None. The gradients of
    gate and up are rounded to the type on the way (fp16: infinite beyond 65504)."""
    dt, t = _half(dtype)
    M, F = dh.shape
    dev = dh.device
    if not (want_dx or want_dw):
        raise ValueError("gemm_gated_backward: no output wanted")
    if (want_dx and w is None) or (want_dw and x is None):
        raise ValueError("gemm_gated_backward: dx needs w, dw needs x")
    if not dh.is_cuda:
        raise ValueError("gemm_gated_backward: dh is not a device tensor")
    H = w.shape[1] if w is not None else x.shape[1]
    for name, v, shape in (("dh", dh, (M, F)), ("gate", gate, (M, F)), ("up", up, (M, F)), ("x", x, (M, H)),
                           ("w", w, (2 * F, H)), ("dx", dx, (M, H)), ("dw", dw, (2 * F, H))):
        if v is not None and not _fits(v, shape, t, dev):
            _want(f"gemm_gated_backward: {name}", v, shape, t, dev)
    with _on(stream, dev):
        dx = (dh.new_empty((M, H)) if dx is None else dx) if want_dx else None
        dw = (dh.new_empty((2 * F, H)) if dw is None else dw) if want_dw else None
        if workspace is None:
            workspace = gated_backward_workspace(dt, M, F, H, want_dx, want_dw, dev)
        _check(load_library().gemm_gated_backward(dt, _ptr(dh), _ptr(gate), _ptr(up), _ptr(x), _ptr(w), _act(act),
                                                  _ptr(dx), _ptr(dw), M, F, H, _ptr(workspace),
                                                  _workspace_bytes("gemm_gated_backward", workspace, dev),
                                                  _stream(stream)), "gemm_gated_backward")
    return dx, dw


def gemm_backward_workspace_size(dtype, M: int, N: int, K: int, want_da=True, want_db=True) -> int:
    """Host-only: workspace bytes of gemm_backward."""
    return _size("gemm_backward_workspace_size", _dt(dtype), M, N, K, int(want_da), int(want_db))


def gemm_backward_plan(dtype, M: int, N: int, K: int, want_da=True, want_db=True, gated=False) -> tuple:
    """Host-only: the kernels of the two products of gemm_backward (gated: of gemm_gated_backward, N is F
    and K is H) for these sizes; None for an output that is not wanted."""
    infos = GemmPlanInfo(), GemmPlanInfo()
    _check(load_library().gemm_backward_plan(_dt(dtype), M, N, K, int(want_da), int(want_db), int(gated),
                                             *(ctypes.byref(i) for i in infos)), "gemm_backward_plan")
    return tuple({name: getattr(i, name) for name, _ in GemmPlanInfo._fields_} if want else None
                 for i, want in zip(infos, (want_da, want_db)))


def backward_workspace(dtype, M: int, N: int, K: int, want_da=True, want_db=True, device="cuda"):
    """A device workspace for gemm_backward (its contents need not be set)."""
    import torch

    return torch.empty(gemm_backward_workspace_size(dtype, M, N, K, want_da, want_db), dtype=torch.uint8,
                       device=device)


def gemm_backward(dtype, dc, a, b, want_da=True, want_db=True, da=None, db=None, workspace=None, stream=None):
    """(da [M, K], db [N, K]) of C = A B^T from dc [M, N]; a [M, K] and b [N, K]
    row-major. An output that is not wanted is None, and the operand that it
    alone needs (b for da, a for db) may be None."""
    dt, t = _half(dtype)
    M, N = dc.shape
    dev = dc.device
    if not (want_da or want_db):
        raise ValueError("gemm_backward: no output wanted")
    if (want_da and b is None) or (want_db and a is None):
        raise ValueError("gemm_backward: da needs b, db needs a")
    if not dc.is_cuda:
        raise ValueError("gemm_backward: dc is not a device tensor")
    K = b.shape[1] if b is not None else a.shape[1]
    for name, v, shape in (("dc", dc, (M, N)), ("a", a, (M, K)), ("b", b, (N, K)), ("da", da, (M, K)),
                           ("db", db, (N, K))):
        if v is not None and not _fits(v, shape, t, dev):
            _want(f"gemm_backward: {name}", v, shape, t, dev)
    with _on(stream, dev):
        da = (dc.new_empty((M, K)) if da is None else da) if want_da else None
        db = (dc.new_empty((N, K)) if db is None else db) if want_db else None
        if workspace is None:
            workspace = backward_workspace(dt, M, N, K, want_da, want_db, dev)
        _check(load_library().gemm_backward(dt, _ptr(dc), _ptr(a), _ptr(b), _ptr(da), _ptr(db), M, N, K,
                                            _ptr(workspace), _workspace_bytes("gemm_backward", workspace, dev),
                                            _stream(stream)), "gemm_backward")
    return da, db


# ---- 4-bit weights with group scales ----

class W4Weights:
    """Laid-out 4-bit weights (gemm_w4a16_preshuffle): the device buffer and what it holds.
    N is the number of output columns (gated: F, from 2 F rows)."""

    __slots__ = ("data", "dtype", "N", "K", "group", "has_zeros", "gated", "device", "gp_dtype")

    def __init__(self, data, dtype, N, K, group, has_zeros, gated):
        self.data, self.dtype, self.N, self.K = data, dtype, N, K
        self.group, self.has_zeros, self.gated = group, has_zeros, gated
        # read once: a decode step's products take a few microseconds each
        self.device = data.device
        self.gp_dtype = next(k for k, v in _HALF.items() if str(dtype) == f"torch.{v}")


def gemm_w4a16_weights_size(N: int, K: int, group: int, has_zeros=False, gated=False) -> int:
    """Host-only: bytes of laid-out 4-bit weights (gated: N = 2 F rows)."""
    return _size("gemm_w4a16_weights_size", N, K, group, int(has_zeros), int(gated))


def gemm_w4a16_preshuffle(q, scales, zeros=None, group=128, gated=False, out=None, stream=None) -> W4Weights:
    """q uint8 [N, K/2] (two's complement 4-bit integers, the even k in the low nibble), scales bf16 or
    fp16 [N, ceil(K/group)], zeros int8 of that shape or None -> W4Weights for gemm_w4a16, or with
    gated (F gate rows, then F up rows) for gemm_w4a16_gated. x has the scales' type."""
    import torch

    where = "gemm_w4a16_preshuffle"
    N, K = q.shape[0], 2 * q.shape[1]
    if scales.dtype not in (torch.bfloat16, torch.float16):
        raise GemmError(GP_EDTYPE, f"{where}: scales are bf16 or fp16")
    dt = GP_BF16 if scales.dtype == torch.bfloat16 else GP_F16
    n = gemm_w4a16_weights_size(N, K, group, zeros is not None, gated)
    groups = -(-K // group)
    _want(f"{where}: q", q, (N, K // 2), torch.uint8)
    _want(f"{where}: scales", scales, (N, groups), scales.dtype, q.device)
    if zeros is not None:
        _want(f"{where}: zeros", zeros, (N, groups), torch.int8, q.device)
    with _on(stream, q.device):
        out = torch.empty(n, dtype=torch.uint8, device=q.device) if out is None else out
        _want(f"{where}: out", out, (n,), torch.uint8, q.device)
        _check(load_library().gemm_w4a16_preshuffle(dt, _ptr(q), _ptr(scales), _ptr(zeros), _ptr(out), N, K, group,
                                                    int(gated), _stream(stream)), where)
    return W4Weights(out, scales.dtype, N // 2 if gated else N, K, int(group), zeros is not None, bool(gated))


def gemm_w4a16_workspace_size(M: int, N: int, K: int, group: int, gated=False) -> int:
    """Host-only: workspace bytes with which a 4-bit product of these sizes (gated: N is F) may split K
    across workgroups (0: it does not)."""
    return _size("gemm_w4a16_workspace_size", M, N, K, group, int(gated))


def gemm_w4a16_plan(M: int, N: int, K: int, group: int, gated=False, with_workspace=False) -> dict:
    """Host-only: the kernel variant of a 4-bit product of these sizes (gated: N is F)."""
    info = GemmPlanInfo()
    _check(load_library().gemm_w4a16_plan(M, N, K, group, int(gated), int(with_workspace), ctypes.byref(info)),
           "gemm_w4a16_plan")
    return {name: getattr(info, name) for name, _ in GemmPlanInfo._fields_}


def w4a16_workspace(M: int, weights: W4Weights):
    """A device workspace for products of M rows on these weights, its counters zero (None when none is needed).
    Zero once here; every call leaves its counters zero again. Calls that may overlap need one each."""
    return _split_workspace(gemm_w4a16_workspace_size(M, weights.N, weights.K, weights.group, weights.gated),
                            weights.device)


def _w4_run(where, gated, x, weights, bias, act, y, workspace, stream):
    """One 4-bit product. A decode step's products take a few microseconds on the GPU, about what this
    function and the launch take on the host, so it asks each thing once."""
    device, dtype, N, K = weights.device, weights.dtype, weights.N, weights.K
    shape = x.shape
    M = shape[0]
    if weights.gated is not gated:
        raise ValueError(f"{where}: the weights were laid out {'not ' if gated else ''}gated")
    if not (x.dtype is dtype and shape == (M, K) and x.is_contiguous() and x.device == device):
        _want(f"{where}: x", x, (M, K), dtype, device)
    if bias is not None:
        import torch

        _want(f"{where}: bias", bias, (N,), torch.float32, device)
        bias = bias.data_ptr()
    if stream is None:
        handle = _stream(None)
        out = x.new_empty((M, N)) if y is None else y
    else:
        handle = _stream(stream)
        with _on(stream, device):
            out = x.new_empty((M, N)) if y is None else y
    if y is not None:
        _want(f"{where}: output", y, (M, N), dtype, device)
    if workspace is None and M > 16 and K > 8192:
        # A split on a workspace made here takes 12.4 us at least, the host's time for making and clearing it:
        # 64 x 392 x 8224 12.5 us against 15.7 unsplit, 32 x 392 x 16384 12.6 (17.7), but 17 x 392 x 8224 12.8
        # (10.1) and 16 x 392 x 16384 12.6 (12.0). With a workspace that the caller keeps 10.1, 8.0, 6.7, 7.5.
        with _on(stream, device):
            workspace = w4a16_workspace(M, weights)
    act = _act(act)
    lib = load_library()
    if workspace is not None:
        status = lib.gemm_w4a16_ws(weights.gp_dtype, x.data_ptr(), weights.data.data_ptr(), weights.has_zeros, bias,
                                    act, out.data_ptr(), M, N, K, weights.group, gated, workspace.data_ptr(),
                                    _workspace_bytes(where, workspace, device), handle)
    elif gated:
        status = lib.gemm_w4a16_gated(weights.gp_dtype, x.data_ptr(), weights.data.data_ptr(), weights.has_zeros,
                                       act, out.data_ptr(), M, N, K, weights.group, handle)
    else:
        status = lib.gemm_w4a16(weights.gp_dtype, x.data_ptr(), weights.data.data_ptr(), weights.has_zeros, bias,
                                 act, out.data_ptr(), M, N, K, weights.group, handle)
    if status:
        _check(status, where)
    return out


def gemm_w4a16(x, weights: W4Weights, bias=None, act="none", y=None, workspace=None, stream=None):
    """y = act(x W^T + bias) on 4-bit weights: x [M, K] of the scales' type, bias fp32 [N] or None.
    workspace: from w4a16_workspace, kept by callers of few rows on a long K. With one K may be split across
    workgroups, without one it is not, except that a call of more than 16 rows on K > 8192 makes its own: the
    order of the fp32 sums, and so the last bits, depend on which. The same call gives the same bits."""
    return _w4_run("gemm_w4a16", False, x, weights, bias, act, y, workspace, stream)


def gemm_w4a16_gated(x, weights: W4Weights, act="silu", h=None, workspace=None, stream=None):
    """h = act(x Wg^T) * (x Wu^T) on 4-bit weights laid out gated: x [M, K] of the scales' type; workspace as
    for gemm_w4a16."""
    return _w4_run("gemm_w4a16_gated", True, x, weights, None, act, h, workspace, stream)
