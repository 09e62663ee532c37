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
    gemm_linear_preshuffle(w, dtype)                 -> weights [N, K] laid out for gemm_linear
    gemm_linear(dtype, x, w_shuf, bias, act, residual, save)
                                                     -> y = act(x W^T + bias) + residual (and z to keep)
    gemm_linear_backward(dtype, dy, z, x, w, act)    -> dx, dw, dbias
    gated_workspace, gated_backward_workspace, backward_workspace, linear_workspace, linear_backward_workspace
                                                     -> device workspaces of these
    gemm_w4a16_preshuffle(q, scales, zeros, group)   -> W4Weights, 4-bit weights laid out with their scales
    gemm_w4a16(x, weights, bias, act)                -> act(x W^T + bias) (BF16 / FP16 activations)
    gemm_w4a16_gated(x, weights, act)                -> act(x Wg^T) * (x Wu^T) on 4-bit weights
    w4a16_workspace(M, weights)                      -> a device workspace of these (None: none needed)
    gemm_norm(dtype, x, residual, norm_in, gate, norm_out)
                                                     -> r = scale * residual + gate * norm_in(x), y = norm_out(r)
    gemm_norm_backward(dtype, dy, dr, x, r, ...)     -> NormGrads
    norm_backward_workspace                          -> a device workspace of it
    gemm_moe_preshuffle(w13, w2, dtype)              -> MoeWeights, the experts' weights laid out
    gemm_moe(dtype, x, router, weights, k, ...)      -> y, ids, gates of a mixture-of-experts layer (a few tokens)
    gemm_moe_route(dtype, x, router, k, ...)         -> ids, gates (the router alone)
    gemm_moe_experts(dtype, x, weights, ids, gates)  -> y (the experts alone)
    moe_workspace(M, k, weights)                     -> a device workspace of these
    gemm_gated_plan, gemm_linear_plan, gemm_w4a16_plan
                                                     -> dict, the kernel they run (host-only)
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
import typing

__all__ = [
    "GemmError", "GemmLibraryMissing", "GemmOpts", "lib_path", "load_library",
    "gemm_preshuffle_b", "gemm_a8w8", "gemm_bf16", "gemm_mxfp4", "gemm_f16", "gemm_w4a8", "gemm_ex",
    "gemm_plan", "ACTS", "gemm_ex_ws", "gemm_ex_noalloc", "gemm_workspace_size", "gemm_plan_ws", "workspace",
    "gemm_gated_preshuffle", "gemm_gated", "gemm_gated_workspace_size", "gated_workspace", "gemm_gated_backward",
    "gemm_gated_backward_workspace_size", "gated_backward_workspace", "gemm_backward", "gemm_backward_workspace_size",
    "backward_workspace", "W4Weights", "gemm_w4a16_weights_size", "gemm_w4a16_preshuffle", "gemm_w4a16",
    "gemm_w4a16_gated", "gemm_w4a16_workspace_size", "w4a16_workspace", "gemm_gated_plan", "gemm_w4a16_plan",
    "gemm_backward_plan", "gemm_linear_preshuffle", "gemm_linear", "gemm_linear_workspace_size", "gemm_linear_plan",
    "linear_workspace", "gemm_linear_backward", "gemm_linear_backward_workspace_size", "linear_backward_workspace", "NORMS", "NormGrads", "gemm_norm", "gemm_norm_backward", "gemm_norm_backward_workspace_size",
    "norm_backward_workspace", "SCORES", "MoeWeights", "gemm_moe_weights_size", "gemm_moe_preshuffle", "gemm_moe_route",
    "gemm_moe_experts", "gemm_moe", "gemm_moe_workspace_size", "moe_workspace", "gemm_status_string", "source_hash", "DTYPES", "EPI_DIRECT", "EPI_CSHUFFLE", "KERNEL_TILE",
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
# gp_norm values of the C ABI
NORMS = {"none": 0, "rms": 1, "layer": 2}
# gp_score values of the C ABI
SCORES = {"softmax": 0, "sigmoid": 1}
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
    lib.gemm_linear_preshuffle.argtypes = [vp, vp, i64, i64, ci, vp]
    lib.gemm_linear.argtypes = [ci, vp, vp, vp, ci, vp, vp, vp, i64, i64, i64, vp, sz, vp]
    lib.gemm_linear_workspace_size.argtypes = [ci, i64, i64, i64, psz]
    lib.gemm_linear_plan.argtypes = [ci, i64, i64, i64, ctypes.POINTER(GemmPlanInfo)]
    lib.gemm_linear_backward.argtypes = [ci, vp, vp, vp, vp, ci, vp, vp, vp, i64, i64, i64, vp, sz, vp]
    lib.gemm_linear_backward_workspace_size.argtypes = [ci, i64, i64, i64, ci, ci, ci, ci, psz]
    cf = ctypes.c_float
    lib.gemm_norm.argtypes = [ci, vp, vp, cf, ci, vp, vp, vp, i64, ci, vp, vp, cf, vp, vp, i64, i64, vp]
    lib.gemm_norm_backward.argtypes = [ci, vp, vp, vp, vp, cf, ci, vp, vp, vp, i64, ci, vp, cf, vp, vp, vp, vp, vp, vp,
                                       vp, i64, i64, vp, sz, vp]
    lib.gemm_norm_backward_workspace_size.argtypes = [ci, i64, i64, i64, psz]
    lib.gemm_moe_weights_size.argtypes = [i64, i64, i64, psz]
    lib.gemm_moe_preshuffle.argtypes = [ci, vp, vp, vp, i64, i64, i64, vp]
    lib.gemm_moe_workspace_size.argtypes = [ci, i64, i64, i64, i64, i64, psz]
    lib.gemm_moe_route.argtypes = [ci, vp, vp, vp, ci, ci, cf, vp, vp, i64, i64, i64, i64, vp, sz, vp]
    lib.gemm_moe_experts.argtypes = [ci, vp, vp, vp, vp, ci, vp, vp, i64, i64, i64, i64, i64, vp, sz, vp]
    lib.gemm_moe.argtypes = [ci, vp, vp, vp, ci, ci, cf, vp, ci, vp, vp, vp, vp, i64, i64, i64, i64, i64, vp, sz, vp]
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
              "gemm_w4a16_plan", "gemm_backward_plan", "gemm_linear_preshuffle", "gemm_linear",
              "gemm_linear_workspace_size", "gemm_linear_plan", "gemm_linear_backward",
              "gemm_linear_backward_workspace_size", "gemm_norm", "gemm_norm_backward",
              "gemm_norm_backward_workspace_size", "gemm_moe_weights_size", "gemm_moe_preshuffle",
              "gemm_moe_workspace_size", "gemm_moe_route", "gemm_moe_experts", "gemm_moe"):
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


def marshal_hash() -> str:
    """SHA-256 of what the binding's compiled marshalling is built from: its source, the header whose signatures it
    calls through, and torch's version."""
    import hashlib

    import torch

    h = hashlib.sha256(torch.__version__.encode())
    for f in (os.path.join(_PKG, "csrc", "marshal.cpp"), os.path.join(os.path.dirname(_PKG), "include", "gemm_preshuffle.h")):
        h.update(open(f, "rb").read())
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


@functools.lru_cache(maxsize=None)
def _cuda():
    """torch's current device index, and the handle of a device's current stream (looked up once: an import
    statement in a call takes 0.3 us)."""
    from torch import _C

    return _C._cuda_getDevice, _C._cuda_getCurrentRawStream


def _stream(stream):
    """The handle of a stream argument: None is torch's current stream, an int a handle, else a torch stream."""
    if stream is None:
        # the handle alone: making the Stream object of torch.cuda.current_stream()
        # took 2.6 us of the 9 us that a small product's call spent on the host
        device, raw = _cuda()
        return raw(device())
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


@functools.lru_cache(maxsize=None)
def _types():
    """(float32, int32, uint8) of torch, and its empty_like."""
    import torch

    return torch.float32, torch.int32, torch.uint8, torch.empty_like


def _device() -> int:
    return _cuda()[0]()


def _is(t, dtype, shape, index) -> bool:
    """A contiguous tensor of this type and shape on device `index`. The operators below check each tensor with it
    once, and name the wrong one (_want) only where a check has failed."""
    return t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous()


def _here(where, name, t, stream):
    """A call's first tensor is on the current device, where its kernels are launched, and so is its stream."""
    if not t.is_cuda:
        raise ValueError(f"{where}: {name} is not a device tensor")
    if t.device.index != _device():
        raise ValueError(f"{where}: {name} is on {t.device}, the current device is cuda:{_device()}")
    if stream is not None and not isinstance(stream, int) and stream.device != t.device:
        raise ValueError(f"{where}: {name} is on {t.device}, the stream on {stream.device}")


@functools.lru_cache(maxsize=None)
def _compiled():
    """The compiled marshalling (csrc/marshal.cpp) of calls on the current stream, bound to the library; None where
    it is not built, or from other sources than these: against another header it would call the entry points through
    other signatures. Its functions do what the Python below them does, in 1 us and not 5, and return None where
    anything is not as it should be: the Python then names what."""
    lib = load_library()
    try:
        from . import _marshal
    except ImportError:
        return None
    try:
        same = getattr(_marshal, "sources", None) == marshal_hash()
    except OSError:    # (no sources beside the binding)
        same = False
    if not same:
        import warnings

        warnings.warn("the compiled marshalling (_marshal.so) was built from other sources than these: calls go through "
                      "ctypes until it is built again", stacklevel=2)
        return None
    _marshal.bind(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in (
        "gemm_norm", "gemm_norm_backward", "gemm_norm_backward_workspace_size", "gemm_linear",
        "gemm_linear_workspace_size", "gemm_linear_backward", "gemm_linear_backward_workspace_size")))
    return _marshal


# ---- linear layer with its epilogue ----

def gemm_linear_preshuffle(w, dtype, out=None, stream=None):
    """w [N, K] -> layout of gemm_linear (uint8, flat)."""
    import torch

    dt, t = _half(dtype)
    _here("gemm_linear_preshuffle", "w", w, stream)
    N, K = w.shape
    _want("gemm_linear_preshuffle: w", w, (N, K), t)
    n = 2 * N * (-(-K // 64) * 64)    # K is filled up to whole 128-byte tiles
    with _on(stream, w.device):
        out = torch.empty(n, dtype=torch.uint8, device=w.device) if out is None else out
        _want("gemm_linear_preshuffle: out", out, (n,), torch.uint8, w.device)
        _check(load_library().gemm_linear_preshuffle(_ptr(w), _ptr(out), N, K, dt, _stream(stream)),
               "gemm_linear_preshuffle")
    return out


def gemm_linear_workspace_size(dtype, M: int, N: int, K: int) -> int:
    """Host-only: workspace bytes of gemm_linear for these sizes (0: none)."""
    return _size("gemm_linear_workspace_size", _dt(dtype), M, N, K)


def gemm_linear_plan(dtype, M: int, N: int, K: int) -> dict:
    """Host-only: the kernel that gemm_linear runs for these sizes."""
    info = GemmPlanInfo()
    _check(load_library().gemm_linear_plan(_dt(dtype), M, N, K, ctypes.byref(info)), "gemm_linear_plan")
    return {name: getattr(info, name) for name, _ in GemmPlanInfo._fields_}


def linear_workspace(dtype, M: int, N: int, K: int, device="cuda"):
    """A device workspace for gemm_linear, its counters zero (None when none is needed). Zero once here;
    every call leaves its counters zero again. Calls that may overlap need one each."""
    return _split_workspace(gemm_linear_workspace_size(dtype, M, N, K), device)


def gemm_linear(dtype, x, w_shuf, bias=None, act="none", residual=None, save=False, y=None, z=None, workspace=None,
                stream=None):
    """y = act(x W^T + bias) + residual: x [M, K], w_shuf from gemm_linear_preshuffle, bias fp32 [N], residual
    [M, N], either of them None. Returns y, or (y, z) with save=True, z = x W^T + bias in x's type. y may be the
    residual. Without a workspace one is made for the call where the plan needs it."""
    where = "gemm_linear"
    dt, t = _half(dtype)
    if stream is None and x.is_cuda and (fast := _compiled()) is not None:
        out = fast.linear(dt, x, w_shuf, bias, _act(act), residual, bool(save), y, z, workspace, _device(), _stream(None))
        if out is not None:
            return out
    M, K = shape = x.shape
    index, device = x.get_device(), x.device
    if stream is not None or index < 0 or index != _device():
        _here(where, "x", x, stream)
    f32, _, u8, _ = _types()
    Kp = -(-K // 64) * 64
    N = w_shuf.numel() // (2 * Kp) if K else 0
    out = (M, N)
    if not (_is(x, t, shape, index) and _is(w_shuf, u8, (2 * N * Kp,), index)
            and (residual is None or _is(residual, t, out, index)) and (bias is None or _is(bias, f32, (N,), index))
            and (y is None or _is(y, t, out, index)) and (z is None or _is(z, t, out, index))):
        for name, v, d, sh in (("x", x, t, shape), ("w_shuf", w_shuf, u8, (2 * N * Kp,)), ("residual", residual, t, out),
                               ("bias", bias, f32, (N,)), ("y", y, t, out), ("z", z, t, out)):
            if v is not None:
                _want(f"{where}: {name}", v, sh, d, device)
    if not save and z is not None:
        raise ValueError(f"{where}: z is written with save=True")
    with _on(stream, device):
        y = x.new_empty(out) if y is None else y
        if save and z is None:
            z = x.new_empty(out)
        if workspace is None:
            workspace = linear_workspace(dt, M, N, K, device)
    status = load_library().gemm_linear(dt, x.data_ptr(), w_shuf.data_ptr(), _ptr(bias), _act(act), _ptr(residual),
                                        y.data_ptr(), _ptr(z), M, N, K, _ptr(workspace),
                                        _workspace_bytes(where, workspace, device), _stream(stream))
    if status:
        _check(status, where)
    return (y, z) if save else y


def gemm_linear_backward_workspace_size(dtype, M: int, N: int, K: int, act="silu", want_dx=True, want_dw=True,
                                        want_dbias=True) -> int:
    """Host-only: workspace bytes of gemm_linear_backward (any activation's serve act="none" too)."""
    return _size("gemm_linear_backward_workspace_size", _dt(dtype), M, N, K, _act(act), int(want_dx), int(want_dw),
                 int(want_dbias))


def linear_backward_workspace(dtype, M: int, N: int, K: int, act="silu", want_dx=True, want_dw=True, want_dbias=True,
                              device="cuda"):
    """A device workspace for gemm_linear_backward (its contents need not be set); one for any activation serves
    act="none" too."""
    import torch

    return torch.empty(gemm_linear_backward_workspace_size(dtype, M, N, K, act, want_dx, want_dw, want_dbias),
                       dtype=torch.uint8, device=device)


def gemm_linear_backward(dtype, dy, z, x, w, act="none", want_dx=True, want_dw=True, want_dbias=True, dx=None, dw=None,
                         dbias=None, workspace=None, stream=None):
    """(dx [M, K], dw [N, K], dbias fp32 [N]) of gemm_linear from dy and the kept z ([M, N]; None without an
    activation); w [N, K] row-major. An output that is not wanted is None, and the operand that it alone needs (w
    for dx, x for dw) may be None. The residual's gradient is dy itself."""
    import torch

    where = "gemm_linear_backward"
    dt, t = _half(dtype)
    if stream is None and dy.is_cuda and (fast := _compiled()) is not None:
        out = fast.linear_backward(dt, dy, z, x, w, _act(act), bool(want_dx), bool(want_dw), bool(want_dbias), dx, dw, dbias,
                                   workspace, _device(), _stream(None))
        if out is not None:
            return out
    _here(where, "dy", dy, stream)
    M, N = dy.shape
    dev = dy.device
    if not (want_dx or want_dw or want_dbias):
        raise ValueError(f"{where}: no output wanted")
    if (want_dx and w is None) or (want_dw and x is None) or (_act(act) and z is None):
        raise ValueError(f"{where}: dx needs w, dw needs x, an activation needs z")
    if (dx is not None and not want_dx) or (dw is not None and not want_dw) or (dbias is not None and not want_dbias):
        raise ValueError(f"{where}: an output is given that is not wanted")
    K = w.shape[1] if w is not None else x.shape[1] if x is not None else 32    # (dbias alone: of no consequence)
    for name, v, shape in (("dy", dy, (M, N)), ("z", z, (M, N)), ("x", x, (M, K)), ("w", w, (N, K)), ("dx", dx, (M, K)),
                           ("dw", dw, (N, K))):
        if v is not None and not _fits(v, shape, t, dev):
            _want(f"{where}: {name}", v, shape, t, dev)
    if dbias is not None:
        _want(f"{where}: dbias", dbias, (N,), torch.float32, dev)
    with _on(stream, dev):
        dx = (dy.new_empty((M, K)) if dx is None else dx) if want_dx else None
        dw = (dy.new_empty((N, K)) if dw is None else dw) if want_dw else None
        if want_dbias and dbias is None:
            dbias = dy.new_empty((N,), dtype=torch.float32)
        if workspace is None:
            workspace = linear_backward_workspace(dt, M, N, K, act, want_dx, want_dw, want_dbias, dev)
        _check(load_library().gemm_linear_backward(dt, _ptr(dy), _ptr(z), _ptr(x), _ptr(w), _act(act), _ptr(dx), _ptr(dw),
                                                   _ptr(dbias), M, N, K, _ptr(workspace),
                                                   _workspace_bytes(where, workspace, dev), _stream(stream)), where)
    return dx, dw, dbias


# ---- norms around a block, with its gate and the residual ----

class NormGrads(typing.NamedTuple):
    """Outputs of gemm_norm_backward; None where there is none or it is not wanted."""
    dx: object = None
    dresidual: object = None
    dw_in: object = None
    db_in: object = None
    dgate: object = None
    dw_out: object = None
    db_out: object = None


def _norm(kind) -> int:
    return NORMS[kind] if isinstance(kind, str) else int(kind)


def _norm_args(where, t, shape, index, dev, w_in, b_in, w_out, b_out, gate, **rows) -> int:
    """Checks of the fp32 vectors over the columns, the gate and, by name, the [M, H] tensors; the gate's rows."""
    f32, vec = _types()[0], shape[1:]
    if not ((w_out is None or _is(w_out, f32, vec, index)) and (w_in is None or _is(w_in, f32, vec, index))
            and (b_out is None or _is(b_out, f32, vec, index)) and (b_in is None or _is(b_in, f32, vec, index))):
        for name, v in (("w_in", w_in), ("b_in", b_in), ("w_out", w_out), ("b_out", b_out)):
            if v is not None:
                _want(f"{where}: {name}", v, vec, f32, dev)
    for name in rows:
        v = rows[name]
        if v is not None and not _is(v, t, shape, index):
            _want(f"{where}: {name}", v, shape, t, dev)
    if gate is None:
        return 0
    gates = gate.shape[0]
    if not _is(gate, f32, (gates, shape[1]), index):
        _want(f"{where}: gate", gate, (gates, shape[1]), f32, dev)
    if not gates:    # (its data pointer is null, which would read as no gate)
        raise ValueError(f"{where}: a gate without rows")
    return gates


def gemm_norm(dtype, x, residual=None, scale=1.0, norm_in="none", w_in=None, b_in=None, gate=None, norm_out="rms",
              w_out=None, b_out=None, eps=1e-6, want_r=True, r=None, y=None, stream=None):
    """(r, y): r = scale * residual + gate * (norm_in(x) * w_in + b_in), y = norm_out(r) * w_out + b_out in one
    pass. x, residual [M, H]; norm_in, norm_out "none", "rms" or "layer"; w_*, b_* fp32 [H] or None (ones, zeros);
    gate fp32 [G, H], a row for each M / G rows of x, or None. y is None with norm_out "none"; with want_r=False r
    is not stored and None. r may be the residual or x, y may be x."""
    where = "gemm_norm"
    dt, t = _half(dtype)
    if stream is None and x.is_cuda and (fast := _compiled()) is not None:
        out = fast.norm(dt, x, residual, scale, _norm(norm_in), w_in, b_in, gate, _norm(norm_out), w_out, b_out, eps,
                        bool(want_r), r, y, _device(), _stream(None))
        if out is not None:
            return out
    M, H = shape = x.shape
    index, dev = x.get_device(), x.device
    if stream is not None or index < 0 or index != _device():
        _here(where, "x", x, stream)
    kin, kout = _norm(norm_in), _norm(norm_out)
    if (r is not None and not want_r) or (y is not None and not kout):
        raise ValueError(f"{where}: an output is given that is not computed")
    gates = _norm_args(where, t, shape, index, dev, w_in, b_in, w_out, b_out, gate, x=x, residual=residual, r=r, y=y)
    with _on(stream, dev):
        like = _types()[3]
        if want_r and r is None:
            r = like(x)
        if kout and y is None:
            y = like(x)
    status = load_library().gemm_norm(dt, x.data_ptr(), _ptr(residual), scale, kin, _ptr(w_in), _ptr(b_in), _ptr(gate),
                                      gates, kout, _ptr(w_out), _ptr(b_out), eps, _ptr(r), _ptr(y), M, H,
                                      _stream(stream))
    if status:
        _check(status, where)
    return r, y


def gemm_norm_backward_workspace_size(dtype, M: int, H: int, gates: int = 0) -> int:
    """Host-only: workspace bytes of gemm_norm_backward (gates: rows of the gate, 0 without one)."""
    return _size("gemm_norm_backward_workspace_size", _dt(dtype), M, H, gates)


def norm_backward_workspace(dtype, M: int, H: int, gates: int = 0, device="cuda"):
    """A device workspace for gemm_norm_backward (its contents need not be set)."""
    import torch

    return torch.empty(gemm_norm_backward_workspace_size(dtype, M, H, gates), dtype=torch.uint8, device=device)


def gemm_norm_backward(dtype, dy, dr, x, r, scale=1.0, norm_in="none", w_in=None, b_in=None, gate=None,
                       norm_out="rms", w_out=None, b_out=None, eps=1e-6, want_dx=True, want_dresidual=True,
                       want_params=True, dx=None, dresidual=None, workspace=None, stream=None) -> NormGrads:
    """Gradients of gemm_norm, called with the same arguments: dy is that of y (None with norm_out "none"), dr what
    reaches r by other ways (None: nothing), r as gemm_norm returned it (None with norm_out "none"). x may be None
    where neither the gate's gradient nor one through norm_in needs it. With want_params the gradients of the
    parameters that are given are computed, in fp32."""
    where = "gemm_norm_backward"
    dt, t = _half(dtype)
    if stream is None and getattr(dr if dy is None else dy, "is_cuda", False) and (fast := _compiled()) is not None:
        out = fast.norm_backward(dt, dy, dr, x, r, scale, _norm(norm_in), w_in, b_in, gate, _norm(norm_out), w_out, b_out,
                                 eps, bool(want_dx), bool(want_dresidual), bool(want_params), dx, dresidual, workspace,
                                 _device(), _stream(None))
        if out is not None:
            return NormGrads._make(out)
    lead = dy if dy is not None else dr
    if lead is None:
        raise ValueError(f"{where}: neither dy nor dr is given")
    M, H = shape = lead.shape
    index, dev = lead.get_device(), lead.device
    if stream is not None or index < 0 or index != _device():
        _here(where, "dr" if dy is None else "dy", lead, stream)
    if (dx is not None and not want_dx) or (dresidual is not None and not want_dresidual):
        raise ValueError(f"{where}: an output is given that is not computed")
    gates = _norm_args(where, t, shape, index, dev, w_in, b_in, w_out, b_out, gate, dy=dy, dr=dr, x=x, r=r, dx=dx,
                       dresidual=dresidual)
    with _on(stream, dev):
        like = _types()[3]
        if want_dx and dx is None:
            dx = like(lead)
        if want_dresidual and dresidual is None:
            dresidual = like(lead)
        grads = [like(v) if v is not None and want_params else None for v in (w_in, b_in, gate, w_out, b_out)]
        if workspace is None and any(g is not None for g in grads):
            workspace = norm_backward_workspace(dt, M, H, gates, dev)
        _check(load_library().gemm_norm_backward(dt, _ptr(dy), _ptr(dr), _ptr(x), _ptr(r), scale, _norm(norm_in),
                                                 _ptr(w_in), _ptr(b_in), _ptr(gate), gates, _norm(norm_out),
                                                 _ptr(w_out), eps, _ptr(dx), _ptr(dresidual), *map(_ptr, grads), M, H,
                                                 _ptr(workspace), _workspace_bytes(where, workspace, dev),
                                                 _stream(stream)), where)
    return NormGrads(dx, dresidual, *grads)


# ---- mixture-of-experts layer for a few tokens ----

class MoeWeights:
    """Laid-out experts' weights (gemm_moe_preshuffle): the device buffer and what it holds."""

    __slots__ = ("data", "dtype", "E", "F", "H", "device", "gp_dtype")

    def __init__(self, data, dtype, gp_dtype, E, F, H):
        self.data, self.dtype, self.gp_dtype = data, dtype, gp_dtype
        self.E, self.F, self.H, self.device = E, F, H, data.device


def gemm_moe_weights_size(E: int, F: int, H: int) -> int:
    """Host-only: bytes of the laid-out weights of E experts."""
    return _size("gemm_moe_weights_size", E, F, H)


def gemm_moe_preshuffle(w13, w2, dtype, out=None, stream=None) -> MoeWeights:
    """w13 [E, 2F, H] (an expert's F gate rows, then its F up rows) and w2 [E, H, F] -> MoeWeights."""
    import torch

    where = "gemm_moe_preshuffle"
    dt, t = _half(dtype)
    _here(where, "w13", w13, stream)
    E, F2, H = w13.shape
    F = F2 // 2
    _want(f"{where}: w13", w13, (E, 2 * F, H), t)
    _want(f"{where}: w2", w2, (E, H, F), t, w13.device)
    n = gemm_moe_weights_size(E, F, H)
    with _on(stream, w13.device):
        out = torch.empty(n, dtype=torch.uint8, device=w13.device) if out is None else out
        _want(f"{where}: out", out, (n,), torch.uint8, w13.device)
        _check(load_library().gemm_moe_preshuffle(dt, _ptr(w13), _ptr(w2), _ptr(out), E, F, H, _stream(stream)), where)
    return MoeWeights(out, t, dt, E, F, H)


def gemm_moe_workspace_size(dtype, M: int, F: int, H: int, E: int, k: int) -> int:
    """Host-only: workspace bytes of gemm_moe, gemm_moe_route (any F) and gemm_moe_experts."""
    return _size("gemm_moe_workspace_size", _dt(dtype), M, F, H, E, k)


def moe_workspace(M: int, k: int, weights: MoeWeights):
    """A device workspace for M tokens with k experts each on these weights, its counters zero. Zero once here;
    every call leaves its counters zero again. Calls that may overlap need one each."""
    return _split_workspace(gemm_moe_workspace_size(weights.gp_dtype, M, weights.F, weights.H, weights.E, k), weights.device)


def _moe_route_args(where, t, x, router, bias, M, H, E, k, ids, gates):
    """Checks of a router's arguments; ids and gates, made where they are not given."""
    import torch

    dev = x.device
    _want(f"{where}: x", x, (M, H), t, dev)
    _want(f"{where}: router", router, (E, H), t, dev)
    if bias is not None:
        _want(f"{where}: bias", bias, (E,), torch.float32, dev)
    ids = torch.empty(M, k, dtype=torch.int32, device=dev) if ids is None else ids
    gates = torch.empty(M, k, dtype=torch.float32, device=dev) if gates is None else gates
    _want(f"{where}: ids", ids, (M, k), torch.int32, dev)
    _want(f"{where}: gates", gates, (M, k), torch.float32, dev)
    return ids, gates


def _score(score) -> int:
    return SCORES[score] if isinstance(score, str) else int(score)


def gemm_moe_route(dtype, x, router, k: int, bias=None, score="softmax", normalize=True, scale=1.0, ids=None, gates=None,
                   workspace=None, stream=None):
    """(ids int32 [M, k], gates fp32 [M, k]): the k experts of largest score (+ bias fp32 [E]) of x's rows, by falling
    score, and their weights. x [M, H], router [E, H]; score "softmax" or "sigmoid"; normalize: the weights of a token
    add up to scale. Without a workspace (gemm_moe_workspace_size) one is made for the call."""
    where = "gemm_moe_route"
    dt, t = _half(dtype)
    _here(where, "x", x, stream)
    (M, H), E = x.shape, router.shape[0]
    with _on(stream, x.device):
        ids, gates = _moe_route_args(where, t, x, router, bias, M, H, E, k, ids, gates)
        if workspace is None:
            workspace = _split_workspace(gemm_moe_workspace_size(dt, M, 16, H, E, k), x.device)
        _check(load_library().gemm_moe_route(dt, _ptr(x), _ptr(router), _ptr(bias), _score(score), int(normalize), scale,
                                             _ptr(ids), _ptr(gates), M, H, E, k, _ptr(workspace),
                                             _workspace_bytes(where, workspace, x.device), _stream(stream)), where)
    return ids, gates


def _moe_experts_args(where, t, x, weights, residual, y, M):
    if weights.dtype is not t:
        raise ValueError(f"{where}: the weights are {weights.dtype}")
    for name, v in (("x", x), ("residual", residual), ("y", y)):
        if v is not None:
            _want(f"{where}: {name}", v, (M, weights.H), t, weights.device)


def gemm_moe_experts(dtype, x, weights: MoeWeights, ids, gates, act="silu", residual=None, y=None, workspace=None,
                     stream=None):
    """y = residual + sum over j of gates[m, j] * (act(x Wg^T) * (x Wu^T)) Wd^T with expert ids[m, j]'s weights: x and
    residual [M, H], ids int32 [M, k] (outside [0, E): adds nothing), gates fp32 [M, k]. y may be the residual."""
    import torch

    where = "gemm_moe_experts"
    dt, t = _half(dtype)
    _here(where, "x", x, stream)
    M, k = ids.shape
    _moe_experts_args(where, t, x, weights, residual, y, M)
    _want(f"{where}: ids", ids, (M, k), torch.int32, x.device)
    _want(f"{where}: gates", gates, (M, k), torch.float32, x.device)
    with _on(stream, x.device):
        y = x.new_empty((M, weights.H)) if y is None else y
        if workspace is None:
            workspace = moe_workspace(M, k, weights)
        _check(load_library().gemm_moe_experts(dt, _ptr(x), _ptr(weights.data), _ptr(ids), _ptr(gates), _act(act),
                                               _ptr(residual), _ptr(y), M, weights.F, weights.H, weights.E, k,
                                               _ptr(workspace), _workspace_bytes(where, workspace, x.device),
                                               _stream(stream)), where)
    return y


def gemm_moe(dtype, x, router, weights: MoeWeights, k: int, bias=None, score="softmax", normalize=True, scale=1.0,
             act="silu", residual=None, y=None, ids=None, gates=None, workspace=None, stream=None):
    """(y, ids, gates): gemm_moe_route, then gemm_moe_experts on what it chose. Up to 256 tokens, 32 experts each and 4096
    pairs of them. Without a workspace (moe_workspace) one is made for the call."""
    where = "gemm_moe"
    dt, t = _half(dtype)
    _here(where, "x", x, stream)
    M, E, F, H = x.shape[0], weights.E, weights.F, weights.H
    _moe_experts_args(where, t, x, weights, residual, y, M)
    with _on(stream, x.device):
        ids, gates = _moe_route_args(where, t, x, router, bias, M, H, E, k, ids, gates)
        y = x.new_empty((M, H)) if y is None else y
        if workspace is None:
            workspace = moe_workspace(M, k, weights)
        _check(load_library().gemm_moe(dt, _ptr(x), _ptr(router), _ptr(bias), _score(score), int(normalize), scale,
                                       _ptr(weights.data), _act(act), _ptr(residual), _ptr(y), _ptr(ids), _ptr(gates), M, F,
                                       H, E, k, _ptr(workspace), _workspace_bytes(where, workspace, x.device),
                                       _stream(stream)), where)
    return y, ids, gates


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
