"""Argument checks of the gated product and the backward passes (host only:
every call fails validation, or is a size query)."""
import ctypes
import os

import pytest

import dense_gemm_preshuffle_amd as gp

OK, EINVAL, ESHAPE, EDTYPE, EWORKSPACE = 0, 1, 2, 3, 6
BF16, F16, FP8 = gp.DTYPES["bf16"], gp.DTYPES["fp16"], gp.DTYPES["fp8"]
P = ctypes.c_void_p(0x100000)     # aligned, never dereferenced: validation fails first
Q = ctypes.c_void_p(0x40000000)
MIS = ctypes.c_void_p(0x100008)


@pytest.fixture
def lib():
    if os.path.exists("/dev/kfd"):
        pytest.skip("fake-pointer validation tests run on hosts without a GPU")
    return gp.load_library()


def size(fn, *args):
    n = ctypes.c_size_t(123)
    return getattr(gp.load_library(), fn)(*args, ctypes.byref(n)), n.value


def test_exports():
    names = gp.header_functions()
    for n in ("gemm_gated_preshuffle", "gemm_gated", "gemm_gated_workspace_size", "gemm_gated_backward",
              "gemm_gated_backward_workspace_size", "gemm_backward", "gemm_backward_workspace_size"):
        assert n in names and hasattr(gp.load_library(), n)
    for n in gp.__all__:
        assert hasattr(gp, n), n


@pytest.mark.parametrize("fn,extra", [("gemm_gated_workspace_size", ()),
                                      ("gemm_gated_backward_workspace_size", (1, 1)),
                                      ("gemm_backward_workspace_size", (1, 1))])
def test_sizes(fn, extra):
    assert size(fn, BF16, 100, 1024, 512, *extra)[0] == OK
    assert size(fn, F16, 1, 32, 32, *extra)[0] == OK
    for bad in ((0, 32, 32), (-1, 32, 32), (4, 0, 32), (4, 32, 0)):
        assert size(fn, BF16, *bad, *extra)[0] == EINVAL
    assert size(fn, FP8, 4, 32, 32, *extra)[0] == EDTYPE
    for bad in ((4, 24, 32), (4, 32, 48), (2 ** 31, 32, 32), (4, 2 ** 31, 32), (4, 32, 2 ** 31), (2 ** 62, 2 ** 62, 32),
                (2 ** 20, 32, 2 ** 20), (32, 2 ** 20, 2 ** 20), (2 ** 20, 2 ** 20, 32)):
        assert size(fn, BF16, *bad, *extra)[0] == ESHAPE, bad
    assert getattr(gp.load_library(), fn)(BF16, 4, 32, 32, *extra, None) == EINVAL


def test_backward_sizes():
    assert size("gemm_backward_workspace_size", BF16, 4, 48, 32, 1, 1)[0] == ESHAPE    # N % 32
    assert size("gemm_gated_backward_workspace_size", BF16, 4, 48, 32, 1, 1)[0] == OK  # 2F = 96
    for fn in ("gemm_backward_workspace_size", "gemm_gated_backward_workspace_size"):
        assert size(fn, BF16, 4, 32, 32, 0, 0)[0] == EINVAL
        both, one = size(fn, BF16, 512, 1024, 512, 1, 1)[1], size(fn, BF16, 512, 1024, 512, 1, 0)[1]
        assert both > one > 0


def test_gated_pointers(lib):
    def call(x=P, w=P, act=2, h=P, gate=None, up=None, dtype=BF16, M=4, F=32, H=32):
        return lib.gemm_gated(dtype, x, w, act, h, gate, up, M, F, H, None, 0, None)
    assert call(x=None) == call(w=None) == call(h=None) == call(x=MIS) == call(h=MIS) == EINVAL
    assert call(gate=P) == call(up=P) == call(gate=P, up=MIS) == EINVAL
    assert call(act=-1) == call(act=4) == EINVAL
    assert call(dtype=FP8) == EDTYPE and call(F=24) == ESHAPE and call(H=16) == ESHAPE
    # a plan that splits K needs a workspace
    assert size("gemm_gated_workspace_size", BF16, 512, 512, 8192)[1] > 0
    assert call(M=512, F=512, H=8192) == EWORKSPACE


def test_preshuffle_pointers(lib):
    f = lib.gemm_gated_preshuffle
    assert f(None, P, 32, 32, BF16, None) == f(P, None, 32, 32, BF16, None) == f(P, MIS, 32, 32, BF16, None) == EINVAL
    assert f(P, ctypes.c_void_p(0x100000 + 4080), 32, 32, BF16, None) == EINVAL     # overlap
    assert f(P, Q, 24, 32, BF16, None) == f(P, Q, 32, 16, BF16, None) == ESHAPE
    assert f(P, Q, 32, 32, FP8, None) == EDTYPE


def test_backward_pointers(lib):
    def gated(dh=P, gate=P, up=P, x=P, w=P, act=2, dx=P, dw=P, ws=P, n=1 << 30, dtype=BF16, F=32):
        return lib.gemm_gated_backward(dtype, dh, gate, up, x, w, act, dx, dw, 4, F, 32, ws, n, None)
    assert gated(dh=None) == gated(gate=None) == gated(up=None) == gated(dx=None, dw=None) == EINVAL
    assert gated(w=None) == gated(x=None) == EINVAL
    assert gated(dh=MIS) == gated(w=MIS) == gated(dw=MIS) == gated(ws=MIS) == gated(act=9) == EINVAL
    assert gated(ws=None) == gated(n=64) == EWORKSPACE
    assert gated(dtype=FP8) == EDTYPE and gated(F=24) == ESHAPE

    def linear(dc=P, a=P, b=P, da=P, db=P, ws=P, n=1 << 30, dtype=BF16, N=32):
        return lib.gemm_backward(dtype, dc, a, b, da, db, 4, N, 32, ws, n, None)
    assert linear(dc=None) == linear(da=None, db=None) == linear(a=None) == linear(b=None) == EINVAL
    assert linear(dc=MIS) == linear(a=MIS) == linear(ws=MIS) == EINVAL
    assert linear(ws=None) == linear(n=64) == EWORKSPACE
    assert linear(dtype=FP8) == EDTYPE and linear(N=48) == ESHAPE
