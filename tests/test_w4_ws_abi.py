"""Argument checks of the 4-bit products with a workspace (host only)."""
import ctypes
import os

import pytest

import dense_gemm_preshuffle_amd as gp

OK, EINVAL, ESHAPE, EDTYPE, EWORKSPACE = 0, 1, 2, 3, 6
BF16, FP8 = gp.DTYPES["bf16"], gp.DTYPES["fp8"]
P = ctypes.c_void_p(0x100000)     # aligned, never dereferenced: validation fails first
MIS = ctypes.c_void_p(0x100008)


def size(M, N, K, group=128, gated=0):
    n = ctypes.c_size_t(77)
    return gp.load_library().gemm_w4a16_workspace_size(M, N, K, group, gated, ctypes.byref(n)), n.value


def test_exports():
    for n in ("gemm_w4a16_ws", "gemm_w4a16_workspace_size"):
        assert n in gp.header_functions() and hasattr(gp.load_library(), n)
    assert "w4a16_workspace" in gp.__all__


def test_sizes():
    assert size(1, 4096, 4096) == (OK, 0)                 # a workgroup per CU
    assert size(1, 64, 256) == (OK, 0)                    # short K
    status, n = size(64, 392, 19520)
    assert status == OK and n > 65536
    assert gp.gemm_w4a16_workspace_size(64, 392, 19520, 128) == n
    assert size(1, 512, 1 << 20)[1] > 65536 and size(40, 200, 16384, 64, 1)[1] > 65536
    for bad in ((0, 32, 64), (-1, 32, 64), (4, 0, 64), (4, 32, 0)):
        assert size(*bad)[0] == EINVAL, bad
    for bad in ((4, 32, 48), (1 << 31, 32, 64), (4, 1 << 31, 64), (4, 32, 1 << 23), (4, 32, 64, 24)):
        assert size(*bad)[0] == ESHAPE, bad
    assert gp.load_library().gemm_w4a16_workspace_size(1, 32, 64, 32, 0, None) == EINVAL


def test_pointers():
    if os.path.exists("/dev/kfd"):
        pytest.skip("fake-pointer validation tests run on hosts without a GPU")
    lib = gp.load_library()

    def call(x=P, w=P, bias=None, act=0, y=P, M=64, N=392, K=19520, gated=0, ws=P, n=1 << 30, dtype=BF16):
        return lib.gemm_w4a16_ws(dtype, x, w, 0, bias, act, y, M, N, K, 128, gated, ws, n, None)
    assert call(x=None) == call(w=None) == call(y=MIS) == call(ws=MIS) == call(act=5) == EINVAL
    assert call(ws=None) == call(n=64) == call(n=0) == EWORKSPACE
    assert call(gated=1, bias=P) == EINVAL
    assert call(dtype=FP8) == EDTYPE and call(K=40) == ESHAPE
