"""Argument checks of the 4-bit products (host only: every call fails
validation, or is a size query)."""
import ctypes
import os

import pytest

import dense_gemm_preshuffle_amd as gp

OK, EINVAL, ESHAPE, EDTYPE = 0, 1, 2, 3
BF16, F16, FP8 = gp.DTYPES["bf16"], gp.DTYPES["fp16"], gp.DTYPES["fp8"]
P = ctypes.c_void_p(0x100000)     # aligned, never dereferenced: validation fails first
Q = ctypes.c_void_p(0x40000000)
MIS = ctypes.c_void_p(0x100008)


@pytest.fixture
def lib():
    if os.path.exists("/dev/kfd"):
        pytest.skip("fake-pointer validation tests run on hosts without a GPU")
    return gp.load_library()


def size(N, K, group, zeros=0, gated=0):
    n = ctypes.c_size_t(77)
    return gp.load_library().gemm_w4a16_weights_size(N, K, group, zeros, gated, ctypes.byref(n)), n.value


def test_exports():
    for n in ("gemm_w4a16_weights_size", "gemm_w4a16_preshuffle", "gemm_w4a16", "gemm_w4a16_gated"):
        assert n in gp.header_functions() and n in gp.__all__ and hasattr(gp.load_library(), n)


def test_sizes():
    assert size(16, 128, 128) == (OK, 1024 + 256)
    assert size(16, 128, 128, 1) == (OK, 1024 + 256 + 256)
    assert size(1, 32, 128) == (OK, 1024 + 256)                 # padded to one block
    assert size(17, 160, 32) == (OK, 2 * 2 * 1024 + 512)        # 2 x 2 blocks of 64 scales
    assert size(2, 128, 128, 0, 1)[1] == size(32, 128, 128)[1]  # a gate and an up block
    assert size(4096, 4096, 1 << 30) == (OK, 4096 * 2048 + 4096 * 2)   # a scale per output
    assert gp.gemm_w4a16_weights_size(4096, 4096, 128, True) == 4096 * 2048 + 4096 * 32 * 3
    for bad in ((0, 32, 32), (4, 0, 32), (4, 32, 0), (-1, 32, 32), (4, 32, -32)):
        assert size(*bad)[0] == EINVAL, bad
    for bad in ((4, 48, 32), (4, 32, 16), (4, 96, 96), (4, 64, 33), (4, 1 << 23, 128), (1 << 31, 32, 32),
                (1 << 30, 1 << 22, 128), (2 ** 62, 32, 32), (4, 2 ** 62, 32)):
        assert size(*bad)[0] == ESHAPE, bad
    assert size(3, 32, 32, 0, 1)[0] == ESHAPE                   # gate rows and up rows
    assert gp.load_library().gemm_w4a16_weights_size(4, 32, 32, 0, 0, None) == EINVAL


def test_preshuffle_pointers(lib):
    def call(q=P, s=P, z=None, w=Q, dtype=BF16, N=32, K=64, group=32, gated=0):
        return lib.gemm_w4a16_preshuffle(dtype, q, s, z, w, N, K, group, gated, None)
    assert call(q=None) == call(s=None) == call(w=None) == EINVAL
    assert call(q=MIS) == call(s=MIS) == call(z=MIS) == call(w=MIS) == EINVAL
    assert call(w=P) == call(q=Q) == EINVAL                                    # overlap
    assert call(s=ctypes.c_void_p(0x40000000 + 16)) == call(z=ctypes.c_void_p(0x40000000 - 16)) == EINVAL
    assert call(dtype=FP8) == EDTYPE and call(K=48) == ESHAPE and call(group=48) == ESHAPE
    assert call(N=31, gated=1) == ESHAPE and call(N=0) == EINVAL


def test_product_pointers(lib):
    def call(x=P, w=P, bias=None, act=0, y=P, M=4, N=32, K=64, group=32, dtype=BF16):
        return lib.gemm_w4a16(dtype, x, w, 0, bias, act, y, M, N, K, group, None)
    assert call(x=None) == call(w=None) == call(y=None) == EINVAL
    assert call(x=MIS) == call(w=MIS) == call(y=MIS) == call(bias=MIS) == EINVAL
    assert call(M=0) == call(M=-1) == call(N=0) == call(act=-1) == call(act=4) == EINVAL
    assert call(dtype=FP8) == EDTYPE
    assert call(K=48) == call(group=24) == call(M=1 << 31) == call(N=1 << 31) == call(M=1 << 30, N=1 << 20) == ESHAPE

    def gated(x=P, w=P, act=2, h=P, M=4, F=32, K=64, group=32, dtype=F16):
        return lib.gemm_w4a16_gated(dtype, x, w, 0, act, h, M, F, K, group, None)
    assert gated(x=None) == gated(w=None) == gated(h=None) == gated(h=MIS) == gated(act=7) == gated(F=0) == EINVAL
    assert gated(dtype=FP8) == EDTYPE and gated(K=40) == gated(F=2 ** 62) == ESHAPE
