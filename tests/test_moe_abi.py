"""Argument checks of the mixture-of-experts layer (host only: every call fails validation, or is a size query)."""
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


def test_exports():
    for n in ("gemm_moe_weights_size", "gemm_moe_preshuffle", "gemm_moe_route", "gemm_moe_experts", "gemm_moe",
              "gemm_moe_workspace_size"):
        assert n in gp.header_functions() and n in gp.__all__ and hasattr(gp.load_library(), n)
    assert gp.SCORES == {"softmax": 0, "sigmoid": 1}


def test_weights_size():
    assert gp.gemm_moe_weights_size(8, 48, 96) == 8 * (4 * 48 * 128 + 2 * 96 * 64)
    lib, n = gp.load_library(), ctypes.c_size_t()

    def size(*a):
        return lib.gemm_moe_weights_size(*a, ctypes.byref(n))
    assert size(0, 16, 32) == size(1, 0, 32) == size(1, 16, 0) == lib.gemm_moe_weights_size(1, 16, 32, None) == EINVAL
    for bad in ((513, 16, 32), (1, 24, 32), (1, 16, 48), (1, 2 ** 28, 32), (1, 2 ** 40, 32), (1, 16, 2 ** 40), (1, 2 ** 18, 2 ** 14)):
        assert size(*bad) == ESHAPE, bad
    assert size(512, 14336, 4096) == OK and n.value == 512 * 6 * 14336 * 4096      # beyond 2^32 bytes together


def test_workspace_size():
    lib, n = gp.load_library(), ctypes.c_size_t()

    def size(M, F, H, E, k, dtype=BF16):
        return lib.gemm_moe_workspace_size(dtype, M, F, H, E, k, ctypes.byref(n))
    assert size(1, 1024, 2048, 64, 8) == size(256, 16, 32, 512, 16) == size(1, 16, 32, 1, 1, F16) == OK
    assert size(0, 16, 32, 4, 1) == size(1, 16, 32, 4, 0) == size(-1, 16, 32, 4, 1) == EINVAL
    assert lib.gemm_moe_workspace_size(BF16, 1, 16, 32, 4, 1, None) == EINVAL
    assert size(1, 16, 32, 4, 1, FP8) == EDTYPE
    for bad in ((257, 16, 32, 4, 1), (1, 16, 32, 4, 5), (1, 16, 32, 64, 33), (256, 16, 32, 64, 17), (1, 16, 2 ** 19, 4, 1)):
        assert size(*bad) == ESHAPE, bad


@pytest.mark.parametrize("inside,outside", [
    # (M, F, H, E, k): the last size on each side of a limit of the header
    ((256, 16, 32, 4, 1), (257, 16, 32, 4, 1)), ((128, 16, 32, 32, 32), (129, 16, 32, 32, 32)),
    ((256, 16, 32, 64, 16), (256, 16, 32, 64, 17)), ((4, 16, 32, 64, 32), (4, 16, 32, 64, 33)),
    ((4, 16, 32, 3, 3), (4, 16, 32, 3, 4)), ((4, 16, 32, 512, 1), (4, 16, 32, 513, 1)),
    ((1, 16, 258048, 4, 1), (1, 16, 258080, 4, 1)),
    ((256, 16, 131072 - 32, 64, 16), (256, 16, 131072, 64, 16)),                      # M k rows of 4 H bytes
    ((256, 2 ** 18 - 16, 32, 64, 16), (256, 2 ** 18, 32, 64, 16)),                    # and of 2 F
    ((1, 2 ** 23 - 16, 64, 4, 1), (1, 2 ** 23, 64, 4, 1)),                            # an expert's matrix
    ((64, 2 ** 17 - 16, 32, 512, 8), (64, 2 ** 17, 32, 512, 8)),                      # min(M k, E) F
    ((64, 16, 258048, 512, 1), (64, 16, 258080, 512, 1))])
def test_documented_limits(inside, outside):
    lib, n = gp.load_library(), ctypes.c_size_t()

    def size(M, F, H, E, k):
        return lib.gemm_moe_workspace_size(BF16, M, F, H, E, k, ctypes.byref(n))
    assert size(*inside) == OK and size(*outside) == ESHAPE


def test_arguments(lib):
    def route(dtype=BF16, x=P, wr=P, bias=P, score=0, ids=P, gates=P, M=2, H=48, E=8, k=2, ws=P, n=1 << 30):
        return lib.gemm_moe_route(dtype, x, wr, bias, score, 1, 1.0, ids, gates, M, H, E, k, ws, n, None)
    assert route() == ESHAPE                                           # (H = 48: everything before it passes)
    assert route(x=None) == route(wr=None) == route(ids=None) == route(gates=None) == EINVAL
    assert route(score=2) == route(score=-1) == EINVAL
    for name in ("x", "wr", "bias", "ids", "gates"):
        assert route(**{name: MIS}) == EINVAL, name
    assert route(H=64, ws=None) == route(H=64, n=65536) == EWORKSPACE and route(H=64, ws=MIS) == EINVAL
    assert route(H=64, dtype=FP8) == EDTYPE and route(H=64, k=9) == ESHAPE

    def experts(dtype=BF16, x=P, w=P, ids=P, gates=P, act=2, res=P, y=P, M=2, F=16, H=48, E=8, k=2, ws=P, n=1 << 30):
        return lib.gemm_moe_experts(dtype, x, w, ids, gates, act, res, y, M, F, H, E, k, ws, n, None)
    assert experts() == ESHAPE
    assert experts(x=None) == experts(w=None) == experts(ids=None) == experts(gates=None) == experts(y=None) == EINVAL
    assert experts(act=4) == experts(act=-1) == EINVAL
    for name in ("x", "w", "ids", "gates", "res", "y"):
        assert experts(**{name: MIS}) == EINVAL, name
    assert experts(H=64, ws=None) == experts(H=64, n=65536) == EWORKSPACE and experts(H=64, ws=MIS) == EINVAL

    def layer(**kw):
        a = dict(x=P, wr=P, w=P, res=P, y=P, ids=P, gates=P, act=2, score=0, H=64, ws=P, n=1 << 30)
        a.update(kw)
        return lib.gemm_moe(BF16, a["x"], a["wr"], None, a["score"], 1, 1.0, a["w"], a["act"], a["res"], a["y"], a["ids"],
                            a["gates"], 2, 16, a["H"], 8, 2, a["ws"], a["n"], None)
    assert layer(H=48) == ESHAPE
    for name in ("x", "wr", "w", "y", "ids", "gates"):
        assert layer(**{name: None}) == layer(**{name: MIS}) == EINVAL, name
    assert layer(act=9) == layer(score=5) == EINVAL and layer(ws=None) == layer(n=4) == EWORKSPACE

    def lay(w13=P, w2=Q, out=ctypes.c_void_p(0x80000000), dtype=BF16, F=16, H=32):
        return lib.gemm_moe_preshuffle(dtype, w13, w2, out, 8, F, H, None)
    assert lay(w13=None) == lay(w2=None) == lay(out=None) == lay(w13=MIS) == lay(out=MIS) == EINVAL
    assert lay(out=P) == lay(out=ctypes.c_void_p(0x40000010)) == EINVAL             # overlaps
    assert lay(dtype=FP8) == EDTYPE and lay(F=24) == lay(H=48) == ESHAPE
