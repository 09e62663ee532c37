"""Argument checks of the norms around a block (host only: every call fails validation, or is a size query)."""
import ctypes
import os

import pytest

import dense_gemm_preshuffle_amd as gp

OK, EINVAL, ESHAPE, EDTYPE, EWORKSPACE = 0, 1, 2, 3, 6
BF16, F16, FP8 = gp.DTYPES["bf16"], gp.DTYPES["fp16"], gp.DTYPES["fp8"]
P = ctypes.c_void_p(0x100000)     # aligned, never dereferenced: validation fails first
MIS = ctypes.c_void_p(0x100004)
NONE, RMS, LAYER = 0, 1, 2


@pytest.fixture
def lib():
    if os.path.exists("/dev/kfd"):
        pytest.skip("fake-pointer validation tests run on hosts without a GPU")
    return gp.load_library()


def test_exports():
    for n in ("gemm_norm", "gemm_norm_backward", "gemm_norm_backward_workspace_size"):
        assert n in gp.header_functions() and n in gp.__all__ and hasattr(gp.load_library(), n)
    assert gp.NORMS == {"none": NONE, "rms": RMS, "layer": LAYER}


def test_sizes():
    def size(M, H, gates, dtype=BF16):
        n = ctypes.c_size_t(123)
        return gp.load_library().gemm_norm_backward_workspace_size(dtype, M, H, gates, ctypes.byref(n)), n.value
    assert size(100, 4096, 0)[0] == size(1, 8, 1, F16)[0] == size(2 ** 31 - 1, 16384, 0)[0] == size(512, 8, 256)[0] == OK
    assert size(0, 8, 0)[0] == size(-1, 8, 0)[0] == size(4, 0, 0)[0] == size(4, 8, -1)[0] == EINVAL
    assert size(4, 8, 0, FP8)[0] == EDTYPE
    for bad in ((4, 12, 0), (4, 16392, 0), (2 ** 31, 8, 0), (4, 8, 3), (514, 8, 257), (4, 2 ** 40, 0)):
        assert size(*bad)[0] == ESHAPE, bad
    assert gp.load_library().gemm_norm_backward_workspace_size(BF16, 4, 8, 0, None) == EINVAL
    # one part per workgroup, each within one gate row
    for M, H, G in ((1, 8, 0), (16384, 4096, 8), (4096, 16384, 256), (777, 7168, 777 // 3), (130, 2048, 130)):
        n = size(M, H, G)[1] // (16 * H)
        assert n % max(G, 1) == 0 and n <= max(2048, G)


def test_forward_arguments(lib):
    def call(dtype=BF16, x=P, res=P, kin=RMS, w_in=P, b_in=P, gate=P, gates=1, kout=RMS, w_out=P, b_out=P, eps=1e-6,
             r=P, y=P, M=4, H=12):
        return lib.gemm_norm(dtype, x, res, 1.0, kin, w_in, b_in, gate, gates, kout, w_out, b_out, eps, r, y, M, H, None)
    assert call() == ESHAPE                                            # (H = 12: everything before it passes)
    assert call(x=None) == call(r=None, y=None) == call(y=None) == EINVAL
    assert call(kin=3) == call(kin=-1) == call(kout=3) == EINVAL
    assert call(kin=NONE) == call(kin=NONE, w_in=None) == call(kin=NONE, b_in=None) == EINVAL
    assert call(kin=NONE, w_in=None, b_in=None) == ESHAPE
    assert call(kout=NONE, y=None) == call(kout=NONE, w_out=None, b_out=None) == EINVAL
    assert call(kout=NONE, w_out=None, b_out=None, y=None) == ESHAPE
    assert call(gate=None) == call(gates=0) == call(gates=-1) == EINVAL
    assert call(eps=-1.0) == call(eps=float("nan")) == EINVAL
    for name in ("x", "res", "w_in", "b_in", "gate", "w_out", "b_out", "r", "y"):
        assert call(**{name: MIS}) == EINVAL, name
    assert call(dtype=FP8, H=8) == EDTYPE and call(gates=3, H=8) == ESHAPE and call(M=0, H=8) == EINVAL


def test_backward_arguments(lib):
    def call(dtype=BF16, dy=P, dr=P, x=P, r=P, kin=RMS, w_in=P, b_in=P, gate=P, gates=1, kout=RMS, w_out=P, eps=1e-6,
             dx=P, dres=P, dw_in=P, db_in=P, dgate=P, dw_out=P, db_out=P, ws=P, n=1 << 30, H=12):
        return lib.gemm_norm_backward(dtype, dy, dr, x, r, 1.0, kin, w_in, b_in, gate, gates, kout, w_out, eps, dx, dres,
                                      dw_in, db_in, dgate, dw_out, db_out, 4, H, ws, n, None)
    assert call() == ESHAPE
    assert call(dy=None) == call(dy=None, dr=None) == call(x=None) == call(r=None) == EINVAL
    none = dict(dx=None, dres=None, dw_in=None, db_in=None, dgate=None, dw_out=None, db_out=None)
    assert call(**none) == EINVAL
    assert call(kin=NONE) == call(kin=NONE, w_in=None, b_in=None) == call(kin=NONE, dw_in=None, db_in=None) == EINVAL
    assert call(kin=NONE, w_in=None, b_in=None, dw_in=None, db_in=None) == ESHAPE
    assert call(kout=NONE) == call(kout=NONE, dy=None, w_out=None) == EINVAL
    assert call(kout=NONE, dy=None, r=None, w_out=None, dw_out=None, db_out=None) == ESHAPE
    assert call(gate=None) == call(gate=None, gates=0) == call(eps=-1.0) == EINVAL
    assert call(gate=None, gates=0, dgate=None) == ESHAPE
    # x is needed for the gate's gradient, dw_in and, through a norm, dx
    assert call(x=None, dgate=None, dw_in=None, dx=None) == ESHAPE
    assert call(x=None, dgate=None, dw_in=None) == call(x=None, dgate=None, dx=None) == EINVAL
    for name in ("dy", "dr", "x", "r", "w_in", "b_in", "gate", "w_out", "ws", *none):
        assert call(**{name: MIS}) == EINVAL, name
    assert call(H=8, ws=None) == call(H=8, n=64) == EWORKSPACE
    assert call(H=8, dtype=FP8) == EDTYPE


def test_binding_refuses_host_tensors():
    import torch

    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    for f in (lambda: gp.gemm_norm("bf16", x), lambda: gp.gemm_norm_backward("bf16", x, None, x, x),
              lambda: gp.gemm_norm_backward("bf16", None, None, x, x)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(gp.GemmError):
        gp.gemm_norm("fp8", x)
