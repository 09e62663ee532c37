"""Argument checks and plans of the linear layer with its epilogue (host only)."""
import ctypes
import math
import os
import random
import re

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
    for n in ("gemm_linear_preshuffle", "gemm_linear", "gemm_linear_workspace_size", "gemm_linear_plan",
              "gemm_linear_backward", "gemm_linear_backward_workspace_size"):
        assert n in gp.header_functions() and n in gp.__all__ and hasattr(gp.load_library(), n)


def test_sizes():
    f = "gemm_linear_workspace_size"
    assert size(f, BF16, 100, 1024, 512)[0] == size(f, F16, 1, 16, 32)[0] == OK
    for bad in ((0, 32, 32), (-1, 32, 32), (4, 0, 32), (4, 32, 0)):
        assert size(f, BF16, *bad)[0] == EINVAL
    assert size(f, FP8, 4, 32, 32)[0] == EDTYPE
    assert size(f, BF16, 4, 32, 48)[0] == OK
    for bad in ((4, 24, 32), (4, 32, 40), (2 ** 31, 32, 32), (4, 2 ** 31, 32), (4, 32, 2 ** 31), (2 ** 62, 2 ** 62, 32),
                (2 ** 20, 32, 2 ** 20), (32, 2 ** 20, 2 ** 20), (2 ** 20, 2 ** 20, 32)):
        assert size(f, BF16, *bad)[0] == ESHAPE, bad
    assert gp.load_library().gemm_linear_workspace_size(BF16, 4, 32, 32, None) == EINVAL
    assert gp.load_library().gemm_linear_plan(BF16, 4, 32, 32, None) == EINVAL


def test_backward_sizes():
    f = "gemm_linear_backward_workspace_size"

    def n(act=2, dx=1, dw=1, db=1, M=512, N=1024, K=512):
        s, v = size(f, BF16, M, N, K, act, dx, dw, db)
        assert s == OK
        return v
    assert n() > n(act=0) > n(act=0, db=0) == size("gemm_backward_workspace_size", BF16, 512, 1024, 512, 1, 1)[1]
    assert n(db=0) - n(act=0, db=0) == 512 * 1024 * 2          # dz
    assert n(act=0, N=1040, db=0) == n(act=2, N=1040, db=0)    # a copy of dy filled up to whole blocks
    assert n(dx=0, dw=0) < n(dw=0)
    assert size(f, BF16, 4, 32, 32, 0, 0, 0, 0)[0] == size(f, BF16, 4, 32, 32, 4, 1, 1, 1)[0] == EINVAL
    assert size(f, BF16, 4, 48, 32, 0, 1, 1, 1)[0] == size(f, BF16, 4, 48, 32, 0, 0, 0, 1)[0] == OK
    assert size(f, BF16, 4, 40, 32, 0, 1, 1, 1)[0] == size(f, BF16, 4, 48, 40, 2, 0, 0, 1)[0] == ESHAPE
    assert size(f, FP8, 4, 32, 32, 0, 1, 1, 1)[0] == EDTYPE


def test_backward_workspace_of_an_activation_serves_none():
    """A workspace for any activation holds a call without one, at sizes where the two run on other plans too."""
    f = "gemm_linear_backward_workspace_size"
    rng = random.Random(7)
    cases = [(F16, 3677, 4064, 14304, 1, 1, 1), (F16, 3870, 3808, 9376, 1, 1, 1)]
    while len(cases) < 12000:
        M = int(math.exp(rng.uniform(0, math.log(16384))))
        N, K = (16 * int(math.exp(rng.uniform(0, math.log(1024)))) for _ in range(2))
        wants = rng.choice(((1, 1, 1), (1, 1, 0), (1, 0, 0), (0, 1, 0), (0, 1, 1), (1, 0, 1), (0, 0, 1)))
        cases.append((rng.choice((BF16, F16)), M, N, K, *wants))
    for c in cases:
        none = size(f, *c[:4], 0, *c[4:])
        assert none[0] == OK, c
        of = [size(f, *c[:4], act, *c[4:]) for act in (1, 2, 3)]
        assert all(s == OK and n >= none[1] for s, n in of) and len(set(of)) == 1, (c, none, of)


def test_forward_arguments(lib):
    def call(dtype=BF16, x=P, w=P, bias=P, act=2, res=P, y=P, z=P, M=4, N=32, K=40, ws=None):
        return lib.gemm_linear(dtype, x, w, bias, act, res, y, z, M, N, K, ws, 0, None)
    assert call() == ESHAPE                                            # (K = 40: everything before it passes)
    assert call(x=None) == call(w=None) == call(y=None) == call(act=-1) == call(act=4) == EINVAL
    for name in ("x", "w", "bias", "res", "y", "z"):
        assert call(**{name: MIS}) == EINVAL, name
    assert call(dtype=FP8, K=32) == EDTYPE and call(N=24, K=32) == ESHAPE
    assert size("gemm_linear_workspace_size", BF16, 512, 1024, 8192)[1] > 0
    assert call(M=512, N=1024, K=8192) == EWORKSPACE


def test_preshuffle_arguments(lib):
    f = lib.gemm_linear_preshuffle
    assert f(None, P, 32, 32, BF16, None) == f(P, None, 32, 32, BF16, None) == f(P, MIS, 32, 32, BF16, None) == EINVAL
    assert f(P, ctypes.c_void_p(0x100000 + 2032), 32, 32, BF16, None) == EINVAL     # overlap
    assert f(P, Q, 24, 32, BF16, None) == f(P, Q, 32, 24, BF16, None) == ESHAPE
    assert f(P, Q, 32, 32, FP8, None) == EDTYPE


def test_backward_arguments(lib):
    def call(dy=P, z=P, x=P, w=P, act=2, dx=P, dw=P, db=P, ws=P, n=1 << 30, dtype=BF16, N=32):
        return lib.gemm_linear_backward(dtype, dy, z, x, w, act, dx, dw, db, 4, N, 32, ws, n, None)
    assert call(dy=None) == call(z=None) == call(dx=None, dw=None, db=None) == call(x=None) == call(w=None) == EINVAL
    for name in ("dy", "z", "x", "w", "dx", "dw", "db", "ws"):
        assert call(**{name: MIS}) == EINVAL, name
    assert call(act=9) == call(act=-1) == EINVAL
    assert call(ws=None) == call(n=64) == EWORKSPACE
    assert call(dtype=FP8) == EDTYPE and call(N=40) == ESHAPE


def test_plans_are_compiled_and_all_reached():
    """Every plan names a compiled variant, and every compiled variant is some plan's."""
    root = os.path.dirname(gp.__file__)
    text = open(os.path.join(root, "csrc", "variants.hpp")).read()

    def listed(macro):
        body = re.search(rf"#define {macro}\(X, DT\)(.*?)\n(?!  X)", text, re.S).group(1)
        return {tuple(v.strip() for v in m.split(",")) for m in re.findall(r"X\(DT, ([^)]*)\)", body)}
    tiles = {(int(a), int(b), c == "true") for a, b, c in listed("GP_TILE_LINEAR")}
    small = {tuple(map(int, v)) for v in listed("GP_SMALL_LINEAR")}
    rng, seen_small, seen = random.Random(5), set(), set()
    for _ in range(12000):
        M, N, K = (max(lo, int(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))
                   for lo, hi in ((1, 16384), (1, 2000), (1, 512)))
        try:
            p = gp.gemm_linear_plan(rng.choice(("bf16", "fp16")), M, 16 * N, 32 * K)
        except gp.GemmError:
            continue                                        # too large
        assert p["workspace_bytes"] == gp.gemm_linear_workspace_size("bf16", M, 16 * N, 32 * K)
        assert (p["workspace_bytes"] > 0) == (p["ksplit"] > 1)
        if p["kernel"] == gp.KERNEL_SPLITK:
            seen_small.add((p["tile_m"] // 8, p["tile_n"] // 16, p["waves"], p["tile_k"] // 64))
        else:
            assert p["kernel"] == gp.KERNEL_TILE and p["tile_m"] <= M and p["tile_n"] <= 16 * N
            seen.add((p["tile_m"], p["tile_n"], p["ksplit"] > 1))
    assert seen_small == small and seen == tiles
