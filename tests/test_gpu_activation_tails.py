"""The activations of the feed-forward and 4-bit products at every magnitude: products that are single numbers,
against float64, relative to the value where it is small."""
import pytest

from tests import _ffn as F64
from tests._parity import say

pytestmark = pytest.mark.gpu

# Relative error of an activation or its derivative before rounding. The largest part is the exponent's: g^2 / 2 or
# g, up to 96 where results still are numbers of the type, through three fp32 roundings: 3 * 2^-24 * 96 < 2^-15.7;
# 2^-15 leaves 2^-16.1 for some ten other roundings and the 1 ulp of the reciprocal and the exponential.
_REL = 2.0 ** -15


def _points(dtype, low, high, n):
    """n values of the type, evenly spaced."""
    import torch

    return torch.linspace(low, high, n, dtype=torch.float64, device="cuda").to(F64.torch_type(dtype))


def _smallest(dtype):
    """What is below the type's normal numbers may be rounded in their step: half of fp16's subnormal step, and for
    bf16 (whose subnormals fp32 arithmetic may drop) its smallest normal number."""
    import torch

    return 2.0 ** -25 if dtype == "fp16" else float(torch.finfo(torch.bfloat16).smallest_normal)


def _close(dtype, got, ref, extra, where):
    """|got - ref| <= half a step and _REL of |ref|, extra and the smallest step."""
    import torch

    hs, _ = F64.half_step(dtype)
    assert bool(torch.isfinite(got).all()), where
    bound = ((1 + hs) * (1 + _REL) - 1) * ref.abs() + extra + _smallest(dtype)
    share = (got.double() - ref).abs() / bound
    say(f"  {where}: {float(share.max()):.3f} of the bound")
    assert float(share.max()) <= 1.0, (where, int(share.argmax()))


LOW = {"gelu": -13.0, "silu": -96.0}


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M", [1, 24, 64, 65, 320])     # one row, few, the small kernel's last, tiles
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_gated(act, M, dtype):
    """Row m: gate p[m, f], up 1, by weights that copy: h is the activation of p."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    F, H, t = 128, 256, F64.torch_type(dtype)
    p = _points(dtype, LOW[act], 6.0, M * F)[torch.randperm(M * F, device="cuda")].view(M, F)
    x = torch.cat((p, torch.ones(M, H - F, dtype=t, device="cuda")), 1)
    w = torch.zeros(2 * F, H, dtype=t, device="cuda")
    w[:F, :F] = torch.eye(F, device="cuda")
    w[F:, F] = 1
    h = gp.gemm_gated(dtype, x, gp.gemm_gated_preshuffle(w, dtype), act=act)
    torch.cuda.synchronize()
    _close(dtype, h, F64.act64(act, p.double())[0], 0.0, f"gated {dtype} {act} M {M}")


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_gated_backward(act, dtype):
    """dh = up = 1 and weights that copy dg or du to dx: the derivative and the activation."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    M, F, t = 200, 64, F64.torch_type(dtype)
    p = _points(dtype, LOW[act], 6.0, M * F).view(M, F)
    one = torch.ones_like(p)
    value, slope = F64.act64(act, p.double())
    for name, ref, row in (("dg", slope, 0), ("du", value, F)):
        w = torch.zeros(2 * F, F, dtype=t, device="cuda")
        w[row:row + F] = torch.eye(F, device="cuda")
        dx, _ = gp.gemm_gated_backward(dtype, one, p, one, None, w, act=act, want_dw=False)
        torch.cuda.synchronize()
        # the derivative is a difference near its zero: the error of its two parts, each below 0.3 there
        extra = 2.0 ** -20 * ((p.abs() < 3).double()) if name == "dg" else 0.0
        _close(dtype, dx, ref, extra, f"{name} {dtype} {act}")


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M", [1, 3, 16, 40])
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_w4(act, M, dtype):
    """Integers 1 at one K per column, scale 1: y is the activation of x's element."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    K, t = 256, F64.torch_type(dtype)
    q = torch.zeros(K, K // 2, dtype=torch.uint8, device="cuda")
    k = torch.arange(K, device="cuda")
    q[k, k // 2] = torch.where(k % 2 == 0, 1, 16).to(torch.uint8)
    w = gp.gemm_w4a16_preshuffle(q, torch.ones(K, 2, dtype=t, device="cuda"), group=128)
    # one element that is not 0 in each row: the integers are exact, so is their sum
    pts = _points(dtype, LOW[act], -0.5, M)
    x = torch.zeros(M, K, dtype=t, device="cuda")
    x[torch.arange(M, device="cuda"), 7 * torch.arange(M, device="cuda") % K] = pts
    y = gp.gemm_w4a16(x, w, act=act)
    torch.cuda.synchronize()
    _close(dtype, y, F64.act64(act, x.double())[0], 0.0, f"w4 {dtype} {act} M {M}")
