"""References in 64 bits and error bounds for the products with 4-bit weights.

Per output the bounds count half a step of the one rounding to 16 bits, and
fp32 accumulation of the products in whatever order, K + a few additions of
2^-24 of the sum of magnitudes. For bf16 the kernel accumulates x (q + 8) and
takes the group's sum of x times (8 + z) away, so the magnitudes are those of
both parts: |x| s (q + 8 + |8 + z|)."""
from __future__ import annotations

from tests import _ffn as F64


def integers(gen, N, K, lo=-8, hi=8):
    """Packed 4-bit integers [N, K/2] and their values [N, K] (int8)."""
    import torch

    v = torch.randint(lo, hi, (N, K), device="cuda", generator=gen, dtype=torch.int8)
    return ((v[:, 0::2] & 15) | (v[:, 1::2] << 4)).view(torch.uint8), v


def make(gen, dtype, N, K, group, zeros):
    """(q packed, values, scales, zeros) with every integer and wide zero points."""
    import torch

    q, v = integers(gen, N, K)
    groups = -(-K // group)
    s = ((torch.rand(N, groups, device="cuda", generator=gen) + 0.5) * (0.4 * K ** -0.5)).to(F64.torch_type(dtype))
    z = torch.randint(-128, 128, (N, groups), device="cuda", generator=gen, dtype=torch.int8) if zeros == "wide" else \
        torch.randint(-3, 4, (N, groups), device="cuda", generator=gen, dtype=torch.int8) if zeros else None
    return q, v, s, z


def spread(t, group, K):
    return t.double().repeat_interleave(group, dim=1)[:, :K]


def product64(dtype, x, v, s, z, group):
    """(y, its bound before rounding) in float64."""
    K = v.shape[1]
    zd = spread(z, group, K) if z is not None else 0.0
    sd = spread(s, group, K)
    xd, vd = x.double(), v.double()
    ref = xd @ (sd * (vd - zd)).t()
    if dtype == "bf16":
        mag = sd * (vd + 8 + (8 + zd).abs() if z is not None else vd + 16)
    else:
        mag = sd * (vd - zd).abs()
    return ref, (K + 24) * 2.0 ** -24 * (xd.abs() @ mag.t())
