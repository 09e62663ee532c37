"""References in 64 bits and error bounds for the gated feed-forward product,
its backward pass and the linear backward pass.

The bounds count, per output: half a step of each rounding to 16 bits (hs =
eps / 2 relative, and half the smallest subnormal for fp16), fp32
accumulation of n products (n * 2^-24 of the sum of magnitudes, whatever the
order), and the activations' own errors (erf to 1.5e-7 absolute, exp, the
reciprocal and the fp32 steps around them to 2^-20 relative)."""
from __future__ import annotations

import math

TYPES = ("bf16", "fp16")
ACTS = ("silu", "gelu", "relu", "none")
_ACT_REL = 2.0 ** -20
_ERF = 1.5e-7


def torch_type(dtype):
    import torch

    return {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]


def half_step(dtype):
    """(relative half step, absolute half step at zero) of a 16-bit type."""
    import torch

    f = torch.finfo(torch_type(dtype))
    return f.eps / 2, f.smallest_normal * f.eps / 2


def act64(act, g):
    """act(g) and act'(g) in float64."""
    import torch

    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g)
    if act == "gelu":
        p = 0.5 * torch.special.erfc(-g * math.sqrt(0.5))
        return g * p, p + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    if act == "relu":
        return torch.relu(g), (g > 0).double()
    return g, torch.ones_like(g)


def gated64(x, w, act):
    """(h, gate, up), bounds of each before rounding: all float64."""
    F = w.shape[0] // 2
    xd, wd = x.double(), w.double()
    z = xd @ wd.t()
    e = (x.shape[1] + 8) * 2.0 ** -24 * (xd.abs() @ wd.abs().t())
    g, u, eg, eu = z[:, :F], z[:, F:], e[:, :F], e[:, F:]
    v, _ = act64(act, g)
    ev = 1.2 * eg + _ACT_REL * v.abs() + (0.5 * _ERF * g.abs() if act == "gelu" else 0)   # |act'| < 1.2
    eh = ev * u.abs() + (v.abs() + ev) * eu + 2.0 ** -23 * (v * u).abs()
    return (v * u, g, u), (eh, eg, eu)


def rounded(dtype, ref, err):
    """Bound after one rounding to the type of values ref +- err."""
    hs, tiny = half_step(dtype)
    return err + hs * (ref.abs() + err) + tiny


def gate_grad64(dtype, dh, gate, up, act):
    """([dg du], bound after their rounding) in float64."""
    import torch

    g, u, d = gate.double(), up.double(), dh.double()
    v, s = act64(act, g)
    es = 4 * _ACT_REL * (1 + g.abs()) * s.abs().clamp(max=1.2) + (_ERF if act == "gelu" else 0)
    if act == "silu":
        # s (1 + g (1 - s)): the error of 1 - s counts g times
        es = es + 4 * _ACT_REL * torch.sigmoid(g) * (1 + g.abs())
    if act in ("relu", "none"):
        es = torch.zeros_like(g)
    ev = _ACT_REL * v.abs() + (0.5 * _ERF * g.abs() if act == "gelu" else 0)
    dg, du = d * u * s, d * v
    eg = (d * u).abs() * es + 2.0 ** -22 * dg.abs()
    eu = d.abs() * ev + 2.0 ** -23 * du.abs()
    return torch.cat((dg, du), 1), torch.cat((rounded(dtype, dg, eg), rounded(dtype, du, eu)), 1)


def product64(a, b, ea=0.0):
    """a b^T and its bound: ea on a's entries, fp32 accumulation."""
    ref = a @ b.t()
    mag = a.abs() + ea
    err = (a.shape[1] + 8) * 2.0 ** -24 * (mag @ b.abs().t())
    if not isinstance(ea, float):
        err = err + ea @ b.abs().t()
    return ref, err


def within(dtype, got, ref, err, where):
    """|got - ref| <= the bound of a value ref +- err rounded to the type; prints the worst share."""
    import torch

    g = got.double()
    assert g.shape == ref.shape, where
    bound = rounded(dtype, ref, err)
    share = ((g - ref).abs() / bound)
    worst = float(share.max()) if share.numel() else 0.0
    assert bool(torch.isfinite(g).all()), f"{where}: not finite"
    assert worst <= 1.0, f"{where}: {worst:.3g} of the bound at {int(share.argmax())}"
    return worst


def guarded(n_rows, n_cols, dtype, fill=7.0):
    """A [rows, cols] tensor inside a larger filled buffer, and a check that nothing around it changed."""
    import torch

    pad = 4096
    n = n_rows * n_cols
    buf = torch.full((n + 2 * pad,), fill, dtype=dtype, device="cuda")
    view = buf[pad:pad + n].view(n_rows, n_cols)

    def untouched():
        return bool((buf[:pad] == fill).all()) and bool((buf[pad + n:] == fill).all())
    return view, untouched
