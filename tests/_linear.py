"""References in 64 bits and error bounds for the linear layer with its epilogue and its backward pass (the same
steps as tests/_ffn.py counts: fp32 accumulation, the activations' own errors, half a step of each rounding)."""
from __future__ import annotations

from tests import _ffn as F64

E = 2.0 ** -24


def forward64(x, w, bias, act, residual):
    """((y, error), (z, error)) before rounding, float64."""
    z, ez = F64.product64(x.double(), w.double())
    if bias is not None:
        z = z + bias.double()
        ez = ez + E * (z.abs() + bias.double().abs())
    v, _ = F64.act64(act, z)
    # |act'| < 1.2 for each activation
    ev = 1.2 * ez + F64._ACT_REL * v.abs() + (0.5 * F64._ERF * z.abs() if act == "gelu" else 0)
    if residual is not None:
        v = v + residual.double()
        ev = ev + E * (v.abs() + residual.double().abs())
    return (v, ev), (z, ez)


def dz64(dtype, dy, z, act):
    """(dz, error before rounding, error after it) in float64."""
    import torch

    d = dy.double()
    if act == "none":
        return d, torch.zeros_like(d), torch.zeros_like(d)
    N = dy.shape[1]
    g, eg = F64.gate_grad64(dtype, dy, z, torch.ones_like(dy), act)
    g, eg = g[:, :N], eg[:, :N]
    hs, tiny = F64.half_step(dtype)
    return g, (eg - hs * g.abs() - tiny) / (1 + hs), eg


def backward64(dtype, dy, z, x, w, act):
    """{dx, dw, dbias: (value, error before its own rounding)}."""
    M = dy.shape[0]
    d, e32, e16 = dz64(dtype, dy, z, act)
    return {"dx": F64.product64(d, w.double().t(), e16), "dw": F64.product64(d.t(), x.double().t(), e16.t()),
            "dbias": (d.sum(0), (e32 + (M + 64) * E * d.abs()).sum(0))}
