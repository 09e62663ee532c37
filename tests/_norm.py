"""References in 64 bits and error bounds for the norms around a block and their
backward pass.

The bounds count half a step of each rounding to 16 bits and fp32 steps at
E = 2^-24 each. A row's sums run over at most 16 values in a lane, 6 steps of a
tree over the wave and 16 waves: 40 additions deep (D), whatever H. Sums over
rows are at most M + 64 deep (a workgroup's rows, then the workgroups')."""
from __future__ import annotations

E = 2.0 ** -24
D = 40 * E


def norm64(kind, v, ev, eps):
    """(n, reciprocal root, error of n, relative error of the root) of rows v +- ev, all float64."""
    if kind == "layer":
        mean = v.mean(1, keepdim=True)
        em = D * v.abs().mean(1, keepdim=True) + ev.mean(1, keepdim=True)
        v = v - mean
        ev = ev + em + E * v.abs()
    s = (v * v).mean(1, keepdim=True) + eps
    rs = s.rsqrt()
    er = 0.5 * D + (v.abs() * ev).mean(1, keepdim=True) / s + 4 * E
    n = v * rs
    return n, rs, rs * ev * (1 + er) + n.abs() * (er + 2 * E), er


def grad64(kind, d, ed, n, en, rs, er):
    """Gradient through a norm of a gradient d +- ed of its normalised rows, and its error."""
    def mean(a):
        return a.mean(1, keepdim=True)
    along, ea = mean(d * n), D * mean((d * n).abs()) + mean(ed * n.abs() + (d.abs() + ed) * en)
    mid, em = (mean(d), D * mean(d.abs()) + mean(ed)) if kind == "layer" else (0 * along, 0 * along)
    inner = d - mid - n * along
    ei = ed + em + en * (along.abs() + ea) + n.abs() * ea + 4 * E * (d.abs() + mid.abs() + (n * along).abs())
    return rs * inner, rs * ei * (1 + er) + (rs * inner).abs() * (er + 2 * E)


def rows_of(gate, M):
    return gate.double().repeat_interleave(M // gate.shape[0], dim=0)


def vec(v, other, like):
    import torch

    return torch.full((1, like.shape[1]), other, dtype=torch.float64, device=like.device) if v is None else v.double()


def forward64(x, residual, scale, norm_in, w_in, b_in, gate, norm_out, w_out, b_out, eps):
    """((r, error), (y, error)) before their rounding; y (None, None) without norm_out."""
    import torch

    M = x.shape[0]
    v = x.double()
    w, b = vec(w_in, 1.0, v), vec(b_in, 0.0, v)
    g = torch.ones_like(v) if gate is None else rows_of(gate, M)
    n, en = (v, torch.zeros_like(v)) if norm_in == "none" else norm64(norm_in, v, torch.zeros_like(v), eps)[::2]
    R = torch.zeros_like(v) if residual is None else scale * residual.double()
    r = g * (n * w + b) + R
    er = en * (g * w).abs() + 4 * E * ((g * n * w).abs() + (g * b).abs() + R.abs())
    if norm_out == "none":
        return (r, er), (None, None)
    n, _, en, _ = norm64(norm_out, r, er, eps)
    wo, bo = vec(w_out, 1.0, v), vec(b_out, 0.0, v)
    return (r, er), (n * wo + bo, en * wo.abs() + 2 * E * ((n * wo).abs() + bo.abs()))


def backward64(dy, dr, x, r, scale, norm_in, w_in, b_in, gate, norm_out, w_out, b_out, eps):
    """{output: (value, error)} before rounding: dx, dresidual and the gradients of the parameters."""
    import torch

    lead = dr if dy is None else dy
    M, H = lead.shape
    zero = torch.zeros(M, H, dtype=torch.float64, device=lead.device)
    depth = (M + 64) * E
    out = {}

    def total(v, ev, groups=1):
        return (v.view(groups, -1, H).sum(1), (ev + (depth + E) * v.abs()).view(groups, -1, H).sum(1))
    t, et = (zero, zero) if dr is None else (dr.double(), zero)
    if norm_out != "none":
        n, rs, en, er = norm64(norm_out, r.double(), zero, eps)
        g = dy.double()
        w = vec(w_out, 1.0, zero)
        d, ed = g * w, E * (g * w).abs()
        back, eb = grad64(norm_out, d, ed, n, en, rs, er)
        out["dw_out"] = tuple(v[0] for v in total(g * n, g.abs() * en))
        out["db_out"] = tuple(v[0] for v in total(g, zero))
        et = eb + 2 * E * (back.abs() + t.abs())
        t = t + back
    out["dresidual"] = (scale * t, abs(scale) * (et + E * t.abs()))
    n, en, rs, er = (zero if x is None else x.double()), zero, None, None
    if norm_in != "none":
        n, rs, en, er = norm64(norm_in, n, zero, eps)
    G = 1 if gate is None else gate.shape[0]
    gv = torch.ones_like(zero) if gate is None else rows_of(gate, M)
    w, b = vec(w_in, 1.0, zero), vec(b_in, 0.0, zero)
    T1, e1 = total(t * n, t.abs() * en + et * (n.abs() + en), G)
    T0, e0 = total(t, et, G)
    out["dgate"] = (w * T1 + b * T0, w.abs() * e1 + b.abs() * e0 + 4 * E * ((w * T1).abs() + (b * T0).abs()))
    gg = torch.ones(1, H, dtype=torch.float64, device=zero.device) if gate is None else gate.double()
    out["dw_in"] = ((gg * T1).sum(0), (gg.abs() * (e1 + depth * T1.abs())).sum(0))
    out["db_in"] = ((gg * T0).sum(0), (gg.abs() * (e0 + depth * T0.abs())).sum(0))
    e = t * gv * w
    ee = et * (gv * w).abs() + 3 * E * e.abs()
    out["dx"] = (e, ee) if norm_in == "none" else grad64(norm_in, e, ee, n, en, rs, er)
    return out


def within32(got, ref, err, where):
    """|got - ref| <= err for fp32 outputs (err counts their rounding too)."""
    import torch

    g = got.double()
    assert g.shape == ref.shape, where
    assert bool(torch.isfinite(g).all()), f"{where}: not finite"
    bound = err + E * ref.abs() + 2.0 ** -140
    worst = float(((g - ref).abs() / bound).max())
    assert worst <= 1.0, f"{where}: {worst:.3g} of the bound"
    return worst
