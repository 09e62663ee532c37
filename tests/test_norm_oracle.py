"""The 64-bit reference of the norms' backward pass against differences of the forward's (CPU)."""
import pytest

from tests import _norm as N


@pytest.mark.parametrize("norm_in,norm_out,G", [("none", "rms", 0), ("rms", "layer", 1), ("layer", "rms", 3),
                                                ("layer", "none", 2), ("none", "layer", 6)])
def test_backward_against_differences(norm_in, norm_out, G):
    import torch

    gen = torch.Generator().manual_seed(7)
    M, H, eps, scale = 6, 16, 1e-3, 0.75

    def normal(*s, mean=0.0):
        return torch.randn(*s, generator=gen, dtype=torch.float64) + mean
    p = {"x": normal(M, H), "residual": normal(M, H)}
    if norm_in != "none":
        p["w_in"], p["b_in"] = normal(H, mean=1.0), normal(H)
    if norm_out != "none":
        p["w_out"], p["b_out"] = normal(H, mean=1.0), normal(H)
    if G:
        p["gate"] = normal(G, H)
    dr, dy = normal(M, H), normal(M, H) if norm_out != "none" else None

    def run(q):
        (r, _), (y, _) = N.forward64(q["x"], q["residual"], scale, norm_in, q.get("w_in"), q.get("b_in"), q.get("gate"),
                                     norm_out, q.get("w_out"), q.get("b_out"), eps)
        return r, y

    def loss(q):
        r, y = run(q)
        return float((r * dr).sum()) + (float((y * dy).sum()) if y is not None else 0.0)
    r = run(p)[0]
    got = N.backward64(dy, dr, p["x"], r, scale, norm_in, p.get("w_in"), p.get("b_in"), p.get("gate"), norm_out,
                       p.get("w_out"), p.get("b_out"), eps)
    h = 1e-5
    for name in p:
        g = got["d" + name][0].reshape(-1)
        for k in range(0, p[name].numel(), 5):
            ends = []
            for step in (h, -h):
                q = {n: v.clone() for n, v in p.items()}
                q[name].view(-1)[k] += step
                ends.append(loss(q))
            diff = (ends[0] - ends[1]) / (2 * h)
            # central differences: h^2 times a third derivative of order 100, and the loss's rounding over h
            assert abs(diff - float(g[k])) < 1e-6, (name, k)
