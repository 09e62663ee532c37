"""The sublayer example runs, and its gradients are those of the sublayer in float64."""
import importlib.util
import os

import pytest

from tests._parity import say

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sublayer.py")
    spec = importlib.util.spec_from_file_location("sublayer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_runs():
    import torch

    out = _example().main(hidden=256, inner=512, tokens=256, steps=3)
    assert len(out["losses"]) == 3 and all(v == v for v in out["losses"])
    assert bool(torch.isfinite(out["y"]).all()) and sorted(out["ids"][0].tolist()) != [] and out["ids"].shape == (1, 2)


def test_gradients():
    """Each gradient against float64 autograd, normwise."""
    import torch

    s = _example().Sublayer(256, 512, 300, seed=4)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    x, residual, dy = (torch.randn(300, 256, generator=gen, device="cuda").bfloat16() for _ in range(3))
    s.forward(x, residual)
    (dx, dres), (dw, d_down, d_bias, d_norm) = s.backward(dy)
    p = [v.double().requires_grad_() for v in (x, residual, s.w, s.down, s.bias, s.w_norm)]
    r = p[0] + p[1]
    n = r * (r * r).mean(1, keepdim=True).add(1e-6).rsqrt() * p[5]
    z = n @ p[2].t()
    h = torch.nn.functional.silu(z[:, :512]) * z[:, 512:]
    (r + h @ p[3].t() + p[4]).backward(dy.double())
    for name, got, ref in zip(("dx", "dresidual", "dw", "d_down", "d_bias", "d_norm"), (dx, dres, dw, d_down, d_bias, d_norm),
                              (v.grad for v in p)):
        err = float((got.double() - ref).norm() / ref.norm())
        say(f"example gradient {name}: {err:.2e}")
        # up to 8 roundings to bf16 on the way (r, n, h, gate, up, dh, dg and du, dn, itself), half a step 2^-9 each
        # (a uniform error of that size: over sqrt(3)), which add up as squares, twice for the products' spread
        assert err <= 2 * (8 / 3) ** 0.5 * 2.0 ** -8
