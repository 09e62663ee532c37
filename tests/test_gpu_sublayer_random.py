"""Random sizes and arguments through the linear layer, the norms and the experts against float64."""
import math
import random

import pytest

from tests import _ffn as F64
from tests import _linear as L64
from tests import _moe as M64
from tests import _norm as N64
from tests._parity import say

pytestmark = pytest.mark.gpu


def _log(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def _draw(seed):
    import torch

    rng = random.Random(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = rng.choice(F64.TYPES)
    t = F64.torch_type(dtype)
    return rng, dtype, t, lambda *s, scale=1.0, mean=0.0: torch.randn(*s, generator=gen, device="cuda") * scale + mean


@pytest.mark.parametrize("seed", range(40))
def test_linear(seed):
    import torch

    import dense_gemm_preshuffle_amd as gp

    rng, dtype, t, normal = _draw(seed)
    M = _log(rng, 1, 64) if rng.random() < 0.5 else _log(rng, 65, 3000)
    N, K = _log(rng, 16, 4096, 16), _log(rng, 16, 4096, 16)
    act = rng.choice(F64.ACTS)
    x, w = normal(M, K).to(t), normal(N, K, scale=K ** -0.5).to(t)
    bias = normal(N) if rng.random() < 0.5 else None
    res = normal(M, N).to(t) if rng.random() < 0.6 else None
    say(f"seed {seed}: linear {dtype} {M}x{N}x{K} {act}")
    y, z = gp.gemm_linear(dtype, x, gp.gemm_linear_preshuffle(w, dtype), bias=bias, act=act, residual=res, save=True)
    ry, rz = L64.forward64(x, w, bias, act, res)
    F64.within(dtype, y, *ry, "y")
    F64.within(dtype, z, *rz, "z")
    dy = normal(M, N).to(t)
    got = gp.gemm_linear_backward(dtype, dy, None if act == "none" else z, x, w, act=act)
    torch.cuda.synchronize()
    ref = L64.backward64(dtype, dy, z, x, w, act)
    F64.within(dtype, got[0], *ref["dx"], "dx")
    F64.within(dtype, got[1], *ref["dw"], "dw")
    N64.within32(got[2], *ref["dbias"], "dbias")


@pytest.mark.parametrize("seed", range(100, 140))
def test_norm(seed):
    import torch

    import dense_gemm_preshuffle_amd as gp

    rng, dtype, t, normal = _draw(seed)
    G = rng.choice([0, 0, 1, rng.randint(2, 40)])
    M = max(G, 1) * _log(rng, 1, 3000 // max(G, 1))
    H = _log(rng, 8, 16384, 8)
    if M * H > 1 << 24:
        M = max(G, 1)
    kin, kout = rng.choice(["none", "rms", "layer"]), rng.choice(["none", "rms", "layer"])
    scale = rng.choice([1.0, 0.25, -1.5])

    def vec(on, mean):
        return normal(H, scale=0.3, mean=mean) if on and rng.random() < 0.7 else None
    kw = {"norm_in": kin, "w_in": vec(kin != "none", 1.0), "b_in": vec(kin != "none", 0.0), "gate": normal(G, H) if G else None,
          "norm_out": kout, "w_out": vec(kout != "none", 1.0), "b_out": vec(kout != "none", 0.0), "eps": 1e-5}
    say(f"seed {seed}: norm {dtype} {M}x{H} gates {G} {kin} -> {kout} scale {scale}")
    x, res = normal(M, H, mean=0.5).to(t), normal(M, H).to(t) if rng.random() < 0.7 else None
    r, y = gp.gemm_norm(dtype, x, residual=res, scale=scale, **kw)
    args = (kin, kw["w_in"], kw["b_in"], kw["gate"], kout, kw["w_out"], kw["b_out"], 1e-5)
    (rr, re), (yr, ye) = N64.forward64(x, res, scale, *args)
    F64.within(dtype, r, rr, re, "r")
    if y is not None:
        F64.within(dtype, y, yr, ye, "y")
    dy = normal(M, H).to(t) if kout != "none" else None
    dr = normal(M, H).to(t) if dy is None or rng.random() < 0.7 else None
    got = gp.gemm_norm_backward(dtype, dy, dr, x, r if dy is not None else None, scale=scale, **kw)
    torch.cuda.synchronize()
    ref = N64.backward64(dy, dr, x, r if dy is not None else None, scale, *args)
    for name, v in got._asdict().items():
        if v is not None:
            (N64.within32(v, *ref[name], name) if v.dtype == torch.float32 else F64.within(dtype, v, *ref[name], name))


@pytest.mark.parametrize("seed", range(200, 240))
def test_experts(seed):
    import torch

    import dense_gemm_preshuffle_amd as gp

    rng, dtype, t, normal = _draw(seed)
    M = 1 if rng.random() < 0.3 else _log(rng, 1, 256)
    E = _log(rng, 1, 200)
    k = rng.randint(1, min(E, 16))
    H, F = _log(rng, 32, 1500, 32), _log(rng, 16, 1500, 16)
    if E * H * F > 1 << 25:
        E, k = 4, min(k, 4)
    x, router = normal(M, H).to(t), normal(E, H, scale=H ** -0.5).to(t)
    w13, w2 = normal(E, 2 * F, H, scale=H ** -0.5).to(t), normal(E, H, F, scale=F ** -0.5).to(t)
    bias = normal(E, scale=0.1) if rng.random() < 0.4 else None
    res = normal(M, H).to(t) if rng.random() < 0.5 else None
    score, normalize, scale, act = rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5, rng.choice([1.0, 2.5]), rng.choice(F64.ACTS)
    say(f"seed {seed}: experts {dtype} {M} tokens, {k} of {E}, {H} x {F} {score} {act}")
    y, ids, gates = gp.gemm_moe(dtype, x, router, gp.gemm_moe_preshuffle(w13, w2, dtype), k, bias=bias, score=score,
                                normalize=normalize, scale=scale, act=act, residual=res)
    torch.cuda.synchronize()
    ri, rg = M64.route64(x, router, k, bias, score, normalize, scale)
    assert torch.equal(ids, ri)
    assert float(((gates.double() - rg).abs() / rg).max()) <= 2.0 ** -24 * (1 + 2.0 ** -20)
    F64.within(dtype, y, *M64.experts64(dtype, x, w13, w2, ids, gates, act, res), "y")
