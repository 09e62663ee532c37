"""Random sizes through the gated product, both backward passes and the 4-bit products, against float64: whatever
kernel the plans choose, with and without a workspace of the caller's."""
import random

import pytest

from tests import _ffn as F64
from tests import _w4
from tests._parity import say

pytestmark = pytest.mark.gpu


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _case(rng):
    """An operator and sizes of at most 3e10 products, rows from one on."""
    while True:
        op = rng.choice(["gated", "gated_backward", "gated_backward", "backward", "backward", "w4", "w4_gated"])
        c = {"op": op, "dtype": rng.choice(F64.TYPES), "act": rng.choice(F64.ACTS), "M": _log(rng, 1, 4000),
             "K": 32 * _log(rng, 1, 200)}
        if op == "gated" or op == "gated_backward":
            c["N"] = 16 * _log(rng, 1, 400)
        elif op == "backward":
            c["N"] = 32 * _log(rng, 1, 400)
        else:
            c["M"] = _log(rng, 1, 100)
            c["N"], c["group"], c["zeros"] = _log(rng, 1, 12000), rng.choice([32, 64, 128, 256]), rng.choice([False, True, "wide"])
        if c["M"] * c["N"] * c["K"] <= 3e10:
            return c


def _product_with_error(d, ed, b):
    return F64.product64(d, b.double().t().contiguous(), ed)


@pytest.mark.parametrize("seed", range(120))
def test_random(seed):
    import torch

    import dense_gemm_preshuffle_amd as gp

    c = _case(random.Random(7000 + seed))
    say("ffn random", c)
    op, dtype, act, M, N, K = (c[k] for k in ("op", "dtype", "act", "M", "N", "K"))
    t = F64.torch_type(dtype)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    normal = lambda *s, scale=1.0: (torch.randn(*s, generator=gen, device="cuda") * scale).to(t)
    x = normal(M, K)
    if op == "gated":
        w = normal(2 * N, K, scale=K ** -0.5)
        outs = [F64.guarded(M, N, t) for _ in range(3)]
        h, gate, up = (v for v, _ in outs)
        gp.gemm_gated(dtype, x, gp.gemm_gated_preshuffle(w, dtype), act=act, save=True, h=h, gate=gate, up=up)
        torch.cuda.synchronize()
        refs, errs = F64.gated64(x, w, act)
        for name, got, ref, err in zip(("h", "gate", "up"), (h, gate, up), refs, errs):
            F64.within(dtype, got, ref, err, name)
        assert all(ok() for _, ok in outs)
    elif op in ("gated_backward", "backward"):
        gated = op == "gated_backward"
        rows = 2 * N if gated else N
        b = normal(rows, K, scale=rows ** -0.5)
        da, ok_a = F64.guarded(M, K, t)
        db, ok_b = F64.guarded(rows, K, t)
        if gated:
            dh, gate, up = normal(M, N, scale=0.1), normal(M, N), normal(M, N)
            gp.gemm_gated_backward(dtype, dh, gate, up, x, b, act=act, dx=da, dw=db)
            d, ed = F64.gate_grad64(dtype, dh, gate, up, act)
        else:
            dc = normal(M, N, scale=0.1)
            gp.gemm_backward(dtype, dc, x, b, da=da, db=db)
            d, ed = dc.double(), 0.0
        torch.cuda.synchronize()
        F64.within(dtype, da, *_product_with_error(d, ed, b), "da")
        F64.within(dtype, db, *_product_with_error(d.t().contiguous(), ed if isinstance(ed, float) else ed.t().contiguous(), x),
                   "db")
        assert ok_a() and ok_b()
    else:
        gated = op == "w4_gated"
        q, v, s, z = _w4.make(gen, dtype, 2 * N if gated else N, K, c["group"], c["zeros"])
        w = gp.gemm_w4a16_preshuffle(q, s, z, group=c["group"], gated=gated)
        ref, err = _w4.product64("bf16", x, v, s, z, c["group"])   # (both types' magnitudes, see _w4)
        g, eg = (ref[:, :N], err[:, :N]) if gated else (ref, err)
        a, _ = F64.act64(act, g)
        ea = 1.2 * eg + 2.0 ** -20 * a.abs() + (0.8e-7 * g.abs() if act == "gelu" else 0)
        if gated:
            u, eu = ref[:, N:], err[:, N:]
            a, ea = a * u, ea * u.abs() + (a.abs() + ea) * eu + 2.0 ** -23 * (a * u).abs()
        for ws in (None, gp.w4a16_workspace(M, w)):
            y, ok = F64.guarded(M, N, t)
            if gated:
                gp.gemm_w4a16_gated(x, w, act=act, h=y, workspace=ws)
            else:
                gp.gemm_w4a16(x, w, act=act, y=y, workspace=ws)
            torch.cuda.synchronize()
            F64.within(dtype, y, a, ea, f"workspace {ws is not None}")
            assert ok()
