"""Backward passes whose first product, laid out for the preshuffled kernels, would split K and whose second would
not: both gradients, alone and together, against float64."""
import pytest

from tests import _ffn as F64
from tests._parity import say
from tests.test_backward_plans import SIZES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,N,K,gated", SIZES)
def test_both_and_each(dtype, M, N, K, gated):
    import torch

    import dense_gemm_preshuffle_amd as gp

    t = F64.torch_type(dtype)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M + N + K)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(t)
    say(f"backward plans {dtype} {M}x{N}x{K} gated {gated}")
    rows = 2 * N if gated else N
    a, b = normal(M, K), normal(rows, K)
    da, ok_a = F64.guarded(M, K, t)
    db, ok_b = F64.guarded(rows, K, t)
    if gated:
        dh, gate, up = normal(M, N), normal(M, N), normal(M, N)
        run = lambda **k: gp.gemm_gated_backward(dtype, dh, gate, up, a, b, **{{"da": "dx", "db": "dw", "want_da": "want_dx",
                                                                               "want_db": "want_dw"}[n]: v for n, v in k.items()})
        d, ed = F64.gate_grad64(dtype, dh, gate, up, "silu")
    else:
        dc = normal(M, N)
        run = lambda **k: gp.gemm_backward(dtype, dc, a, b, **k)
        d, ed = dc.double(), 0.0
    run(da=da, db=db)
    one_a, one_b = run(want_db=False)[0], run(want_da=False)[1]
    torch.cuda.synchronize()
    F64.within(dtype, da, *F64.product64(d, b.double().t().contiguous(), ed), "da")
    F64.within(dtype, db, *F64.product64(d.t().contiguous(), a.double().t().contiguous(), ed if isinstance(ed, float) else
                                         ed.t().contiguous()), "db")
    assert ok_a() and ok_b(), "written outside the outputs"
    assert torch.equal(one_a, da) and torch.equal(one_b, db)
