"""Backward products whose output rows are so long that a tile's rows span more than 2^31 bytes."""
import pytest

from tests import _ffn as F64
from tests._parity import say

pytestmark = pytest.mark.gpu


# 32 or 2 rows of 2 K bytes: those that a 128-row tile has beyond them must be stored nowhere
@pytest.mark.parametrize("dtype,M,N,K", [("bf16", 2, 32, 8650752), ("fp16", 33, 64, 8454208)])
def test_rows_past_the_matrix(dtype, M, N, K):
    import torch

    import dense_gemm_preshuffle_amd as gp

    t = F64.torch_type(dtype)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M)
    normal = lambda *shape: torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(t)
    dc, a, b = normal(M, N), normal(M, K), normal(N, K)
    say(f"backward limits {dtype} {M}x{N}x{K}")
    da, ok_a = F64.guarded(M, K, t)
    db, ok_b = F64.guarded(N, K, t)
    gp.gemm_backward(dtype, dc, a, b, da=da, db=db)
    torch.cuda.synchronize()
    for k0 in range(0, K, 1 << 20):
        s = slice(k0, k0 + (1 << 20))
        F64.within(dtype, da[:, s], *F64.product64(dc.double(), b[:, s].double().t()), f"da {k0}")
        F64.within(dtype, db[:, s], *F64.product64(dc.double().t(), a[:, s].double().t()), f"db {k0}")
    assert ok_a() and ok_b(), "written outside the outputs"
