"""The backward products on row-major operands, tile by tile, and the plans beside them."""
import pytest

from tests import _ffn as F64
from tests._parity import say

pytestmark = pytest.mark.gpu


def _gen(seed):
    import torch

    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(gen, *shape, t, scale=1.0):
    import torch

    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(t)


# M x N x K of C = A B^T: rows around 64, K axes that end inside a tile and a
# group of 8 rows, every tile size, with and without a K split, sizes below the
# tiles, and edge tiles in both directions
LINEAR = [(63, 128, 128), (64, 128, 128), (65, 192, 160), (71, 4096, 288), (100, 512, 2048), (129, 1024, 96), (130, 4160, 2048),
          (257, 320, 1056), (500, 2048, 1024), (515, 8192, 512), (1000, 4096, 4096), (1027, 96, 4096), (2049, 4128, 1120),
          (4099, 256, 256), (4100, 4160, 4128)]


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear(dtype, M, N, K):
    import torch

    import dense_gemm_preshuffle_amd as gp

    t = F64.torch_type(dtype)
    gen = _gen(M + 2 * N + K)
    dc, a, b = _normal(gen, M, N, t=t), _normal(gen, M, K, t=t), _normal(gen, N, K, t=t, scale=K ** -0.5)
    say(f"backward rows {dtype} {M}x{N}x{K}")
    ws = gp.backward_workspace(dtype, M, N, K)
    ws.fill_(255)
    outs = [F64.guarded(M, K, t), F64.guarded(N, K, t)]
    gp.gemm_backward(dtype, dc, a, b, da=outs[0][0], db=outs[1][0], workspace=ws)
    torch.cuda.synchronize()
    x = F64.within(dtype, outs[0][0], *F64.product64(dc.double(), b.double().t()), "da")
    y = F64.within(dtype, outs[1][0], *F64.product64(dc.double().t(), a.double().t()), "db")
    say("  shares of the bounds", round(x, 3), round(y, 3))
    assert all(ok() for _, ok in outs), "written outside the outputs"
    da, db = gp.gemm_backward(dtype, dc, a, b, workspace=ws)
    assert torch.equal(da, outs[0][0]) and torch.equal(db, outs[1][0])


@pytest.mark.parametrize("dtype", F64.TYPES)
def test_rows_do_not_mix(dtype):
    """A row of dc that is not finite changes its row of da alone; a column, its row of db alone."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    t, (M, N, K) = F64.torch_type(dtype), (201, 320, 288)
    gen = _gen(9)
    dc, a, b = _normal(gen, M, N, t=t), _normal(gen, M, K, t=t), _normal(gen, N, K, t=t)
    da, db = gp.gemm_backward(dtype, dc, a, b)
    for row, col in ((0, 0), (M - 1, N - 1), (77, 130)):
        bad = dc.clone()
        bad[row, col] = float("inf")
        da2, db2 = gp.gemm_backward(dtype, bad, a, b)
        torch.cuda.synchronize()
        keep = torch.arange(M, device="cuda") != row
        assert torch.equal(da2[keep], da[keep]) and not bool(torch.isfinite(da2[row]).all())
        keep = torch.arange(N, device="cuda") != col
        assert torch.equal(db2[keep], db[keep]) and not bool(torch.isfinite(db2[col]).all())


GATED = [(64, 64, 128), (100, 272, 160), (129, 2064, 2048), (300, 528, 1056), (1001, 1040, 4096), (2050, 4112, 512)]


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,F,H", GATED)
def test_gated(dtype, M, F, H):
    import torch

    import dense_gemm_preshuffle_amd as gp

    t = F64.torch_type(dtype)
    gen = _gen(M + 3 * F + H)
    x, w = _normal(gen, M, H, t=t), _normal(gen, 2 * F, H, t=t, scale=H ** -0.5)
    gate, up, dh = _normal(gen, M, F, t=t), _normal(gen, M, F, t=t), _normal(gen, M, F, t=t)
    act = F64.ACTS[(M + F // 16 + H // 32) % 4]
    say(f"gated backward rows {dtype} {M}x{F}x{H} {act}")
    ws = gp.gated_backward_workspace(dtype, M, F, H)
    ws.fill_(255)
    dx, dw = gp.gemm_gated_backward(dtype, dh, gate, up, x, w, act=act, workspace=ws)
    torch.cuda.synchronize()
    d, ed = F64.gate_grad64(dtype, dh, gate, up, act)
    F64.within(dtype, dx, *F64.product64(d, w.double().t(), ed), "dx")
    F64.within(dtype, dw, *F64.product64(d.t(), x.double().t(), ed.t()), "dw")
    assert torch.equal(gp.gemm_gated_backward(dtype, dh, gate, up, None, w, act=act, want_dw=False)[0], dx)
    assert torch.equal(gp.gemm_gated_backward(dtype, dh, gate, up, x, None, act=act, want_dx=False)[1], dw)


def test_workspace_of_another_size():
    """A larger workspace serves a smaller call (its contents need not be set)."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    gen = _gen(2)
    ws = torch.full((gp.gemm_backward_workspace_size("bf16", 1000, 4096, 4096),), 255, dtype=torch.uint8, device="cuda")
    for M, N, K in ((130, 4160, 2048), (40, 512, 1024), (1000, 4096, 4096)):
        t = torch.bfloat16
        dc, a, b = _normal(gen, M, N, t=t), _normal(gen, M, K, t=t), _normal(gen, N, K, t=t, scale=K ** -0.5)
        if gp.gemm_backward_workspace_size("bf16", M, N, K) > ws.numel():
            continue
        da, db = gp.gemm_backward("bf16", dc, a, b, workspace=ws)
        torch.cuda.synchronize()
        F64.within("bf16", da, *F64.product64(dc.double(), b.double().t()), "da")
        F64.within("bf16", db, *F64.product64(dc.double().t(), a.double().t()), "db")
