"""Backward products smaller than a tile, and K ranges that differ in length."""
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


# rows and columns below every tile; long K axes whose tiles no split divides
@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,N,K", [(1, 64, 32), (2, 128, 64), (7, 64, 4096), (31, 13568, 352), (33, 3968, 2752), (40, 64, 32),
                                   (53, 6208, 96), (63, 1024, 1056), (195, 13504, 352), (606, 9792, 448), (1000, 64, 64),
                                   (3999, 320, 288), (2000, 14336, 544), (127, 8256, 32)])
def test_linear(dtype, M, N, K):
    import torch

    import dense_gemm_preshuffle_amd as gp

    t = F64.torch_type(dtype)
    gen = _gen(M + 5 * N + K)
    dc, a, b = _normal(gen, M, N, t=t), _normal(gen, M, K, t=t), _normal(gen, N, K, t=t, scale=K ** -0.5)
    say(f"backward small {dtype} {M}x{N}x{K}")
    ws = gp.backward_workspace(dtype, M, N, K)
    ws.fill_(255)
    outs = [F64.guarded(M, K, t), F64.guarded(N, K, t)]
    gp.gemm_backward(dtype, dc, a, b, da=outs[0][0], db=outs[1][0], workspace=ws)
    torch.cuda.synchronize()
    F64.within(dtype, outs[0][0], *F64.product64(dc.double(), b.double().t()), "da")
    F64.within(dtype, outs[1][0], *F64.product64(dc.double().t(), a.double().t()), "db")
    assert all(ok() for _, ok in outs), "written outside the outputs"
    da, db = gp.gemm_backward(dtype, dc, a, b)
    assert torch.equal(da, outs[0][0]) and torch.equal(db, outs[1][0])


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M", [3, 50])
def test_rows_do_not_mix_below_a_tile(dtype, M):
    import torch

    import dense_gemm_preshuffle_amd as gp

    t, (N, K) = F64.torch_type(dtype), (192, 96)
    gen = _gen(M)
    dc, a, b = _normal(gen, M, N, t=t), _normal(gen, M, K, t=t), _normal(gen, N, K, t=t)
    da, db = gp.gemm_backward(dtype, dc, a, b)
    for row, col in ((0, 0), (M - 1, N - 1)):
        bad = dc.clone()
        bad[row, col] = float("nan")
        da2, db2 = gp.gemm_backward(dtype, bad, a, b)
        torch.cuda.synchronize()
        keep = torch.arange(M, device="cuda") != row
        assert torch.equal(da2[keep], da[keep]) and bool(torch.isnan(da2[row]).all())
        keep = torch.arange(N, device="cuda") != col
        assert torch.equal(db2[keep], db[keep]) and bool(torch.isnan(db2[col]).all())


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,F,H", [(1, 32, 64), (13, 6752, 352), (53, 1968, 2752), (195, 6752, 352), (606, 4896, 448)])
def test_gated(dtype, M, F, H):
    import torch

    import dense_gemm_preshuffle_amd as gp

    t = F64.torch_type(dtype)
    gen = _gen(M + 7 * F + H)
    x, w = _normal(gen, M, H, t=t), _normal(gen, 2 * F, H, t=t, scale=H ** -0.5)
    gate, up, dh = _normal(gen, M, F, t=t), _normal(gen, M, F, t=t), _normal(gen, M, F, t=t)
    say(f"gated backward small {dtype} {M}x{F}x{H}")
    ws = gp.gated_backward_workspace(dtype, M, F, H)
    ws.fill_(255)
    dx, dw = gp.gemm_gated_backward(dtype, dh, gate, up, x, w, workspace=ws)
    torch.cuda.synchronize()
    d, ed = F64.gate_grad64(dtype, dh, gate, up, "silu")
    F64.within(dtype, dx, *F64.product64(d, w.double().t(), ed), "dx")
    F64.within(dtype, dw, *F64.product64(d.t(), x.double().t(), ed.t()), "dw")
    assert torch.equal(gp.gemm_gated_backward(dtype, dh, gate, up, None, w, want_dw=False)[0], dx)
    assert torch.equal(gp.gemm_gated_backward(dtype, dh, gate, up, x, None, want_dx=False)[1], dw)
