"""NaN through the activations of the feed-forward and 4-bit products, and workspaces that are refused."""
import pytest

from tests import _ffn as F64
from tests import _w4

pytestmark = pytest.mark.gpu


def _gen(seed):
    import torch

    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# one row, the small kernel, tiles; a NaN gate weight makes that output column NaN and no other
@pytest.mark.parametrize("act", F64.ACTS)
@pytest.mark.parametrize("M", [1, 20, 64, 65, 300])
def test_gated(M, act):
    import torch

    import dense_gemm_preshuffle_amd as gp

    gen, F, H = _gen(M), 160, 96
    x = torch.randn(M, H, device="cuda", generator=gen).bfloat16()
    w = torch.randn(2 * F, H, device="cuda", generator=gen).bfloat16()
    want = gp.gemm_gated("bf16", x, gp.gemm_gated_preshuffle(w, "bf16"), act=act)
    w[37, 5] = float("nan")
    got = gp.gemm_gated("bf16", x, gp.gemm_gated_preshuffle(w, "bf16"), act=act)
    torch.cuda.synchronize()
    keep = torch.arange(F, device="cuda") != 37
    assert bool(torch.isnan(got[:, 37]).all()) and torch.equal(got[:, keep], want[:, keep])


@pytest.mark.parametrize("act", F64.ACTS)
def test_gated_backward(act):
    import torch

    import dense_gemm_preshuffle_amd as gp

    gen, M, F, H = _gen(3), 70, 64, 96
    t = lambda *s: torch.randn(*s, device="cuda", generator=gen).half()
    dh, gate, up, x, w = t(M, F), t(M, F), t(M, F), t(M, H), t(2 * F, H)
    dx, dw = gp.gemm_gated_backward("fp16", dh, gate, up, x, w, act=act)
    gate[11, 9] = float("nan")
    dx2, dw2 = gp.gemm_gated_backward("fp16", dh, gate, up, x, w, act=act)
    torch.cuda.synchronize()
    keep = torch.arange(M, device="cuda") != 11
    rows = torch.arange(2 * F, device="cuda")
    # du of that element is dh act(NaN); dg is dh up act'(NaN), which relu and none take as a number
    assert bool(torch.isnan(dx2[11]).all()) and torch.equal(dx2[keep], dx[keep])
    assert bool(torch.isnan(dw2[F + 9]).all())
    keep = (rows != 9) & (rows != F + 9)
    assert torch.equal(dw2[keep], dw[keep])


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", F64.ACTS)
@pytest.mark.parametrize("M", [1, 4, 40])
def test_w4(M, act, gated):
    import torch

    import dense_gemm_preshuffle_amd as gp

    gen, N, K, group = _gen(M), 80, 256, 64
    x = torch.randn(M, K, device="cuda", generator=gen).half()
    q, _, s, _ = _w4.make(gen, "fp16", 2 * N if gated else N, K, group, False)
    run = gp.gemm_w4a16_gated if gated else gp.gemm_w4a16
    want = run(x, gp.gemm_w4a16_preshuffle(q, s, group=group, gated=gated), act=act)
    s[13, 2] = float("nan")
    got = run(x, gp.gemm_w4a16_preshuffle(q, s, group=group, gated=gated), act=act)
    torch.cuda.synchronize()
    keep = torch.arange(N, device="cuda") != 13
    assert bool(torch.isnan(got[:, 13]).all()) and torch.equal(got[:, keep], want[:, keep])


def test_workspaces_elsewhere_are_refused():
    import torch

    import dense_gemm_preshuffle_amd as gp

    gen, M, F, H = _gen(1), 8, 64, 4096
    x = torch.randn(M, H, device="cuda", generator=gen).half()
    w = torch.randn(2 * F, H, device="cuda", generator=gen).half()
    g = torch.randn(M, F, device="cuda", generator=gen).half()
    q, _, s, _ = _w4.make(gen, "fp16", F, H, 128, False)
    w4, laid = gp.gemm_w4a16_preshuffle(q, s, group=128), gp.gemm_gated_preshuffle(w, "fp16")
    for ws in (torch.zeros(1 << 22, dtype=torch.uint8), torch.zeros(1 << 23, dtype=torch.uint8, device="cuda")[::2]):
        for call in (lambda: gp.gemm_gated("fp16", x, laid, workspace=ws),
                     lambda: gp.gemm_gated_backward("fp16", g, g, g, x, w, workspace=ws),
                     lambda: gp.gemm_backward("fp16", g, x, w[:F], workspace=ws),
                     lambda: gp.gemm_w4a16(x, w4, workspace=ws)):
            with pytest.raises(ValueError, match="workspace"):
                call()
    torch.cuda.synchronize()
