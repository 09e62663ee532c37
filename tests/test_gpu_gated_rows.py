"""The gated product by its row classes and column pairs, and hidden sizes that end inside a K tile."""
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


# the small kernel's row classes (1, 8, 16, 32, 48, 64) with few, some and many
# column pairs, the last workgroup's pairs cut short, K a few chunks and one half;
# above 64 rows tiles whose last K tile is half empty
SHAPES = [(1, 16, 64), (1, 6160, 96), (2, 48, 32), (8, 1040, 224), (9, 6160, 160), (16, 400, 2080), (24, 8208, 160),
          (32, 48, 96), (32, 8208, 288), (33, 400, 4128), (40, 6160, 544), (48, 8224, 96), (48, 16, 2080), (49, 1040, 352),
          (60, 6160, 160), (64, 12304, 96), (64, 12352, 64), (65, 1040, 96), (80, 2048, 32), (259, 2192, 6560),
          (130, 4096, 416), (700, 512, 8224), (300, 1040, 2144), (1030, 4112, 352)]


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,F,H", SHAPES)
def test_forward(dtype, M, F, H):
    import torch

    import dense_gemm_preshuffle_amd as gp

    t = F64.torch_type(dtype)
    gen = _gen(M * 3 + F + H)
    x, w = _normal(gen, M, H, t=t), _normal(gen, 2 * F, H, t=t, scale=H ** -0.5)
    w_shuf = gp.gemm_gated_preshuffle(w, dtype)
    act = F64.ACTS[(M + F // 16 + H // 32) % 4]
    say(f"gated rows {dtype} {M}x{F}x{H} {act}")
    ws = gp.gated_workspace(dtype, M, F, H)
    outs = [F64.guarded(M, F, t) for _ in range(3)]
    h, gate, up = (v for v, _ in outs)
    gp.gemm_gated(dtype, x, w_shuf, act=act, save=True, h=h, gate=gate, up=up, workspace=ws)
    h2 = gp.gemm_gated(dtype, x, w_shuf, act=act, workspace=ws)
    torch.cuda.synchronize()
    refs, errs = F64.gated64(x, w, act)
    for name, got, ref, err in zip(("h", "gate", "up"), (h, gate, up), refs, errs):
        F64.within(dtype, got, ref, err, name)
    assert torch.equal(h, h2)
    assert all(ok() for _, ok in outs), "written outside the outputs"


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,F,H", [(1, 64, 96), (8, 64, 96), (40, 64, 160), (100, 256, 96), (300, 256, 6560)])
def test_rows_do_not_mix_past_k(dtype, M, F, H):
    """What lies past a row's K (the next row, the end of the buffer) stays out, not finite as it may be."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    t = F64.torch_type(dtype)
    gen = _gen(5)
    buf = torch.full((M * H + 4096,), float("nan"), dtype=t, device="cuda")
    x = buf[:M * H].view(M, H)
    x.copy_(_normal(gen, M, H, t=t))
    w = _normal(gen, 2 * F, H, t=t, scale=H ** -0.5)
    w_shuf = gp.gemm_gated_preshuffle(w, dtype)
    clean = gp.gemm_gated(dtype, x, w_shuf)
    assert bool(torch.isfinite(clean).all())
    if M > 1:
        x[1] = float("inf")
        x[M - 1] = float("nan")
        h = gp.gemm_gated(dtype, x, w_shuf)
        torch.cuda.synchronize()
        keep = torch.ones(M, dtype=torch.bool, device="cuda")
        keep[1] = keep[M - 1] = False
        assert torch.equal(h[keep], clean[keep]) and not bool(torch.isfinite(h[~keep]).any())


def test_workspace_contents_stay_out():
    """The partial sums' part of a workspace may hold anything."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    for M, F, H in ((512, 512, 8192), (300, 544, 8448), (600, 1696, 4224)):
        n = gp.gemm_gated_workspace_size("bf16", M, F, H)
        ws = torch.full((max(n, 1 << 17),), 255, dtype=torch.uint8, device="cuda")
        ws[:65536] = 0
        gen = _gen(M)
        x, w = _normal(gen, M, H, t=torch.bfloat16), _normal(gen, 2 * F, H, t=torch.bfloat16, scale=H ** -0.5)
        h = gp.gemm_gated("bf16", x, gp.gemm_gated_preshuffle(w, "bf16"), workspace=ws)
        torch.cuda.synchronize()
        refs, errs = F64.gated64(x, w, "silu")
        F64.within("bf16", h, refs[0], errs[0], "h")
