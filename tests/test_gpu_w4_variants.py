"""Every compiled variant of the 4-bit products against float64: types, groups inside a block, of a block and longer,
with and without zero points, outputs guarded on both sides whatever their size."""
import pytest

from tests import _ffn as F64
from tests import _w4, _w4_variants
from tests._parity import say

pytestmark = pytest.mark.gpu


def _gen(seed):
    import torch

    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bounds(ref, err, act):
    """act(ref) and its bound before rounding: |act'| < 1.2, the activation's own error as in _ffn."""
    a, _ = F64.act64(act, ref)
    return a, 1.2 * err + 2.0 ** -20 * a.abs() + (0.8e-7 * ref.abs() if act == "gelu" else 0)


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("zeros", [False, "wide"])
@pytest.mark.parametrize("group", [32, 64, 128, 512])
@pytest.mark.parametrize("variant,M,N,K,gated", list(_w4_variants.shapes()))
def test_variant(variant, M, N, K, gated, group, zeros, dtype):
    import torch

    import dense_gemm_preshuffle_amd as gp

    t, gen = F64.torch_type(dtype), _gen(M + N + K + group)
    x = torch.randn(M, K, device="cuda", generator=gen).to(t)
    q, v, s, z = _w4.make(gen, dtype, 2 * N if gated else N, K, group, zeros)
    act = F64.ACTS[(M + N + group // 32 + bool(zeros)) % 4]
    w = gp.gemm_w4a16_preshuffle(q, s, z, group=group, gated=gated)
    y, untouched = F64.guarded(M, N, t)
    say(f"w4 variant {variant} {dtype} {M}x{N}x{K} gated {gated} group {group} zeros {zeros} {act}")
    # both types accumulate x (q + 8) and take the group's sum of x times (8 + z) away: the bound of either
    # counts the magnitudes of both parts, as _w4.product64 has them under "bf16"
    ref, err = _w4.product64("bf16", x, v, s, z, group)
    if gated:
        gp.gemm_w4a16_gated(x, w, act=act, h=y)
        a, ea = _bounds(ref[:, :N], err[:, :N], act)
        u, eu = ref[:, N:], err[:, N:]
        ref, err = a * u, ea * u.abs() + (a.abs() + ea) * eu + 2.0 ** -23 * (a * u).abs()
    else:
        bias = torch.randn(N, device="cuda", generator=gen) if group != 64 else None
        gp.gemm_w4a16(x, w, bias=bias, act=act, y=y)
        if bias is not None:
            ref = ref + bias.double()
            err = err + 2.0 ** -24 * ref.abs()
        ref, err = _bounds(ref, err, act)
    torch.cuda.synchronize()
    F64.within(dtype, y, ref, err, "y")
    assert untouched(), "written outside the output"


# the shapes whose last column block, or last workgroup's rows, end inside; a workspace where K is split
@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,N,K,gated", [(1, 1, 32, False), (1, 17, 160, False), (2, 33, 96, False), (5, 4091, 288, False),
                                         (17, 31, 288, False), (33, 77, 640, False), (65, 99, 544, False), (1, 1, 32, True),
                                         (3, 515, 288, True), (7, 33, 416, True), (64, 129, 928, True), (90, 47, 352, True),
                                         (1, 33, 28704, False), (40, 77, 16416, True), (100, 48, 20000, False)])
def test_nothing_is_written_outside(M, N, K, gated, dtype):
    import torch

    import dense_gemm_preshuffle_amd as gp

    t, gen = F64.torch_type(dtype), _gen(M + N + K)
    x = torch.randn(M, K, device="cuda", generator=gen).to(t)
    q, v, s, z = _w4.make(gen, dtype, 2 * N if gated else N, K, 128, True)
    w = gp.gemm_w4a16_preshuffle(q, s, z, group=128, gated=gated)
    n = gp.gemm_w4a16_workspace_size(M, N, K, 128, gated)
    say(f"w4 guarded {dtype} {M}x{N}x{K} gated {gated} workspace {n}")
    run = (lambda **k: gp.gemm_w4a16_gated(x, w, h=k.pop("y"), **k)) if gated else (lambda **k: gp.gemm_w4a16(x, w, **k))
    ref, err = _w4.product64("bf16", x, v, s, z, 128)
    if gated:
        a, ea = _bounds(ref[:, :N], err[:, :N], "silu")
        u, eu = ref[:, N:], err[:, N:]
        ref, err = a * u, ea * u.abs() + (a.abs() + ea) * eu + 2.0 ** -23 * (a * u).abs()
    else:
        ref, err = _bounds(ref, err, "silu")
    for ws in [None] + ([n] if n else []):
        y, untouched = F64.guarded(M, N, t)
        buf = None
        if ws:
            buf = torch.full((n + 4096,), 255, dtype=torch.uint8, device="cuda")
            buf[:65536] = 0
        run(y=y, act="silu", workspace=buf[:n] if ws else None)
        torch.cuda.synchronize()
        F64.within(dtype, y, ref, err, f"workspace {ws}")
        assert untouched() and (buf is None or bool((buf[n:] == 255).all()))
