"""Gated feed-forward product and backward passes on the GPU against float64."""
import numpy as np
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


# rows: one token, one block and one more, the small kernel's last row count and
# the tiles' first, edge tiles; F: a single pair of blocks, columns no tile
# divides; H: one 64-byte block, odd block counts (K shares that differ)
FORWARD = [(1, 16, 32), (1, 272, 96), (1, 1040, 2048), (3, 2064, 160), (16, 256, 512), (17, 48, 544), (33, 272, 1024),
           (64, 1040, 352), (65, 144, 512), (65, 2064, 160), (100, 16, 64), (129, 1040, 96), (300, 2064, 512),
           (512, 512, 8192), (777, 1040, 2048), (256, 4096, 4096), (1025, 4112, 1024), (2048, 8192, 256)]


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,F,H", FORWARD)
def test_gated_forward(dtype, M, F, H):
    import torch

    import dense_gemm_preshuffle_amd as gp

    t = F64.torch_type(dtype)
    gen = _gen(M * 7 + F + H)
    x, w = _normal(gen, M, H, t=t), _normal(gen, 2 * F, H, t=t, scale=H ** -0.5)
    w_shuf = gp.gemm_gated_preshuffle(w, dtype)
    act = F64.ACTS[(M + F // 16 + H // 32) % 4]
    say(f"gated {dtype} {M}x{F}x{H} {act} workspace {gp.gemm_gated_workspace_size(dtype, M, F, H)}")
    ws = gp.gated_workspace(dtype, M, F, H)
    outs = [F64.guarded(M, F, t) for _ in range(3)]
    h, gate, up = (v for v, _ in outs)
    gp.gemm_gated(dtype, x, w_shuf, act=act, save=True, h=h, gate=gate, up=up, workspace=ws)
    h2 = gp.gemm_gated(dtype, x, w_shuf, act=act, workspace=ws)
    torch.cuda.synchronize()
    refs, errs = F64.gated64(x, w, act)
    worst = [F64.within(dtype, v, r, e, n) for v, r, e, n in zip((h, gate, up), refs, errs, ("h", "gate", "up"))]
    say("  shares of the bounds", [round(v, 3) for v in worst])
    assert all(ok() for _, ok in outs), "written outside the outputs"
    assert torch.equal(h, h2), "h differs with and without keeping gate and up, or between calls"


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("act", F64.ACTS)
@pytest.mark.parametrize("M", [5, 200])
def test_gated_activations(dtype, act, M):
    """Every activation in both kernels, over the arguments where it saturates."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    t, H, F = F64.torch_type(dtype), 64, 256
    gen = _gen(3)
    x = torch.zeros(M, H, dtype=t, device="cuda")
    x[:, 0] = torch.linspace(-1, 1, M, device="cuda").to(t)
    x[:, 1] = 1
    w = _normal(gen, 2 * F, H, t=t)
    w[:F, 0] = torch.linspace(0, 100, F, device="cuda").to(t)   # gates from -100 to 100
    h = gp.gemm_gated(dtype, x, gp.gemm_gated_preshuffle(w, dtype), act=act)
    torch.cuda.synchronize()
    refs, errs = F64.gated64(x, w, act)
    say(f"gated act {dtype} {act} M {M}", F64.within(dtype, h, refs[0], errs[0], act))


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M", [37, 201])
def test_rows_do_not_mix(dtype, M):
    """A row of x that is not finite changes that row of h alone, edge tiles included."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    t, H, F = F64.torch_type(dtype), 160, 528
    gen = _gen(5)
    x, w = _normal(gen, M, H, t=t), _normal(gen, 2 * F, H, t=t, scale=H ** -0.5)
    w_shuf = gp.gemm_gated_preshuffle(w, dtype)
    clean = gp.gemm_gated(dtype, x, w_shuf)
    for row, v in ((0, float("nan")), (M - 1, float("inf")), (M // 2, float("-inf"))):
        bad = x.clone()
        bad[row, 3] = v
        h = gp.gemm_gated(dtype, bad, w_shuf)
        torch.cuda.synchronize()
        keep = torch.arange(M, device="cuda") != row
        assert torch.equal(h[keep], clean[keep])
        assert bool(torch.isnan(h[row]).any()) or bool(torch.isinf(h[row]).any())


BACKWARD = [(1, 16, 32), (2, 48, 96), (31, 272, 160), (32, 256, 512), (33, 1040, 544), (65, 2064, 160), (130, 2064, 2048),
            (257, 1040, 1024), (500, 512, 4096), (1000, 4112, 256), (2049, 1024, 1024)]


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,F,H", BACKWARD)
def test_gated_backward(dtype, M, F, H):
    import torch

    import dense_gemm_preshuffle_amd as gp

    t = F64.torch_type(dtype)
    gen = _gen(M + 3 * F + H)
    x, w = _normal(gen, M, H, t=t), _normal(gen, 2 * F, H, t=t, scale=H ** -0.5)
    gate, up, dh = _normal(gen, M, F, t=t), _normal(gen, M, F, t=t), _normal(gen, M, F, t=t)
    act = F64.ACTS[(M + F // 16 + H // 32) % 4]
    say(f"gated backward {dtype} {M}x{F}x{H} {act}")
    ws = gp.gated_backward_workspace(dtype, M, F, H)
    ws.fill_(255)   # whatever the workspace holds (NaN in both types) stays out of the results
    outs = [F64.guarded(M, H, t), F64.guarded(2 * F, H, t)]
    gp.gemm_gated_backward(dtype, dh, gate, up, x, w, act=act, dx=outs[0][0], dw=outs[1][0], workspace=ws)
    torch.cuda.synchronize()
    d, ed = F64.gate_grad64(dtype, dh, gate, up, act)
    ref, err = F64.product64(d, w.double().t(), ed)
    a = F64.within(dtype, outs[0][0], ref, err, "dx")
    ref, err = F64.product64(d.t(), x.double().t(), ed.t())
    b = F64.within(dtype, outs[1][0], ref, err, "dw")
    say("  shares of the bounds", round(a, 3), round(b, 3))
    assert all(ok() for _, ok in outs), "written outside the outputs"
    # one output alone: the same bits
    dx, none = gp.gemm_gated_backward(dtype, dh, gate, up, None, w, act=act, want_dw=False)
    assert none is None and torch.equal(dx, outs[0][0])
    none, dw = gp.gemm_gated_backward(dtype, dh, gate, up, x, None, act=act, want_dx=False)
    assert none is None and torch.equal(dw, outs[1][0])


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("act", F64.ACTS)
def test_gate_gradients_where_they_saturate(dtype, act):
    """dg and du themselves, read through a weight of ones: gates from -100 to 100 and exact zeros."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    t, M, F, H = F64.torch_type(dtype), 64, 32, 64
    gate = torch.linspace(-100, 100, M * F, device="cuda").view(M, F).to(t)
    gate[0, :8] = 0
    gen = _gen(11)
    up, dh = _normal(gen, M, F, t=t), _normal(gen, M, F, t=t)
    w = torch.zeros(2 * F, H, dtype=t, device="cuda")
    w[torch.arange(2 * F), torch.arange(2 * F)] = 1     # dx = [dg du]
    dx, _ = gp.gemm_gated_backward(dtype, dh, gate, up, None, w, act=act, want_dw=False)
    torch.cuda.synchronize()
    d, ed = F64.gate_grad64(dtype, dh, gate, up, act)
    say(f"gate grad {dtype} {act}", F64.within(dtype, dx, d, ed, act))


@pytest.mark.parametrize("act", F64.ACTS)
def test_gradients_against_differences(act):
    """dx and dw along a direction against central differences of the whole block in float64
    (the forward as the library defines it), so that the formula itself is checked."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    dtype, M, F, H = "fp16", 48, 64, 96
    t = torch.float16
    gen = _gen(17)
    x, w = _normal(gen, M, H, t=t), _normal(gen, 2 * F, H, t=t, scale=H ** -0.5)
    dh = _normal(gen, M, F, t=t)
    _, gate, up = gp.gemm_gated(dtype, x, gp.gemm_gated_preshuffle(w, dtype), act=act, save=True)
    dx, dw = gp.gemm_gated_backward(dtype, dh, gate, up, x, w, act=act)

    def loss(x_, w_):
        z = x_ @ w_.t()
        return float((F64.act64(act, z[:, :F])[0] * z[:, F:] * dh.double()).sum())
    step = 1e-6
    for k, (g, v) in enumerate(((dx, x), (dw, w))):
        d = torch.randn(v.shape, generator=gen, device="cuda", dtype=torch.float64)
        a = [x.double(), w.double()]
        plus, minus = list(a), list(a)
        plus[k], minus[k] = a[k] + step * d, a[k] - step * d
        diff = (loss(*plus) - loss(*minus)) / (2 * step)
        got = float((g.double() * d).sum())
        # each gradient entry is off by a few fp16 roundings of its terms (gate, up, dg, du, itself):
        # 8 half steps of its own magnitude plus the same of a typical entry, against a random direction
        scale = float(g.double().norm()) * 8 * 2.0 ** -11 * 4
        # relu: a gate within the kept rounding of zero may fall on the other side
        say(f"differences {act} {'dx' if k == 0 else 'dw'}: {got:.6g} against {diff:.6g}, allowed {scale:.3g}")
        assert abs(got - diff) <= scale


LINEAR = [(1, 32, 32), (33, 96, 160), (100, 4096, 1024), (300, 1056, 544), (2000, 512, 2048)]


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear_backward(dtype, M, N, K):
    import torch

    import dense_gemm_preshuffle_amd as gp

    t = F64.torch_type(dtype)
    gen = _gen(M + N + K)
    dc, a, b = _normal(gen, M, N, t=t), _normal(gen, M, K, t=t), _normal(gen, N, K, t=t, scale=K ** -0.5)
    say(f"linear backward {dtype} {M}x{N}x{K}")
    ws = gp.backward_workspace(dtype, M, N, K)
    ws.fill_(255)
    da, db = gp.gemm_backward(dtype, dc, a, b, workspace=ws)
    torch.cuda.synchronize()
    F64.within(dtype, da, *F64.product64(dc.double(), b.double().t()), "da")
    F64.within(dtype, db, *F64.product64(dc.double().t(), a.double().t()), "db")
    assert torch.equal(gp.gemm_backward(dtype, dc, None, b, want_db=False)[0], da)
    assert torch.equal(gp.gemm_backward(dtype, dc, a, None, want_da=False)[1], db)


def test_another_stream_and_graph_replays():
    """Forward and backward on a side stream, then captured and replayed between eager calls:
    every result the same bits."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    dtype, t = "bf16", torch.bfloat16
    for M, F, H in ((1, 1024, 512), (300, 1040, 544), (512, 512, 8192)):
        gen = _gen(M)
        x, w = _normal(gen, M, H, t=t), _normal(gen, 2 * F, H, t=t, scale=H ** -0.5)
        dh = _normal(gen, M, F, t=t)
        w_shuf = gp.gemm_gated_preshuffle(w, dtype)
        ws, wb = gp.gated_workspace(dtype, M, F, H), gp.gated_backward_workspace(dtype, M, F, H)

        def step(stream=None):
            h, gate, up = gp.gemm_gated(dtype, x, w_shuf, save=True, workspace=ws, stream=stream)
            dx, dw = gp.gemm_gated_backward(dtype, dh, gate, up, x, w, workspace=wb, stream=stream)
            return h, gate, up, dx, dw
        want = [v.clone() for v in step()]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        for s in (side, side.cuda_stream):
            side.wait_stream(torch.cuda.current_stream())
            got = step(s)
            torch.cuda.current_stream().wait_stream(side)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        for k in range(4):
            for o in out:
                o.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), (M, k)
            assert all(torch.equal(a, b) for a, b in zip(step(), want)), (M, k)
        say(f"streams and graph {M}x{F}x{H}: ok")


def test_workspace_serves_every_size():
    """One workspace through calls of different plans, in both orders: its counters come back to zero."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    shapes = [(512, 512, 8192), (256, 1024, 4096), (512, 512, 8192), (96, 512, 8192)]
    n = max(gp.gemm_gated_workspace_size("bf16", *s) for s in shapes)
    assert n > 0
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for M, F, H in shapes:
        gen = _gen(M + H)
        x = _normal(gen, M, H, t=torch.bfloat16)
        w = _normal(gen, 2 * F, H, t=torch.bfloat16, scale=H ** -0.5)
        w_shuf = gp.gemm_gated_preshuffle(w, "bf16")
        h = gp.gemm_gated("bf16", x, w_shuf, workspace=ws)
        torch.cuda.synchronize()
        refs, errs = F64.gated64(x, w, "silu")
        F64.within("bf16", h, refs[0], errs[0], "h")
        assert not bool(ws[:65536].any())


def test_binding_refusals():
    import torch

    import dense_gemm_preshuffle_amd as gp

    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda")
    s = gp.gemm_gated_preshuffle(w, "bf16")
    with pytest.raises(gp.GemmError):
        gp.gemm_gated("fp8", x, s)
    with pytest.raises(ValueError):
        gp.gemm_gated("bf16", x.half(), s)
    with pytest.raises(ValueError):
        gp.gemm_gated("bf16", torch.zeros(64, 4, dtype=torch.bfloat16, device="cuda").t(), s)
    with pytest.raises(ValueError):
        gp.gemm_gated("bf16", x, s, gate=torch.empty(4, 32, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(gp.GemmError):
        gp.gemm_gated("bf16", x[:0], s)
    with pytest.raises(ValueError):
        gp.gemm_gated_backward("bf16", x[:, :32].contiguous(), x, x, x, w)
    with pytest.raises(ValueError):
        gp.gemm_backward("bf16", x, x, None)
    with pytest.raises(KeyError):
        gp.gemm_gated("bf16", x, s, act="tanh")
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    h = x[:, :32].contiguous()
    with pytest.raises(gp.GemmError) as e:
        gp.gemm_gated_backward("bf16", h, h, h, x, w, workspace=small)
    assert e.value.status == gp.GP_EWORKSPACE
    assert np.isfinite(float(gp.gemm_gated("bf16", x, s).float().sum()))
