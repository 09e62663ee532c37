"""The linear layer with its epilogue and its backward pass on the GPU against float64."""
import pytest

from tests import _ffn as F64
from tests import _linear as L64
from tests import _norm as N64
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


# rows: one token, each small variant's last and first count, the tiles' first, edge
# tiles; N: one block, columns no tile divides; K: one 64-byte block, odd block
# counts (K shares that differ), K split across workgroups
SHAPES = [(1, 16, 32), (1, 272, 16), (5, 1040, 48), (40, 528, 2064), (130, 2048, 2064), (300, 272, 80), (1025, 1040, 1040), (1, 4096, 96), (1, 9232, 2048), (3, 2064, 160), (8, 48, 544), (9, 8208, 96), (16, 256, 512), (17, 48, 544),
          (32, 8448, 160), (33, 272, 1024), (48, 8208, 352), (64, 1040, 352), (64, 8448, 416), (64, 512, 8192), (65, 144, 512),
          (65, 112, 160), (100, 16, 64), (129, 1040, 96), (300, 2064, 512), (512, 1024, 8192), (777, 1040, 2048),
          (256, 4096, 4096), (1025, 4112, 1024), (2048, 8192, 256), (2100, 8208, 1056)]


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_forward(dtype, M, N, K):
    import torch

    import dense_gemm_preshuffle_amd as gp

    t = F64.torch_type(dtype)
    gen = _gen(M * 7 + N + K)
    x, w = _normal(gen, M, K, t=t), _normal(gen, N, K, t=t, scale=K ** -0.5)
    bias, residual = torch.randn(N, generator=gen, device="cuda"), _normal(gen, M, N, t=t, scale=2.0)
    act = F64.ACTS[(M + N // 16 + K // 32) % 4]
    plan = gp.gemm_linear_plan(dtype, M, N, K)
    say(f"linear {dtype} {M}x{N}x{K} {act} kernel {plan['kernel']} {plan['tile_m']}x{plan['tile_n']} ksplit {plan['ksplit']}")
    w_shuf = gp.gemm_linear_preshuffle(w, dtype)
    if K % 64 == 0:
        assert torch.equal(w_shuf, gp.gemm_preshuffle_b(w, dtype))
    ws = gp.linear_workspace(dtype, M, N, K)
    (y, y_ok), (z, z_ok) = F64.guarded(M, N, t), F64.guarded(M, N, t)
    gp.gemm_linear(dtype, x, w_shuf, bias=bias, act=act, residual=residual, save=True, y=y, z=z, workspace=ws)
    torch.cuda.synchronize()
    ref_y, ref_z = L64.forward64(x, w, bias, act, residual)
    a, b = F64.within(dtype, y, *ref_y, "y"), F64.within(dtype, z, *ref_z, "z")
    say("  shares of the bounds", round(a, 3), round(b, 3))
    assert y_ok() and z_ok(), "written outside the outputs"
    # in place of the residual, without z, on a workspace of the call's own: the same bits
    inplace = residual.clone()
    gp.gemm_linear(dtype, x, w_shuf, bias=bias, act=act, residual=inplace, y=inplace)
    assert torch.equal(inplace, y)
    # the plain product
    plain = gp.gemm_linear(dtype, x, w_shuf, workspace=ws)
    torch.cuda.synchronize()
    F64.within(dtype, plain, *L64.forward64(x, w, None, "none", None)[0], "plain")
    assert ws is None or not bool(ws[:65536].any())


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("act", F64.ACTS)
@pytest.mark.parametrize("M", [5, 200])
def test_activations(dtype, act, M):
    """Every activation in both kernels, over the arguments where it saturates."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    t, K, N = F64.torch_type(dtype), 64, 256
    x = torch.zeros(M, K, dtype=t, device="cuda")
    x[:, 0] = torch.linspace(-1, 1, M, device="cuda").to(t)
    w = torch.zeros(N, K, dtype=t, device="cuda")
    w[:, 0] = torch.linspace(0, 100, N, device="cuda").to(t)
    y = gp.gemm_linear(dtype, x, gp.gemm_linear_preshuffle(w, dtype), act=act)
    torch.cuda.synchronize()
    say(f"linear act {dtype} {act} M {M}", F64.within(dtype, y, *L64.forward64(x, w, None, act, None)[0], act))


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M", [37, 201])
def test_rows_do_not_mix(dtype, M):
    import torch

    import dense_gemm_preshuffle_amd as gp

    t, K, N = F64.torch_type(dtype), 160, 528
    gen = _gen(5)
    x, w = _normal(gen, M, K, t=t), _normal(gen, N, K, t=t, scale=K ** -0.5)
    res = _normal(gen, M, N, t=t)
    w_shuf = gp.gemm_linear_preshuffle(w, dtype)
    clean = gp.gemm_linear(dtype, x, w_shuf, act="relu", residual=res)
    for row, v in ((0, float("nan")), (M - 1, float("nan")), (M // 2, float("inf"))):
        for bad_x in (True, False):
            bad, r = x.clone(), res.clone()
            (bad if bad_x else r)[row, 3] = v
            y = gp.gemm_linear(dtype, bad, w_shuf, act="relu", residual=r)
            torch.cuda.synchronize()
            keep = torch.arange(M, device="cuda") != row
            assert torch.equal(y[keep], clean[keep])
            wrong = ~torch.isfinite(y[row])
            assert bool(wrong.any()) if bad_x else (bool(wrong[3]) and int(wrong.sum()) == 1)


BACKWARD = [(1, 32, 32), (3, 64, 16), (130, 2048, 2064), (300, 272, 80), (70, 1040, 1040), (4100, 544, 1040), (1, 16, 32), (2, 96, 96), (31, 544, 160), (31, 528, 160), (130, 2064, 2048), (4100, 1040, 512), (33, 1056, 544), (65, 2080, 160), (130, 2080, 2048), (257, 1056, 1024),
            (500, 512, 4096), (1000, 4128, 256), (2049, 1024, 1024), (4100, 992, 512),
            (2300, 480, 1376), (3001, 256, 2048)]   # dw's workgroups the longer ones of the launch of both


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,N,K", BACKWARD)
def test_backward(dtype, M, N, K):
    import torch

    import dense_gemm_preshuffle_amd as gp

    t = F64.torch_type(dtype)
    gen = _gen(M + 3 * N + K)
    x, w = _normal(gen, M, K, t=t), _normal(gen, N, K, t=t, scale=K ** -0.5)
    z, dy = _normal(gen, M, N, t=t), _normal(gen, M, N, t=t)
    for act in (F64.ACTS[(M + N // 32 + K // 32) % 3], "none"):
        say(f"linear backward {dtype} {M}x{N}x{K} {act}")
        kept = None if act == "none" else z
        n = gp.gemm_linear_backward_workspace_size(dtype, M, N, K, act)
        ws = torch.full((n + 4096,), 255, dtype=torch.uint8, device="cuda")
        (dx, ok1), (dw, ok2) = F64.guarded(M, K, t), F64.guarded(N, K, t)
        db, ok3 = F64.guarded(1, N, torch.float32)
        gp.gemm_linear_backward(dtype, dy, kept, x, w, act=act, dx=dx, dw=dw, dbias=db[0], workspace=ws[:n])
        torch.cuda.synchronize()
        ref = L64.backward64(dtype, dy, z, x, w, act)
        shares = [F64.within(dtype, dx, *ref["dx"], "dx"), F64.within(dtype, dw, *ref["dw"], "dw"),
                  N64.within32(db[0], *ref["dbias"], "dbias")]
        say("  shares of the bounds", [round(v, 3) for v in shares])
        assert ok1() and ok2() and ok3() and bool((ws[n:] == 255).all()), "written outside the outputs or the workspace"
        # one output alone: the same bits
        got = gp.gemm_linear_backward(dtype, dy, kept, None, w, act=act, want_dw=False, want_dbias=False)
        assert got[1] is None and got[2] is None and torch.equal(got[0], dx)
        got = gp.gemm_linear_backward(dtype, dy, kept, x, None, act=act, want_dx=False, want_dbias=False)
        assert got[0] is None and torch.equal(got[1], dw)
        got = gp.gemm_linear_backward(dtype, dy, kept, None, None, act=act, want_dx=False, want_dw=False)
        assert got[0] is None and got[1] is None and torch.equal(got[2], db[0])


@pytest.mark.parametrize("M,N,K", [(2706, 32, 8608), (3870, 3808, 9376)])
def test_backward_without_an_activation_on_the_default_workspace(M, N, K):
    """The workspace for any activation serves the call without one where that call's plans need more than its own."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    dtype, t = "fp16", torch.float16
    gen = _gen(M)
    x, w, dy = _normal(gen, M, K, t=t), _normal(gen, N, K, t=t, scale=K ** -0.5), _normal(gen, M, N, t=t, scale=0.1)
    say(f"linear backward {dtype} {M}x{N}x{K} none on the workspace of any activation")
    ws = gp.linear_backward_workspace(dtype, M, N, K)
    want = gp.gemm_linear_backward(dtype, dy, None, x, w)
    got = gp.gemm_linear_backward(dtype, dy, None, x, w, workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ref = L64.backward64(dtype, dy, None, x, w, "none")
    F64.within(dtype, got[0], *ref["dx"], "dx")
    F64.within(dtype, got[1], *ref["dw"], "dw")
    N64.within32(got[2], *ref["dbias"], "dbias")


@pytest.mark.parametrize("act", F64.ACTS)
def test_gradients_against_differences(act):
    """Each gradient along a direction against central differences of the layer in float64."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    dtype, t, M, N, K = "fp16", torch.float16, 48, 64, 96
    gen = _gen(17)
    x, w, dy = _normal(gen, M, K, t=t), _normal(gen, N, K, t=t, scale=K ** -0.5), _normal(gen, M, N, t=t)
    bias = torch.randn(N, generator=gen, device="cuda")
    _, z = gp.gemm_linear(dtype, x, gp.gemm_linear_preshuffle(w, dtype), bias=bias, act=act, save=True)
    grads = gp.gemm_linear_backward(dtype, dy, z, x, w, act=act)

    def loss(x_, w_, b_):
        return float((F64.act64(act, x_ @ w_.t() + b_)[0] * dy.double()).sum())
    step = 1e-6
    for k, (g, v) in enumerate(zip(grads, (x, w, bias))):
        d = torch.randn(v.shape, generator=gen, device="cuda", dtype=torch.float64)
        a = [x.double(), w.double(), bias.double()]
        plus, minus = list(a), list(a)
        plus[k], minus[k] = a[k] + step * d, a[k] - step * d
        diff = (loss(*plus) - loss(*minus)) / (2 * step)
        got = float((g.double() * d).sum())
        # each entry is off by a few fp16 roundings of its terms (z, dz, itself): 8 half steps of its own magnitude
        # plus the same of a typical entry, against a random direction
        scale = float(g.double().norm()) * 8 * 2.0 ** -11 * 4
        say(f"differences {act} {k}: {got:.6g} against {diff:.6g}, allowed {scale:.3g}")
        assert abs(got - diff) <= scale


def test_another_stream_and_graph_replays():
    import torch

    import dense_gemm_preshuffle_amd as gp

    dtype, t = "bf16", torch.bfloat16
    for M, N, K in ((1, 1024, 512), (40, 336, 6720), (300, 1056, 544), (512, 1024, 8192)):
        gen = _gen(M)
        x, w = _normal(gen, M, K, t=t), _normal(gen, N, K, t=t, scale=K ** -0.5)
        dy, res = _normal(gen, M, N, t=t), _normal(gen, M, N, t=t)
        bias = torch.randn(N, generator=gen, device="cuda")
        w_shuf = gp.gemm_linear_preshuffle(w, dtype)
        ws, wb = gp.linear_workspace(dtype, M, N, K), gp.linear_backward_workspace(dtype, M, N, K)

        def step(stream=None, ws=ws, wb=wb):
            out = list(gp.gemm_linear(dtype, x, w_shuf, bias=bias, act="silu", residual=res, save=True, workspace=ws,
                                      stream=stream))
            out += gp.gemm_linear_backward(dtype, dy, out[1], x, w, act="silu", workspace=wb, stream=stream)
            return out
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
            out = step(ws=None, wb=None)     # workspaces of the calls' own
        for k in range(4):
            for o in out:
                o.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), (M, k)
            assert all(torch.equal(a, b) for a, b in zip(step(), want)), (M, k)
        say(f"streams and graph {M}x{N}x{K}: ok")


def test_workspace_serves_every_size():
    """One workspace through calls of different plans and operators: its counters come back to zero."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    shapes = [(512, 1024, 8192), (40, 336, 6720), (256, 2048, 4096), (512, 1024, 8192), (96, 1024, 8192)]
    assert all(gp.gemm_linear_workspace_size("bf16", *s) for s in shapes)
    ws = torch.zeros(max(gp.gemm_linear_workspace_size("bf16", *s) for s in shapes), dtype=torch.uint8, device="cuda")
    for M, N, K in shapes:
        gen = _gen(M + K)
        x, w = _normal(gen, M, K, t=torch.bfloat16), _normal(gen, N, K, t=torch.bfloat16, scale=K ** -0.5)
        y = gp.gemm_linear("bf16", x, gp.gemm_linear_preshuffle(w, "bf16"), workspace=ws)
        torch.cuda.synchronize()
        F64.within("bf16", y, *L64.forward64(x, w, None, "none", None)[0], "y")
        assert not bool(ws[:65536].any())


def test_binding_refusals(monkeypatch):
    import torch

    import dense_gemm_preshuffle_amd as gp

    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(32, 64, dtype=torch.bfloat16, device="cuda")
    s = gp.gemm_linear_preshuffle(w, "bf16")
    y = gp.gemm_linear("bf16", x, s)
    assert y.shape == (4, 32) and not bool(y.any())
    bad = [lambda: gp.gemm_linear("bf16", x.half(), s), lambda: gp.gemm_linear("bf16", x, s, bias=torch.zeros(32).bfloat16().cuda()),
           lambda: gp.gemm_linear("bf16", x, s, bias=torch.zeros(31, device="cuda")),
           lambda: gp.gemm_linear("bf16", x, s, residual=y[:2]), lambda: gp.gemm_linear("bf16", x, s, z=y),
           lambda: gp.gemm_linear("bf16", x.cpu(), s), lambda: gp.gemm_linear("bf16", x, s.cpu()),
           lambda: gp.gemm_linear("bf16", x[:, ::2], s), lambda: gp.gemm_linear_backward("bf16", y, None, x, w, act="silu"),
           lambda: gp.gemm_linear_backward("bf16", y, None, None, w), lambda: gp.gemm_linear_backward("bf16", y, y[:2], x, w),
           lambda: gp.gemm_linear_backward("bf16", y, None, x, w, want_dx=False, dx=x)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: gp.gemm_linear("fp8", x, s), lambda: gp.gemm_linear("bf16", x[:0], s),
              lambda: gp.gemm_linear_backward("bf16", y, None, x, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(gp.GemmError):
            f()
    monkeypatch.setattr(gp, "_device", lambda: 1)
    for f in (lambda: gp.gemm_linear("bf16", x, s), lambda: gp.gemm_linear_backward("bf16", y, None, x, w),
              lambda: gp.gemm_linear_preshuffle(w, "bf16")):
        with pytest.raises(ValueError, match="current device"):
            f()
