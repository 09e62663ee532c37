"""Small products whose K is split across workgroups: few output columns, long K."""
import pytest

from tests import _ffn as F64
from tests import _w4
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


def _dirty(n):
    """A workspace of n bytes: counters zero, the rest anything."""
    import torch

    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    ws[:65536] = 0
    return ws


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,F,H", [(1, 368, 6784), (5, 16, 8192), (16, 512, 8224), (32, 336, 6720), (40, 336, 6720),
                                   (64, 48, 16416), (48, 2048, 4096)])
def test_gated(dtype, M, F, H):
    import torch

    import dense_gemm_preshuffle_amd as gp

    t = F64.torch_type(dtype)
    gen = _gen(M + F + H)
    x, w = _normal(gen, M, H, t=t), _normal(gen, 2 * F, H, t=t, scale=H ** -0.5)
    w_shuf = gp.gemm_gated_preshuffle(w, dtype)
    n = gp.gemm_gated_workspace_size(dtype, M, F, H)
    assert n > 65536
    say(f"gated split {dtype} {M}x{F}x{H} workspace {n}")
    ws = _dirty(n)
    outs = [F64.guarded(M, F, t) for _ in range(3)]
    h, gate, up = (v for v, _ in outs)
    gp.gemm_gated(dtype, x, w_shuf, save=True, h=h, gate=gate, up=up, workspace=ws)
    torch.cuda.synchronize()
    refs, errs = F64.gated64(x, w, "silu")
    for name, got, ref, err in zip(("h", "gate", "up"), (h, gate, up), refs, errs):
        F64.within(dtype, got, ref, err, name)
    assert all(ok() for _, ok in outs) and not bool(ws[:65536].any())
    for _ in range(20):    # whatever the order of arrival: the same bits
        assert torch.equal(gp.gemm_gated(dtype, x, w_shuf, workspace=ws), h)
    assert torch.equal(gp.gemm_gated(dtype, x, w_shuf), h)
    with pytest.raises(gp.GemmError) as e:
        gp.gemm_gated(dtype, x, w_shuf, workspace=ws[:n - 16])
    assert e.value.status == gp.GP_EWORKSPACE


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,N,K,group,zeros,gated", [(1, 1024, 28672, 128, True, False), (1, 33, 28704, 32, "wide", False),
                                                     (4, 500, 16384, 64, False, True), (16, 1266, 18816, 128, True, False),
                                                     (20, 70, 20000, 256, False, False), (40, 77, 16416, 64, True, True),
                                                     (64, 392, 19520, 64, True, False), (100, 48, 28672, 1024, "wide", False)])
def test_w4(dtype, M, N, K, group, zeros, gated):
    import torch

    import dense_gemm_preshuffle_amd as gp

    t = F64.torch_type(dtype)
    gen = _gen(M + N + K)
    x = _normal(gen, M, K, t=t)
    q, v, s, z = _w4.make(gen, dtype, 2 * N if gated else N, K, group, zeros)
    w = gp.gemm_w4a16_preshuffle(q, s, z, group=group, gated=gated)
    n = gp.gemm_w4a16_workspace_size(M, N, K, group, gated)
    assert n > 65536
    say(f"w4 split {dtype} {M}x{N}x{K} group {group} gated {gated} workspace {n}")
    ws = _dirty(n)
    run = gp.gemm_w4a16_gated if gated else gp.gemm_w4a16
    y = run(x, w, act="silu", workspace=ws)
    torch.cuda.synchronize()
    ref, err = _w4.product64(dtype, x, v, s, z, group)
    g, eg = (ref[:, :N], err[:, :N]) if gated else (ref, err)
    a, _ = F64.act64("silu", g)
    ea = 1.2 * eg + 2.0 ** -20 * a.abs()
    if gated:
        u, eu = ref[:, N:], err[:, N:]
        ea = ea * u.abs() + (a.abs() + ea) * eu + 2.0 ** -23 * (a * u).abs()
        a = a * u
    F64.within(dtype, y, a, ea, "y")
    assert not bool(ws[:65536].any())
    for _ in range(20):
        assert torch.equal(run(x, w, act="silu", workspace=ws), y)
    F64.within(dtype, run(x, w, act="silu"), a, ea, "without a workspace of the caller's")
    with pytest.raises(gp.GemmError) as e:
        run(x, w, workspace=ws[:n - 16])
    assert e.value.status == gp.GP_EWORKSPACE


@pytest.mark.parametrize("dtype", F64.TYPES)
def test_rows_that_are_not_finite(dtype):
    import torch

    import dense_gemm_preshuffle_amd as gp

    t, M, N, K = F64.torch_type(dtype), 24, 40, 20000
    gen = _gen(1)
    x = _normal(gen, M, K, t=t)
    q, v, s, z = _w4.make(gen, dtype, N, K, 128, True)
    w = gp.gemm_w4a16_preshuffle(q, s, z, group=128)
    ws = gp.w4a16_workspace(M, w)
    clean = gp.gemm_w4a16(x, w, workspace=ws)
    weights = _w4.spread(s, 128, K) * (v.double() - _w4.spread(z, 128, K))
    for row, k, value in ((0, 5, float("inf")), (23, 19999, float("-inf")), (7, 10000, float("nan"))):
        bad = x.clone()
        bad[row, k] = value
        y = gp.gemm_w4a16(bad, w, workspace=ws)
        torch.cuda.synchronize()
        want, got = (bad[row].double()[None, :] * weights).sum(1), y[row].double()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)])
        keep = torch.arange(M, device="cuda") != row
        assert torch.equal(y[keep], clean[keep])


def test_graph_replays():
    import torch

    import dense_gemm_preshuffle_amd as gp

    gen = _gen(4)
    t = torch.bfloat16
    x = _normal(gen, 32, 8192, t=t)
    w = gp.gemm_gated_preshuffle(_normal(gen, 672, 8192, t=t, scale=0.01), "bf16")
    q, v, s, z = _w4.make(gen, "bf16", 200, 8192, 128, True)
    w4 = gp.gemm_w4a16_preshuffle(q, s, z, group=128)
    ws, ws4 = gp.gated_workspace("bf16", 32, 336, 8192), gp.w4a16_workspace(32, w4)
    assert ws is not None and ws4 is not None

    def step():
        return gp.gemm_gated("bf16", x, w, workspace=ws), gp.gemm_w4a16(x, w4, workspace=ws4)
    want = [o.clone() for o in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(5):
        for o in out:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for a, b in zip(step(), want))
    say("small split graph: ok")
