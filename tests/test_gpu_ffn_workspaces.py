"""Calls that make a workspace of their own, eagerly and in a captured graph: counters zero, the rest anything."""
import pytest

from tests import _w4
from tests._parity import say

pytestmark = pytest.mark.gpu


def test_own_workspaces_and_graph_replays():
    import torch

    import dense_gemm_preshuffle_amd as gp

    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    t = torch.bfloat16
    normal = lambda *s, scale=1.0: (torch.randn(*s, generator=gen, device="cuda") * scale).to(t)
    # a split tile, a split small gated product, a split 4-bit product
    assert gp.gemm_gated_plan("bf16", 259, 2192, 6560)["ksplit"] > 1 and gp.gemm_gated_plan("bf16", 40, 336, 6720)["ksplit"] > 1
    assert gp.gemm_w4a16_plan(40, 200, 16384, 128, with_workspace=True)["ksplit"] > 1
    x1, w1 = normal(259, 6560), gp.gemm_gated_preshuffle(normal(2 * 2192, 6560, scale=0.01), "bf16")
    x2, w2 = normal(40, 6720), gp.gemm_gated_preshuffle(normal(2 * 336, 6720, scale=0.01), "bf16")
    q, v, s, z = _w4.make(gen, "bf16", 200, 16384, 128, True)
    x3, w3 = normal(40, 16384), gp.gemm_w4a16_preshuffle(q, s, z, group=128)

    def step(ws=(None, None, None)):
        return [gp.gemm_gated("bf16", x1, w1, workspace=ws[0]), gp.gemm_gated("bf16", x2, w2, workspace=ws[1]),
                gp.gemm_w4a16(x3, w3, workspace=ws[2])]
    kept = (gp.gated_workspace("bf16", 259, 2192, 6560), gp.gated_workspace("bf16", 40, 336, 6720), gp.w4a16_workspace(40, w3))
    want = [o.clone() for o in step(kept)]
    # memory that the calls' own workspaces are likely to get: not zero
    torch.full((40 << 20,), 255, dtype=torch.uint8, device="cuda")
    assert all(torch.equal(a, b) for a, b in zip(step(), want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(5):
        for o in out:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), k
        torch.full((40 << 20,), 255, dtype=torch.uint8, device="cuda")
        assert all(torch.equal(a, b) for a, b in zip(step(), want)), k
    say("own workspaces: ok")
