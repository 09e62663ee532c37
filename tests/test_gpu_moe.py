"""The mixture-of-experts layer for a few tokens on the GPU against float64."""
import pytest

from tests import _ffn as F64
from tests import _moe as M64
from tests._parity import say

pytestmark = pytest.mark.gpu


def _gen(seed):
    import torch

    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _layer(dtype, M, E, k, H, F, seed):
    import torch

    t, gen = F64.torch_type(dtype), _gen(seed)

    def normal(*s, scale=1.0):
        return (torch.randn(*s, generator=gen, device="cuda") * scale).to(t)
    return (normal(M, H), normal(E, H, scale=H ** -0.5), normal(E, 2 * F, H, scale=H ** -0.5), normal(E, H, F, scale=F ** -0.5),
            normal(M, H, scale=2.0), torch.randn(E, generator=gen, device="cuda") * 0.1)


# tokens: one, each row variant's last and first, more pairs than experts and fewer;
# F: one block, odd block counts, a K that is no whole chunk; H likewise
SHAPES = [(1, 8, 2, 64, 16), (1, 64, 8, 2048, 1024), (1, 5, 5, 96, 48), (2, 128, 8, 544, 272), (7, 16, 4, 160, 80), (8, 4, 1, 1024, 528),
          (9, 300, 6, 96, 144), (16, 8, 2, 512, 1040), (17, 4, 2, 2080, 96), (33, 8, 2, 1056, 272), (64, 128, 8, 256, 128),
          (64, 2, 2, 544, 48), (200, 7, 3, 160, 64), (256, 32, 16, 64, 16), (1, 512, 32, 96, 32)]


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,E,k,H,F", SHAPES)
def test_layer(dtype, M, E, k, H, F):
    import torch

    import dense_gemm_preshuffle_amd as gp

    x, router, w13, w2, residual, bias = _layer(dtype, M, E, k, H, F, M + E + H)
    act = F64.ACTS[(M + E) % 4]
    score, normalize, scale = ("softmax", True, 1.0) if E % 2 else ("sigmoid", M % 2 == 1, 2.5)
    b = bias if H % 64 else None
    say(f"moe {dtype} {M} tokens, {k} of {E}, {H} x {F} {act} {score}{' bias' if b is not None else ''}")
    weights = gp.gemm_moe_preshuffle(w13, w2, dtype)
    ws = gp.moe_workspace(M, k, weights)
    ws[65536:].fill_(255)
    y, ok = F64.guarded(M, H, F64.torch_type(dtype))
    args = dict(bias=b, score=score, normalize=normalize, scale=scale)
    got, ids, gates = gp.gemm_moe(dtype, x, router, weights, k, act=act, residual=residual, y=y, workspace=ws, **args)
    torch.cuda.synchronize()
    ref_ids, ref_gates = M64.route64(x, router, k, b, score, normalize, scale)
    assert torch.equal(ids, ref_ids)
    # scores in 64 bits, rounded once to fp32
    assert float(((gates.double() - ref_gates).abs() / ref_gates).max()) <= 2.0 ** -24 * (1 + 2.0 ** -20)
    share = F64.within(dtype, y, *M64.experts64(dtype, x, w13, w2, ids, gates, act, residual), "y")
    say("  share of the bound", round(share, 3))
    assert ok(), "written outside the output"
    assert not bool(ws[:65536].any()), "counters left set"
    # the two parts alone, on workspaces of their own, y in place of the residual: the same bits
    ids2, gates2 = gp.gemm_moe_route(dtype, x, router, k, **args)
    assert torch.equal(ids2, ids) and torch.equal(gates2, gates)
    inplace = residual.clone()
    gp.gemm_moe_experts(dtype, x, weights, ids, gates, act=act, residual=inplace, y=inplace)
    assert torch.equal(inplace, y)


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,E,k", [(1, 8, 4), (5, 64, 4), (40, 6, 3)])
def test_given_choices(dtype, M, E, k):
    """The same expert twice for a token, experts that are elsewhere, tokens without any, all tokens on one expert."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    H, F = 160, 80
    x, _, w13, w2, residual, _ = _layer(dtype, M, E, k, H, F, 3)
    weights = gp.gemm_moe_preshuffle(w13, w2, dtype)
    gen = _gen(4)
    gates = torch.rand(M, k, generator=gen, device="cuda") + 0.1
    some = torch.randint(0, E, (M, k), generator=gen, device="cuda", dtype=torch.int32)
    twice = some.clone()
    twice[:, 1] = twice[:, 0]
    away = some.clone()
    away[::2, 0] = -1
    away[:, k - 1] = E
    away[M // 2] = 2 ** 31 - 1
    none = torch.full_like(some, -5)
    one = torch.full_like(some, E - 1)
    for name, ids in (("twice", twice), ("away", away), ("none", none), ("one", one)):
        for res in (residual, None):
            y = gp.gemm_moe_experts(dtype, x, weights, ids, gates, act="gelu", residual=res)
            torch.cuda.synchronize()
            say(f"moe choices {dtype} {M} {name}")
            F64.within(dtype, y, *M64.experts64(dtype, x, w13, w2, ids, gates, "gelu", res), name)
            if name == "none":
                assert torch.equal(y, torch.zeros_like(y) if res is None else res)


def test_ties_and_not_finite():
    """Equal experts: the lowest first. A token that is not finite: distinct experts, weights NaN, its own row alone."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    M, E, k, H, F = 6, 70, 5, 96, 48
    x, router, w13, w2, residual, _ = _layer("bf16", M, E, k, H, F, 8)
    weights = gp.gemm_moe_preshuffle(w13, w2, "bf16")
    same = router[:1].expand(E, H).contiguous()
    ids, gates = gp.gemm_moe_route("bf16", x, same, k)
    assert torch.equal(ids, torch.arange(k, dtype=torch.int32, device="cuda").expand(M, k))
    assert torch.equal(gates, torch.full_like(gates, 1 / k))
    pairs = router.repeat_interleave(2, 0)[:E].contiguous()
    ids, _ = gp.gemm_moe_route("bf16", x, pairs, 4, score="sigmoid")
    assert torch.equal(ids, M64.route64(x, pairs, 4, score="sigmoid")[0])
    clean = gp.gemm_moe("bf16", x, router, weights, k, residual=residual)
    for v in (float("nan"), float("inf")):
        bad = x.clone()
        bad[2, 5] = v
        y, ids, gates = gp.gemm_moe("bf16", bad, router, weights, k, residual=residual)
        torch.cuda.synchronize()
        keep = torch.arange(M, device="cuda") != 2
        assert all(torch.equal(a[keep], b[keep]) for a, b in zip((y, ids, gates), clean))
        assert len(set(ids[2].tolist())) == k and all(0 <= i < E for i in ids[2].tolist())
        assert not bool(torch.isfinite(y[2]).any())


@pytest.mark.parametrize("M", [1, 5])
def test_one_expert_not_finite(M):
    """NaN in one expert's router row: softmax weights have it through the sum over the experts, whichever are chosen;
    sigmoid weights only where that expert is."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    E, k, H, F = 70, 5, 96, 48
    x, router, _, _, _, bias = _layer("bf16", M, E, k, H, F, 9)
    for bad in (3, 69):
        wr = router.clone()
        wr[bad, 7] = float("nan")
        for normalize in (True, False):
            for b in (None, bias):
                say(f"moe router NaN in expert {bad}, normalize {normalize}, bias {b is not None}")
                ids, gates = gp.gemm_moe_route("bf16", x, wr, k, bias=b, normalize=normalize)
                assert bool(torch.isnan(gates).all())
                assert all(len(set(row)) == k and all(0 <= i < E for i in row) for row in ids.tolist())
                assert b is not None or not bool((ids == bad).any())
                ids, gates = gp.gemm_moe_route("bf16", x, wr, k, bias=b, score="sigmoid", normalize=normalize)
                assert not bool((ids == bad).any()) and bool(torch.isfinite(gates).all())
                # (all experts: that one is chosen last)
                ids, gates = gp.gemm_moe_route("bf16", x, wr[64:].contiguous(), 6, score="sigmoid", normalize=normalize)
                if bad == 69:
                    assert bool((ids[:, 5] == 5).all()) and bool(torch.isnan(gates[:, 5]).all())
                    assert bool(torch.isnan(gates[:, :5]).all()) if normalize else bool(torch.isfinite(gates[:, :5]).all())


def test_weights_beyond_4_gib():
    """Experts whose weights lie more than 2^32 bytes into the given and the laid-out ones, in both matrices: against
    float64, and one token against the same experts laid out alone."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    E, F, H, k, gen = 300, 2048, 4096, 2, _gen(12)
    used = [0, 43, 171, 299]     # (171 and 43 lie 2^32 bytes before 299 in the one and the other matrix)
    w13 = torch.zeros(E, 2 * F, H, dtype=torch.bfloat16, device="cuda")
    w2 = torch.zeros(E, H, F, dtype=torch.bfloat16, device="cuda")
    for e in used:
        w13[e].normal_(0.0, H ** -0.5, generator=gen)
        w2[e].normal_(0.0, F ** -0.5, generator=gen)
    assert 299 * w13[0].nbytes > 2 ** 32 and 299 * w2[0].nbytes > 2 ** 32
    weights = gp.gemm_moe_preshuffle(w13, w2, "bf16")
    few13, few2 = w13[used].contiguous(), w2[used].contiguous()
    del w13, w2
    few = gp.gemm_moe_preshuffle(few13, few2, "bf16")
    for M in (1, 5, 40):
        x = torch.randn(M, H, generator=gen, device="cuda").bfloat16()
        gates = torch.rand(M, k, generator=gen, device="cuda") + 0.1
        at = torch.randint(0, len(used), (M, k), generator=gen, device="cuda")
        at[0, 0] = 3
        ids = torch.tensor(used, device="cuda")[at].int()
        say(f"moe beyond 4 GiB: {M} tokens")
        y = gp.gemm_moe_experts("bf16", x, weights, ids, gates)
        torch.cuda.synchronize()
        F64.within("bf16", y, *M64.experts64("bf16", x, few13, few2, at.int(), gates, "silu", None), "y")
        if M == 1:
            assert torch.equal(y, gp.gemm_moe_experts("bf16", x, few, at.int(), gates))


def test_streams_graph_and_one_workspace():
    """A side stream, a captured and replayed layer, one workspace through layers of different sizes."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    layers = []
    for M, E, k, H, F in ((1, 64, 8, 512, 256), (33, 8, 2, 1056, 272), (16, 128, 6, 256, 64)):
        x, router, w13, w2, residual, _ = _layer("bf16", M, E, k, H, F, M)
        layers.append((x, router, gp.gemm_moe_preshuffle(w13, w2, "bf16"), k, residual))
    n = max(gp.gemm_moe_workspace_size("bf16", l[0].shape[0], l[2].F, l[2].H, l[2].E, l[3]) for l in layers)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")

    def step(stream=None, ws=ws):
        out = []
        for x, router, weights, k, residual in layers:
            out += gp.gemm_moe("bf16", x, router, weights, k, residual=residual, workspace=ws, stream=stream)
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
        out = step(ws=None)
    for r in range(4):
        for o in out:
            o.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), r
        assert all(torch.equal(a, b) for a, b in zip(step(), want)), r
    assert not bool(ws[:65536].any())


def test_binding_refusals(monkeypatch):
    import torch

    import dense_gemm_preshuffle_amd as gp

    x, router, w13, w2, residual, bias = _layer("bf16", 3, 4, 2, 64, 16, 1)
    weights = gp.gemm_moe_preshuffle(w13, w2, "bf16")
    ids, gates = gp.gemm_moe_route("bf16", x, router, 2)
    bad = [lambda: gp.gemm_moe("fp16", x.half(), router.half(), weights, 2), lambda: gp.gemm_moe("bf16", x[:, :32].contiguous(), router, weights, 2),
           lambda: gp.gemm_moe("bf16", x, router[:3], weights, 2), lambda: gp.gemm_moe("bf16", x, router, weights, 2, bias=bias.half()),
           lambda: gp.gemm_moe("bf16", x, router, weights, 2, residual=residual[:2]), lambda: gp.gemm_moe("bf16", x.cpu(), router, weights, 2),
           lambda: gp.gemm_moe("bf16", x, router, weights, 2, ids=ids.long()), lambda: gp.gemm_moe_route("bf16", x, router.cpu(), 2),
           lambda: gp.gemm_moe_experts("bf16", x, weights, ids.long(), gates), lambda: gp.gemm_moe_experts("bf16", x, weights, ids, gates.half()),
           lambda: gp.gemm_moe_experts("bf16", x, weights, ids[:2], gates), lambda: gp.gemm_moe_preshuffle(w13, w2[:, :32].contiguous(), "bf16")]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: gp.gemm_moe("bf16", x, router, weights, 5), lambda: gp.gemm_moe("fp8", x, router, weights, 2),
              lambda: gp.gemm_moe("bf16", x, router, weights, 2, workspace=torch.zeros(65536, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(gp.GemmError):
            f()
    monkeypatch.setattr(gp, "_device", lambda: 1)
    for f in (lambda: gp.gemm_moe("bf16", x, router, weights, 2), lambda: gp.gemm_moe_route("bf16", x, router, 2),
              lambda: gp.gemm_moe_experts("bf16", x, weights, ids, gates), lambda: gp.gemm_moe_preshuffle(w13, w2, "bf16")):
        with pytest.raises(ValueError, match="current device"):
            f()
