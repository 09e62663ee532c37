"""The norms around a block and their backward pass on the GPU against float64."""
import pytest

from tests import _ffn as F64
from tests import _norm as N64
from tests._parity import say

pytestmark = pytest.mark.gpu


def _gen(seed):
    import torch

    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _case(dtype, M, H, G, affine, seed, mean=0.0):
    import torch

    t, gen = F64.torch_type(dtype), _gen(seed)

    def normal(*s, scale=1.0, mean=0.0):
        return torch.randn(*s, generator=gen, device="cuda") * scale + mean
    c = {"x": normal(M, H, mean=mean).to(t), "residual": normal(M, H, scale=2.0).to(t), "r": normal(M, H, mean=mean).to(t),
         "dy": normal(M, H).to(t), "dr": normal(M, H).to(t), "gate": normal(G, H) if G else None}
    for side in ("in", "out"):
        c["w_" + side] = normal(H, mean=1.0, scale=0.3)
        c["b_" + side] = normal(H) if affine else None
    return c


# rows: one, a workgroup's and one more, more than the workgroups at once; H: one
# piece, lanes that idle, every waves-by-pieces shape at its first and last size; G
# of every kind
SHAPES = [(1, 8, 0, "none", "rms"), (1, 4096, 1, "rms", "layer"), (3, 512, 3, "layer", "rms"), (5, 520, 1, "none", "layer"),
          (130, 1024, 0, "rms", "rms"), (64, 1032, 32, "layer", "layer"), (257, 2048, 1, "none", "rms"), (18, 2056, 9, "rms", "none"),
          (256, 4096, 256, "layer", "rms"), (77, 4104, 0, "none", "layer"), (33, 8192, 1, "rms", "layer"),
          (12, 8200, 4, "layer", "rms"), (40, 16384, 2, "rms", "layer"), (9000, 264, 6, "rms", "rms"),
          (2500, 2048, 5, "none", "layer"), (600, 16384, 1, "layer", "rms"),
          # rows shared unevenly by gate rows that leave CUs idle; both sides of 3000 rows
          (129 * 5, 264, 129, "none", "rms"), (86 * 7, 4096, 86, "rms", "layer"), (200 * 3, 8200, 200, "none", "layer"),
          (2999, 2568, 0, "rms", "rms"), (3000, 2568, 0, "rms", "rms")]


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,H,G,norm_in,norm_out", SHAPES)
def test_forward(dtype, M, H, G, norm_in, norm_out):
    import torch

    import dense_gemm_preshuffle_amd as gp

    affine = (M + H // 8) % 2 == 0
    c = _case(dtype, M, H, G, affine, M + H)
    t = F64.torch_type(dtype)
    say(f"norm {dtype} {M}x{H} gates {G} {norm_in} -> {norm_out}")
    kw = {"norm_in": norm_in, "gate": c["gate"], "norm_out": norm_out, "eps": 1e-5}
    if norm_in != "none":
        kw.update(w_in=c["w_in"], b_in=c["b_in"])
    if norm_out != "none":
        kw.update(w_out=c["w_out"], b_out=c["b_out"])
    (r, r_ok), (y, y_ok) = F64.guarded(M, H, t), F64.guarded(M, H, t)
    got = gp.gemm_norm(dtype, c["x"], residual=c["residual"], scale=0.5, r=r, y=None if norm_out == "none" else y, **kw)
    torch.cuda.synchronize()
    (rr, re), (yr, ye) = N64.forward64(c["x"], c["residual"], 0.5, norm_in, kw.get("w_in"), kw.get("b_in"), c["gate"],
                                       norm_out, kw.get("w_out"), kw.get("b_out"), 1e-5)
    F64.within(dtype, r, rr, re, "r")
    if norm_out != "none":
        F64.within(dtype, y, yr, ye, "y")
        # y alone, and in place of x; r in place of the residual
        only = gp.gemm_norm(dtype, c["x"], residual=c["residual"], scale=0.5, want_r=False, **kw)
        assert only[0] is None and torch.equal(only[1], y)
    else:
        assert got[1] is None
    x2, res2 = c["x"].clone(), c["residual"].clone()
    gp.gemm_norm(dtype, x2, residual=res2, scale=0.5, r=res2, y=None if norm_out == "none" else x2, **kw)
    torch.cuda.synchronize()
    assert torch.equal(res2, r) and (norm_out == "none" or torch.equal(x2, y))
    assert r_ok() and y_ok(), "written outside the outputs"


@pytest.mark.parametrize("dtype", F64.TYPES)
def test_forward_without_residual_and_far_mean(dtype):
    """No residual; layer norms of rows whose mean is 30 times their spread."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    c = _case(dtype, 37, 1040, 0, True, 5, mean=30.0)
    r, y = gp.gemm_norm(dtype, c["x"], norm_out="layer", w_out=c["w_out"], b_out=c["b_out"], eps=0.0)
    torch.cuda.synchronize()
    (rr, re), (yr, ye) = N64.forward64(c["x"], None, 1.0, "none", None, None, None, "layer", c["w_out"], c["b_out"], 0.0)
    assert torch.equal(r, c["x"])
    say("far mean", F64.within(dtype, y, yr, ye, "y"))


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,H,G,norm_in,norm_out", SHAPES)
def test_backward(dtype, M, H, G, norm_in, norm_out):
    import torch

    import dense_gemm_preshuffle_amd as gp

    affine = (M + H // 8) % 2 == 1
    c = _case(dtype, M, H, G, affine, M * 3 + H)
    t = F64.torch_type(dtype)
    say(f"norm backward {dtype} {M}x{H} gates {G} {norm_in} -> {norm_out}")
    kin, kout = norm_in != "none", norm_out != "none"
    kw = {"norm_in": norm_in, "w_in": c["w_in"] if kin else None, "b_in": c["b_in"] if kin else None, "gate": c["gate"],
          "norm_out": norm_out, "w_out": c["w_out"] if kout else None, "b_out": c["b_out"] if kout else None, "eps": 1e-5}
    dy, r = (c["dy"], c["r"]) if kout else (None, None)
    dr = c["dr"] if M % 4 or not kout else None
    x = c["x"] if kin or G else None
    (dx, ok1), (dres, ok2) = F64.guarded(M, H, t), F64.guarded(M, H, t)
    ws = torch.full((gp.gemm_norm_backward_workspace_size(dtype, M, H, G) + 4096,), 255, dtype=torch.uint8, device="cuda")
    got = gp.gemm_norm_backward(dtype, dy, dr, x, r, scale=0.5, dx=dx, dresidual=dres, workspace=ws[:-4096], **kw)
    again = gp.gemm_norm_backward(dtype, dy, dr, x, r, scale=0.5, want_dresidual=False, **kw)
    torch.cuda.synchronize()
    ref = N64.backward64(dy, dr, x, r, 0.5, norm_in, kw["w_in"], kw["b_in"], c["gate"], norm_out, kw["w_out"],
                         kw["b_out"], 1e-5)
    for name, v in got._asdict().items():
        given = {"dx": True, "dresidual": True}.get(name, kw.get(name[1:]) is not None)
        assert (v is not None) == given, name
        if v is None:
            continue
        if v.dtype == torch.float32:
            N64.within32(v, *ref[name], name)
        else:
            F64.within(dtype, v, *ref[name], name)
        if name != "dresidual":
            assert torch.equal(v, getattr(again, name)), f"{name} differs between calls"
    assert ok1() and ok2() and bool((ws[-4096:] == 255).all()), "written outside the outputs or the workspace"


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("H", [72, 2048, 8192])
def test_rows_do_not_mix(dtype, H):
    import torch

    import dense_gemm_preshuffle_amd as gp

    M = 1030
    c = _case(dtype, M, H, 0, True, 9)
    kw = dict(residual=c["residual"], norm_in="layer", w_in=c["w_in"], b_in=c["b_in"], norm_out="rms", w_out=c["w_out"])
    clean = gp.gemm_norm(dtype, c["x"], **kw)
    for row, v in ((0, float("nan")), (M - 1, float("inf")), (M // 2, float("-inf"))):
        bad = c["x"].clone()
        bad[row, H // 2] = v
        got = gp.gemm_norm(dtype, bad, **kw)
        torch.cuda.synchronize()
        keep = torch.arange(M, device="cuda") != row
        for a, b in zip(got, clean):
            assert torch.equal(a[keep], b[keep]) and not bool(torch.isfinite(a[row]).all())


def test_zero_rows_and_equal_rows():
    """A row of zeros gives the biases; a layer norm of a constant row too (eps > 0)."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    x = torch.zeros(3, 264, dtype=torch.bfloat16, device="cuda")
    x[1] = 3.0
    b = torch.arange(264, device="cuda", dtype=torch.float32)
    _, y = gp.gemm_norm("bf16", x, norm_out="layer", b_out=b, eps=1e-6)
    assert torch.equal(y, b.bfloat16().expand(3, -1))
    _, y = gp.gemm_norm("bf16", x[::2].contiguous(), norm_out="rms", b_out=b, eps=1e-6)
    assert torch.equal(y, b.bfloat16().expand(2, -1))


def test_large_offsets():
    """Matrices beyond 2^32 bytes: the last rows are those of a call of their own."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    M, H = 300000, 8192
    x = torch.zeros(M, H, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(7, H, device="cuda").bfloat16()
    x[-7:] = tail
    r, y = gp.gemm_norm("bf16", x, residual=x, norm_out="rms", eps=1e-6)
    r2, y2 = gp.gemm_norm("bf16", tail, residual=tail, norm_out="rms", eps=1e-6)
    assert torch.equal(r[-7:], r2) and torch.equal(y[-7:], y2) and not bool(r[:-7].any())
    g = gp.gemm_norm_backward("bf16", x, None, None, r, norm_out="rms", eps=1e-6, want_dresidual=False)
    g2 = gp.gemm_norm_backward("bf16", tail, None, None, r2, norm_out="rms", eps=1e-6, want_dresidual=False)
    assert torch.equal(g.dx[-7:], g2.dx)


def test_streams_graph_and_autograd():
    """Another stream, a captured and replayed pass, and the gradients as an autograd function would return them."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    c = _case("bf16", 300, 2056, 3, True, 11)
    kw = dict(norm_in="rms", w_in=c["w_in"], b_in=c["b_in"], gate=c["gate"], norm_out="layer", w_out=c["w_out"],
              b_out=c["b_out"])

    def step(stream=None):
        r, y = gp.gemm_norm("bf16", c["x"], residual=c["residual"], stream=stream, **kw)
        g = gp.gemm_norm_backward("bf16", c["dy"], c["dr"], c["x"], r, stream=stream, **kw)
        return [r, y, *g]
    want = [v.clone() for v in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        for o in out:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), k
        assert all(torch.equal(a, b) for a, b in zip(step(), want)), k


def test_another_device_is_refused(monkeypatch):
    import torch

    import dense_gemm_preshuffle_amd as gp

    x = torch.zeros(2, 8, dtype=torch.bfloat16, device="cuda")
    monkeypatch.setattr(gp, "_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        gp.gemm_norm("bf16", x)
    with pytest.raises(ValueError, match="current device"):
        gp.gemm_norm_backward("bf16", x, None, x, x)


@pytest.mark.parametrize("compiled", [True, False])
def test_a_gate_without_rows_is_refused(monkeypatch, compiled):
    """Zero rows of a gate divide no M: an error, not a call without a gate."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    if not compiled:
        monkeypatch.setattr(gp, "_compiled", lambda: None)
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    gate = torch.empty(0, 64, device="cuda")
    for call in (lambda: gp.gemm_norm("bf16", x, gate=gate), lambda: gp.gemm_norm_backward("bf16", x, x, x, x, gate=gate)):
        with pytest.raises(ValueError, match="gate"):
            call()


@pytest.mark.parametrize("seed", range(30))
def test_every_subset_of_the_gradients(seed):
    """Any of the backward pass's outputs may be missing, and x where none of the rest needs it: the same bits as of all
    of them together, which are within their bounds."""
    import random

    import torch

    import dense_gemm_preshuffle_amd as gp

    rng, gen = random.Random(seed), torch.Generator(device="cuda")
    gen.manual_seed(seed)
    G = rng.choice([0, 0, 1, rng.randint(2, 256)])
    M = max(G, 1) * rng.randint(1, max(1, 600 // max(G, 1)))
    H = 8 * rng.choice([rng.randint(1, 64), rng.randint(65, 256), rng.randint(257, 1024), rng.randint(1025, 2048)])
    M = M if M * H <= 1 << 22 else max(G, 1)
    kin, kout = rng.choice(["none", "rms", "layer"]), rng.choice(["none", "rms", "layer"])
    dtype = rng.choice(F64.TYPES)
    dt, t = gp.DTYPES[dtype], F64.torch_type(dtype)
    x, r, dy, dr = (torch.randn(M, H, generator=gen, device="cuda").to(t) for _ in range(4))
    w_in, b_in, w_out, b_out = (torch.randn(H, generator=gen, device="cuda") if kind != "none" and rng.random() < 0.7 else None
                                for kind in (kin, kin, kout, kout))
    gate = torch.randn(G, H, generator=gen, device="cuda") if G else None
    dy, r = (dy, r) if kout != "none" else (None, None)
    dr = None if dy is not None and rng.random() < 0.3 else dr
    possible = [True, True, kin != "none", kin != "none", G > 0, kout != "none", kout != "none"]
    say(f"seed {seed}: norm backward {dtype} {M}x{H} gates {G} {kin} -> {kout}")
    size = gp.gemm_norm_backward_workspace_size(dtype, M, H, G)

    def call(want):
        shapes = [(M, H)] * 2 + [(H,), (H,), (G, H), (H,), (H,)]
        out = [torch.full(s, float("nan"), dtype=t if i < 2 else torch.float32, device="cuda") if want[i] else None
               for i, s in enumerate(shapes)]
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        use_x = (kin != "none" and (want[0] or want[2])) or want[4]
        gp._check(gp.load_library().gemm_norm_backward(
            dt, gp._ptr(dy), gp._ptr(dr), gp._ptr(x) if use_x else None, gp._ptr(r), 0.7, gp.NORMS[kin], gp._ptr(w_in), gp._ptr(b_in),
            gp._ptr(gate), G, gp.NORMS[kout], gp._ptr(w_out), 1e-5, *map(gp._ptr, out), M, H, gp._ptr(ws) if any(want[2:]) else None,
            size, gp._stream(None)), "gemm_norm_backward")
        return out
    whole = call(possible)
    ref = N64.backward64(dy, dr, x, r, 0.7, kin, w_in, b_in, gate, kout, w_out, b_out, 1e-5)
    for name, v in zip(gp.NormGrads._fields, whole):
        if v is not None:
            (N64.within32(v, *ref[name], name) if v.dtype == torch.float32 else F64.within(dtype, v, *ref[name], name))
    wants = [[i == j for j in range(7)] for i in range(7) if possible[i]]
    wants += [[p and rng.random() < 0.5 for p in possible] for _ in range(6)]
    for want in wants:
        if any(want):
            assert all(a is None or torch.equal(a, b) for a, b in zip(call(want), whole)), want
