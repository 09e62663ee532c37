"""The operators as a model runs them: a feed-forward sublayer forward and backward (norm, gated product, linear layer
into the residual stream), and a mixture-of-experts decode step, eagerly and in captured graphs."""
import pytest

from tests import _ffn as F64
from tests import _linear as L64
from tests import _moe as M64
from tests import _norm as N64
from tests._parity import say

pytestmark = pytest.mark.gpu


def _gen(seed):
    import torch

    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


class Sublayer:
    """r = residual + gate * x, out = r + (silu(n Wg^T) * (n Wu^T)) Wd^T + b with n = norm(r)."""

    def __init__(self, dtype, M, H, F, seed):
        import torch

        import dense_gemm_preshuffle_amd as gp

        self.gp, self.dtype, self.t, gen = gp, dtype, F64.torch_type(dtype), _gen(seed)

        def normal(*s, scale=1.0, mean=0.0):
            return torch.randn(*s, generator=gen, device="cuda") * scale + mean
        self.x, self.residual = normal(M, H).to(self.t), normal(M, H).to(self.t)
        self.gate, self.w_norm, self.b = normal(1, H, mean=1.0, scale=0.2), normal(H, mean=1.0, scale=0.2), normal(H, scale=0.2)
        self.w = normal(2 * F, H, scale=H ** -0.5).to(self.t)
        self.wd = normal(H, F, scale=F ** -0.5).to(self.t)
        self.dout = normal(M, H).to(self.t)
        self.w_shuf, self.wd_shuf = gp.gemm_gated_preshuffle(self.w, dtype), gp.gemm_linear_preshuffle(self.wd, dtype)

    def forward(self):
        gp, d = self.gp, self.dtype
        self.r, self.n = gp.gemm_norm(d, self.x, residual=self.residual, gate=self.gate, norm_out="rms", w_out=self.w_norm, eps=1e-5)
        self.h, self.g, self.u = gp.gemm_gated(d, self.n, self.w_shuf, save=True)
        self.out = gp.gemm_linear(d, self.h, self.wd_shuf, bias=self.b, residual=self.r)
        return self.out

    def backward(self):
        gp, d = self.gp, self.dtype
        self.dh, self.dwd, self.db = gp.gemm_linear_backward(d, self.dout, None, self.h, self.wd)
        self.dn, self.dw = gp.gemm_gated_backward(d, self.dh, self.g, self.u, self.n, self.w)
        self.grads = gp.gemm_norm_backward(d, self.dn, self.dout, self.x, self.r, gate=self.gate, norm_out="rms",
                                           w_out=self.w_norm, eps=1e-5)
        return [self.dwd, self.db, self.dw, *(v for v in self.grads if v is not None)]


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,H,F", [(1, 64, 16), (37, 544, 272), (300, 1056, 2064), (2048, 512, 1024)])
def test_each_stage_on_what_the_one_before_gave(dtype, M, H, F):
    """Every stage within its bound on the inputs that the stages before it really gave."""
    import torch

    s = Sublayer(dtype, M, H, F, M + H)
    s.forward()
    s.backward()
    torch.cuda.synchronize()
    (rr, re), (nr, ne) = N64.forward64(s.x, s.residual, 1.0, "none", None, None, s.gate, "rms", s.w_norm, None, 1e-5)
    refs, errs = F64.gated64(s.n, s.w, "silu")
    out = L64.forward64(s.h, s.wd, s.b, "none", s.r)[0]
    lb = L64.backward64(dtype, s.dout, None, s.h, s.wd, "none")
    d, ed = F64.gate_grad64(dtype, s.dh, s.g, s.u, "silu")
    nb = N64.backward64(s.dn, s.dout, s.x, s.r, 1.0, "none", None, None, s.gate, "rms", s.w_norm, None, 1e-5)
    shares = [F64.within(dtype, s.r, rr, re, "r"), F64.within(dtype, s.n, nr, ne, "n"),
              F64.within(dtype, s.h, refs[0], errs[0], "h"), F64.within(dtype, s.out, *out, "out"),
              F64.within(dtype, s.dh, *lb["dx"], "dh"), F64.within(dtype, s.dwd, *lb["dw"], "dwd"),
              N64.within32(s.db, *lb["dbias"], "db"),
              F64.within(dtype, s.dn, *F64.product64(d, s.w.double().t(), ed), "dn"),
              F64.within(dtype, s.dw, *F64.product64(d.t(), s.n.double().t(), ed.t()), "dw"),
              F64.within(dtype, s.grads.dx, *nb["dx"], "dx"), F64.within(dtype, s.grads.dresidual, *nb["dresidual"], "dresidual"),
              N64.within32(s.grads.dgate, *nb["dgate"], "dgate"), N64.within32(s.grads.dw_out, *nb["dw_out"], "dw_out")]
    say(f"sublayer {dtype} {M}x{H}x{F}: largest share of a bound {max(shares):.3f}")


def test_gradients_against_differences():
    """Each gradient of the whole sublayer along a direction against central differences in float64."""
    import torch

    s = Sublayer("fp16", 96, 256, 192, 5)
    s.forward()
    s.backward()
    names = {"x": s.grads.dx, "residual": s.grads.dresidual, "gate": s.grads.dgate, "w_norm": s.grads.dw_out, "w": s.dw,
             "wd": s.dwd, "b": s.db}

    def loss(p):
        r = p["residual"] + p["gate"] * p["x"]
        n = r * (r * r).mean(1, keepdim=True).add(1e-5).rsqrt() * p["w_norm"]
        z = n @ p["w"].t()
        F = z.shape[1] // 2
        out = r + (F64.act64("silu", z[:, :F])[0] * z[:, F:]) @ p["wd"].t() + p["b"]
        return float((out * s.dout.double()).sum())
    p = {n: getattr(s, n).double() for n in names}
    gen, step = _gen(9), 1e-6
    for name, g in names.items():
        d = torch.randn(p[name].shape, generator=gen, device="cuda", dtype=torch.float64)
        ends = [loss({**p, name: p[name] + e * d}) for e in (step, -step)]
        diff = (ends[0] - ends[1]) / (2 * step)
        got = float((g.double() * d).sum())
        # each entry of a gradient passes up to 8 roundings to fp16 on its way (n, h, gate, up, dh, dg and du, dn,
        # itself; half a step, 2^-11, each), and a random direction adds the entries' errors up like their values:
        # 8 of them of the gradient's norm, four standard deviations
        allowed = float(g.double().norm()) * 8 * 2.0 ** -11 * 4
        say(f"differences {name}: {got:.6g} against {diff:.6g}, allowed {allowed:.3g}")
        assert abs(got - diff) <= allowed, name


def test_training_step_in_a_graph():
    """Captured, replayed between eager steps, on workspaces of the calls' own: the same bits each time."""
    import torch

    s = Sublayer("bf16", 260, 544, 528, 3)
    want = [v.clone() for v in [s.forward(), *s.backward()]]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = [s.forward(), *s.backward()]
    for k in range(4):
        for o in out:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), k
        e = Sublayer("bf16", 260, 544, 528, 3)
        assert all(torch.equal(a, b) for a, b in zip([e.forward(), *e.backward()], want)), k


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M", [1, 5, 24])
def test_decode_step_with_experts(dtype, M):
    """norm -> experts into the residual stream -> norm -> linear head, twice in graphs that share one workspace."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    t, E, k, H, F, V, gen = F64.torch_type(dtype), 16, 4, 544, 144, 1040, _gen(M)

    def normal(*s, scale=1.0):
        return (torch.randn(*s, generator=gen, device="cuda") * scale).to(t)
    x, residual, router = normal(M, H), normal(M, H), normal(E, H, scale=H ** -0.5)
    w13, w2, head = normal(E, 2 * F, H, scale=H ** -0.5), normal(E, H, F, scale=F ** -0.5), normal(V, H, scale=H ** -0.5)
    w_norm = torch.rand(H, generator=gen, device="cuda") + 0.5
    experts, head_shuf = gp.gemm_moe_preshuffle(w13, w2, dtype), gp.gemm_linear_preshuffle(head, dtype)
    ws = torch.zeros(max(gp.gemm_moe_workspace_size(dtype, M, F, H, E, k), gp.gemm_linear_workspace_size(dtype, M, V, H)),
                     dtype=torch.uint8, device="cuda")

    def step():
        r, n = gp.gemm_norm(dtype, x, residual=residual, norm_out="rms", w_out=w_norm)
        y, ids, gates = gp.gemm_moe(dtype, n, router, experts, k, residual=r, workspace=ws)
        _, n2 = gp.gemm_norm(dtype, y, norm_out="rms", w_out=w_norm, want_r=False)
        return r, n, y, ids, gates, n2, gp.gemm_linear(dtype, n2, head_shuf, workspace=ws)
    r, n, y, ids, gates, n2, logits = want = step()
    torch.cuda.synchronize()
    assert torch.equal(ids, M64.route64(n, router, k)[0])
    F64.within(dtype, y, *M64.experts64(dtype, n, w13, w2, ids, gates, "silu", r), "y")
    F64.within(dtype, n2, *N64.forward64(y, None, 1.0, "none", None, None, None, "rms", w_norm, None, 1e-6)[1], "n2")
    F64.within(dtype, logits, *L64.forward64(n2, head, None, "none", None)[0], "logits")
    want = [v.clone() for v in want]
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, step()))
    for _ in range(3):
        for g, out in graphs:
            for o in out:
                o.zero_()
            g.replay()
            assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for a, b in zip(step(), want))
    assert not bool(ws[:65536].any())
