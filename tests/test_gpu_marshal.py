"""The compiled marshalling of the linear layer's and the norms' calls against the binding's Python: the same results
and the same refusals."""
import pytest

pytestmark = pytest.mark.gpu


def _calls():
    import torch

    import dense_gemm_preshuffle_amd as gp

    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    half = lambda *s: normal(*s).bfloat16()
    x, res, z, dy, w = half(40, 512), half(40, 336), half(40, 336), half(40, 336), half(336, 512)
    w_shuf, bias = gp.gemm_linear_preshuffle(w, "bf16"), normal(336)
    long = half(40, 6720)
    long_w = gp.gemm_linear_preshuffle(half(336, 6720), "bf16")
    ws = gp.linear_workspace("bf16", 40, 336, 6720)
    a, b, c, d = (half(12, 264) for _ in range(4))
    v = [normal(264) for _ in range(4)]
    gate = normal(3, 264)
    kw = dict(norm_in="rms", w_in=v[0], b_in=v[1], gate=gate, norm_out="layer", w_out=v[2], b_out=v[3], scale=0.5, eps=1e-5)
    nws = gp.norm_backward_workspace("bf16", 12, 264, 3)
    lws = gp.linear_backward_workspace("bf16", 40, 336, 512)
    y, r = torch.empty_like(res), torch.empty_like(a)
    return {
        "linear": lambda: gp.gemm_linear("bf16", x, w_shuf),
        "linear all": lambda: gp.gemm_linear("bf16", x, w_shuf, bias=bias, act="gelu", residual=res, save=True, y=y),
        "linear split": lambda: gp.gemm_linear("bf16", long, long_w, workspace=ws),
        "linear own workspace": lambda: gp.gemm_linear("bf16", long, long_w),
        "linear backward": lambda: gp.gemm_linear_backward("bf16", dy, z, x, w, act="silu"),
        "linear backward one": lambda: gp.gemm_linear_backward("bf16", dy, None, x, None, want_dx=False, want_dbias=False, workspace=lws),
        "linear backward bias": lambda: gp.gemm_linear_backward("bf16", dy, None, None, None, want_dx=False, want_dw=False),
        "norm": lambda: gp.gemm_norm("bf16", a),
        "norm all": lambda: gp.gemm_norm("bf16", a, residual=b, r=r, **kw),
        "norm y": lambda: gp.gemm_norm("bf16", a, residual=b, want_r=False, **kw),
        "norm r": lambda: gp.gemm_norm("bf16", a, norm_in="rms", norm_out="none"),
        "norm backward": lambda: gp.gemm_norm_backward("bf16", a, b, c, d, **kw),
        "norm backward workspace": lambda: gp.gemm_norm_backward("bf16", a, None, c, d, workspace=nws, dx=r, **kw),
        "norm backward data": lambda: gp.gemm_norm_backward("bf16", a, b, None, d, want_params=False, want_dresidual=False),
        # refused
        "type": lambda: gp.gemm_linear("bf16", x.half(), w_shuf), "rows": lambda: gp.gemm_linear("bf16", x, w_shuf, residual=res[:4]),
        "z": lambda: gp.gemm_linear("bf16", x, w_shuf, z=z), "host": lambda: gp.gemm_norm("bf16", a.cpu()),
        "stride": lambda: gp.gemm_norm("bf16", a[:, ::2]), "gate": lambda: gp.gemm_norm("bf16", a, gate=normal(5, 264)),
        "vector": lambda: gp.gemm_norm("bf16", a, w_out=normal(263)), "half vector": lambda: gp.gemm_norm("bf16", a, w_out=half(264)),
        "eps": lambda: gp.gemm_norm("bf16", a, eps=-1.0), "nothing": lambda: gp.gemm_norm("bf16", a, want_r=False, norm_out="none"),
        "1-d": lambda: gp.gemm_norm("bf16", a[0]), "empty": lambda: gp.gemm_norm("bf16", a[:0]),
        "small workspace": lambda: gp.gemm_norm_backward("bf16", a, b, c, d, workspace=nws[:64], **kw),
        "dx": lambda: gp.gemm_norm_backward("bf16", a, b, c, d, want_dx=False, dx=r, **kw),
        "w": lambda: gp.gemm_linear_backward("bf16", dy, None, x, w[:, :256]), "x": lambda: gp.gemm_linear_backward("bf16", dy, None, None, w),
        "no z": lambda: gp.gemm_linear_backward("bf16", dy, None, x, w, act="silu"),
        "list": lambda: gp.gemm_norm("bf16", a, residual=[1.0]),
        "workspace list": lambda: gp.gemm_linear("bf16", x, w_shuf, workspace=[1]),
        "backward workspace list": lambda: gp.gemm_linear_backward("bf16", dy, None, x, w, workspace=[1]),
        "norm workspace list": lambda: gp.gemm_norm_backward("bf16", a, b, c, d, workspace=[1], **kw),
    }


def _flat(out):
    import torch

    return [out] if isinstance(out, torch.Tensor) else list(out)


def test_both_ways(monkeypatch):
    import torch

    import dense_gemm_preshuffle_amd as gp

    assert gp._compiled() is not None, "not built"
    calls = _calls()

    def run():
        got = {}
        for name, f in calls.items():
            try:
                got[name] = [None if v is None else v.clone() for v in _flat(f())]
            except Exception as e:
                got[name] = type(e)
        return got
    compiled = run()
    monkeypatch.setattr(gp, "_compiled", lambda: None)
    python = run()
    refused = list(calls).index("type")
    for i, name in enumerate(calls):
        a, b = compiled[name], python[name]
        if i >= refused:
            assert isinstance(a, type) and a is b, name
            continue
        assert len(a) == len(b) and all((p is None) == (q is None) and (p is None or torch.equal(p, q)) for p, q in zip(a, b)), name


def test_current_stream():
    """Calls under torch's stream context run on that stream, and their outputs belong to it."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    x = torch.randn(300, 4096, device="cuda").bfloat16()
    want = gp.gemm_norm("bf16", x)[1].clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        big = torch.randn(8192, 8192, device="cuda")
        for _ in range(5):
            big = big @ big * 1e-4
        y = x * 1                    # written after the products on the side stream
        out = gp.gemm_norm("bf16", y)[1]
    side.synchronize()
    assert torch.equal(out, want)


def test_the_interpreter_runs_meanwhile(tmp_path):
    """The entry points are called without the interpreter's lock, allocation and launch may wait: a copy of the module
    is bound to CPython's own question whether this thread holds the lock, whose 0 for "no" reads as success."""
    import ctypes
    import importlib.machinery
    import importlib.util
    import shutil

    import torch

    import dense_gemm_preshuffle_amd as gp

    path = shutil.copy(gp._compiled().__file__, tmp_path / "_marshal.so")
    loader = importlib.machinery.ExtensionFileLoader("_marshal", str(path))
    m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_marshal", loader))
    loader.exec_module(m)
    held = ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value
    assert ctypes.PyDLL(None).PyGILState_Check() == 1       # (as such a call would answer with the lock)
    m.bind(*[held] * 7)
    half, f32 = dict(dtype=torch.bfloat16, device="cuda"), dict(device="cuda")
    a, v, w = torch.zeros(4, 64, **half), torch.zeros(64, **f32), torch.zeros(32, 64, **half)
    laid, dy = torch.zeros(2 * 32 * 64, dtype=torch.uint8, device="cuda"), torch.zeros(4, 32, **half)
    bf16, here = gp.GP_BF16, torch.cuda.current_device()
    y = m.linear(bf16, a, laid, None, 0, None, False, None, None, None, here, 0)
    assert y is not None and y.shape == (4, 32)
    out = m.linear_backward(bf16, dy, None, a, w, 0, True, True, True, None, None, None, None, here, 0)
    assert [tuple(t.shape) for t in out] == [(4, 64), (32, 64), (32,)]
    out = m.norm(bf16, a, a, 1.0, 1, v, None, None, 1, v, None, 1e-6, True, None, None, here, 0)
    assert [tuple(t.shape) for t in out] == [(4, 64)] * 2
    out = m.norm_backward(bf16, a, a, a, a, 1.0, 1, v, None, None, 1, v, None, 1e-6, True, True, True, None, None, None, here, 0)
    assert [None if t is None else tuple(t.shape) for t in out] == [(4, 64)] * 2 + [(64,), None, None, (64,), None]


def test_calls_from_several_threads():
    """Each thread on a stream of its own, all at once: every call of a thread gives the bits of its first."""
    import threading

    import torch

    import dense_gemm_preshuffle_amd as gp

    wrong = []

    def work(k):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                gen = torch.Generator(device="cuda")
                gen.manual_seed(k)
                half = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
                x, w, dy, z, a = half(40 + k, 512), half(336, 512), half(40 + k, 336), half(40 + k, 336), half(60, 1024)
                w_shuf, w_out = gp.gemm_linear_preshuffle(w, "bf16"), torch.ones(1024, device="cuda")

                def step():
                    out = [gp.gemm_linear("bf16", x, w_shuf, act="silu")]
                    out += gp.gemm_linear_backward("bf16", dy, z, x, w, act="gelu")
                    out += gp.gemm_norm("bf16", a, w_out=w_out)
                    return out + [v for v in gp.gemm_norm_backward("bf16", a, a, a, a, w_out=w_out) if v is not None]
                first = [v.clone() for v in step()]
                for i in range(100):
                    if not all(torch.equal(p, q) for p, q in zip(step(), first)):
                        wrong.append((k, i))
                stream.synchronize()
        except Exception as e:
            wrong.append((k, repr(e)))
    threads = [threading.Thread(target=work, args=(k,)) for k in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:5]
