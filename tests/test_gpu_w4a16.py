"""Products with 4-bit weights and group scales on the GPU against float64."""
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


# rows: one, blocks and one more; columns: one, odd ones, a block and one more;
# K: one step, a part of a block, several blocks per wave; groups: inside a
# block, a block, several blocks, longer than K, and last groups cut short
SHAPES = [(1, 1, 32, 32, False), (1, 16, 128, 128, True), (1, 17, 160, 64, "wide"), (1, 67, 4096, 32, True),
          (1, 4096, 4096, 128, False), (1, 9001, 416, 256, True), (2, 33, 96, 256, "wide"), (3, 250, 1056, 32, False),
          (5, 4091, 7168, 64, True), (15, 48, 2080, 512, "wide"), (16, 130, 1152, 128, False), (17, 31, 288, 64, "wide"),
          (31, 1000, 4064, 1 << 20, True), (32, 64, 2048, 32, False), (33, 77, 640, 128, True), (48, 520, 896, 256, False),
          (64, 1040, 3008, 64, "wide"), (65, 99, 544, 32, True), (200, 264, 1312, 128, False)]


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,N,K,group,zeros", SHAPES)
def test_product(dtype, M, N, K, group, zeros):
    import torch

    import dense_gemm_preshuffle_amd as gp

    t = F64.torch_type(dtype)
    gen = _gen(M + 3 * N + K)
    x = _normal(gen, M, K, t=t)
    q, v, s, z = _w4.make(gen, dtype, N, K, group, zeros)
    act = F64.ACTS[(M + N + K // 32) % 4]
    bias = torch.randn(N, device="cuda", generator=gen) if N % 2 else None
    say(f"w4 {dtype} {M}x{N}x{K} group {group} zeros {zeros} {act}")
    w = gp.gemm_w4a16_preshuffle(q, s, z, group=group)
    y, ok = F64.guarded(M, N, t) if (M * N) % 8 == 0 else (torch.empty(M, N, dtype=t, device="cuda"), lambda: True)
    gp.gemm_w4a16(x, w, bias=bias, act=act, y=y)
    torch.cuda.synchronize()
    ref, err = _w4.product64(dtype, x, v, s, z, group)
    if bias is not None:
        ref = ref + bias.double()
        err = err + 2.0 ** -24 * ref.abs()
    a, _ = F64.act64(act, ref)
    err = 1.2 * err + 2.0 ** -20 * a.abs() + (0.8e-7 * ref.abs() if act == "gelu" else 0)
    say("  share of the bound", round(F64.within(dtype, y, a, err, "y"), 3))
    assert ok(), "written outside the output"
    assert torch.equal(gp.gemm_w4a16(x, w, bias=bias, act=act), y)


GATED = [(1, 1, 32, 32, False), (1, 40, 1056, 64, "wide"), (1, 2064, 4096, 128, True), (3, 515, 2048, 128, False),
         (7, 33, 4096, 256, True), (16, 17, 480, 32, "wide"), (20, 300, 1024, 128, True), (64, 129, 928, 64, False),
         (90, 48, 352, 256, True)]


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,F,K,group,zeros", GATED)
def test_gated(dtype, M, F, K, group, zeros):
    import torch

    import dense_gemm_preshuffle_amd as gp

    t = F64.torch_type(dtype)
    gen = _gen(M + 5 * F + K)
    x = _normal(gen, M, K, t=t)
    q, v, s, z = _w4.make(gen, dtype, 2 * F, K, group, zeros)
    w = gp.gemm_w4a16_preshuffle(q, s, z, group=group, gated=True)
    ref, err = _w4.product64(dtype, x, v, s, z, group)
    g, u, eg, eu = ref[:, :F], ref[:, F:], err[:, :F], err[:, F:]
    for act in F64.ACTS:
        say(f"w4 gated {dtype} {M}x{F}x{K} group {group} zeros {zeros} {act}")
        h = gp.gemm_w4a16_gated(x, w, act=act)
        torch.cuda.synchronize()
        a, _ = F64.act64(act, g)
        ea = 1.2 * eg + 2.0 ** -20 * a.abs() + (0.8e-7 * g.abs() if act == "gelu" else 0)
        eh = ea * u.abs() + (a.abs() + ea) * eu + 2.0 ** -23 * (a * u).abs()
        F64.within(dtype, h, a * u, eh, act)


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("zeros", [None, -8, 7, -128, 127])
def test_every_integer_is_exact(dtype, zeros):
    """Unit rows of x read single weights back: s (q - z) for all 16 integers, exact up to the rounding of y."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    t, N, K = F64.torch_type(dtype), 16, 256
    v = ((torch.arange(N, device="cuda")[:, None] + torch.arange(K, device="cuda")[None, :]) % 16 - 8).to(torch.int8)
    q = ((v[:, 0::2] & 15) | (v[:, 1::2] << 4)).view(torch.uint8)
    s = torch.full((N, K // 32), 0.375, dtype=t, device="cuda")
    z = None if zeros is None else torch.full((N, K // 32), zeros, dtype=torch.int8, device="cuda")
    w = gp.gemm_w4a16_preshuffle(q, s, z, group=32)
    y = torch.cat([gp.gemm_w4a16(x.contiguous(), w) for x in torch.eye(K, dtype=t, device="cuda").split(16)])
    want = (0.375 * (v.float() - (0 if zeros is None else zeros))).t().to(t)
    assert torch.equal(y, want)
    one = gp.gemm_w4a16(torch.eye(K, dtype=t, device="cuda")[37:38].contiguous(), w)
    assert torch.equal(one[0], want[37])


@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M", [1, 9, 40])
def test_rows_that_are_not_finite(dtype, M):
    """Infinities and NaN give what the formula gives, in their own row alone."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    t, N, K = F64.torch_type(dtype), 70, 416
    gen = _gen(M)
    x = _normal(gen, M, K, t=t)
    q, v, s, z = _w4.make(gen, dtype, N, K, 64, True)
    w = gp.gemm_w4a16_preshuffle(q, s, z, group=64)
    clean = gp.gemm_w4a16(x, w)
    weights = _w4.spread(s, 64, K) * (v.double() - _w4.spread(z, 64, K))
    inf = float("inf")
    for row, cells in ((0, {3: inf}), (M - 1, {415: -inf}), (M // 2, {100: inf, 101: inf}), (0, {7: float("nan")}),
                       (M - 1, {0: inf, 200: -inf})):
        bad = x.clone()
        for k, value in cells.items():
            bad[row, k] = value
        y = gp.gemm_w4a16(bad, w)
        torch.cuda.synchronize()
        # elementwise products, so that the pattern is the formula's and not a library's
        want = (bad[row].double()[None, :] * weights).sum(1)
        got = y[row].double()
        assert torch.equal(torch.isnan(got), torch.isnan(want)), (row, cells)
        assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)]), (row, cells)
        keep = torch.arange(M, device="cuda") != row
        assert torch.equal(y[keep], clean[keep])


def test_sums_that_overflow_on_the_way():
    """bf16 values whose group sums pass fp32's range although the results do not."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    N, K = 16, 128
    v = (torch.arange(N * K, device="cuda").view(N, K) % 3 - 1).to(torch.int8)
    q = ((v[:, 0::2] & 15) | (v[:, 1::2] << 4)).view(torch.uint8)
    s = torch.full((N, 1), 2.0 ** -10, dtype=torch.bfloat16, device="cuda")
    w = gp.gemm_w4a16_preshuffle(q, s, group=128)
    x = torch.full((2, K), 2.0 ** 121, dtype=torch.bfloat16, device="cuda")
    y = gp.gemm_w4a16(x, w)
    want = (x.double() @ (v.double() * 2.0 ** -10).t())
    torch.cuda.synchronize()
    F64.within("bf16", y, want, K * 2.0 ** -24 * (x.double().abs() @ (v.double().abs() * 2.0 ** -10).t()), "y")


def test_offsets_past_32_bits():
    """Weights of more than 2^31 bytes: the last columns."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    N, K, group = 280000, 16384, 128
    gen = _gen(0)
    q = torch.randint(0, 256, (N, K // 2), device="cuda", generator=gen, dtype=torch.uint8)
    s = torch.full((N, K // group), 0.01, dtype=torch.bfloat16, device="cuda")
    z = torch.randint(-4, 4, (N, K // group), device="cuda", generator=gen, dtype=torch.int8)
    x = _normal(gen, 2, K, t=torch.bfloat16)
    say("w4 offsets past 32 bits")
    w = gp.gemm_w4a16_preshuffle(q, s, z, group=group)
    y = gp.gemm_w4a16(x, w)
    torch.cuda.synchronize()
    for rows in (slice(0, 40), slice(N // 2, N // 2 + 40), slice(N - 40, N)):
        b = q[rows].to(torch.int16)
        v = torch.stack((b & 15, b >> 4), 2).flatten(1)
        v = torch.where(v > 7, v - 16, v).to(torch.int8)
        ref, err = _w4.product64("bf16", x, v, s[rows], z[rows], group)
        F64.within("bf16", y[:, rows], ref, err, str(rows))


def test_another_stream_and_graph_replays():
    import torch

    import dense_gemm_preshuffle_amd as gp

    for M, N, K, group in ((1, 4096, 4096, 128), (16, 515, 2080, 32), (40, 300, 1024, 64)):
        gen = _gen(M)
        q, v, s, z = _w4.make(gen, "bf16", 2 * N, K, group, True)
        w = gp.gemm_w4a16_preshuffle(q, s, z, group=group)
        wg = gp.gemm_w4a16_preshuffle(q, s, z, group=group, gated=True)
        x = _normal(gen, M, K, t=torch.bfloat16)

        def step(stream=None):
            return gp.gemm_w4a16(x, w, stream=stream), gp.gemm_w4a16_gated(x, wg, stream=stream)
        want = [o.clone() for o in step()]
        side = torch.cuda.Stream()
        for st in (side, side.cuda_stream):
            side.wait_stream(torch.cuda.current_stream())
            got = step(st)
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
        say(f"w4 streams and graph {M}x{N}x{K}: ok")


def test_binding_refusals():
    import torch

    import dense_gemm_preshuffle_amd as gp

    bf = torch.bfloat16
    q = torch.zeros(32, 64, dtype=torch.uint8, device="cuda")
    s = torch.ones(32, 4, dtype=bf, device="cuda")
    w = gp.gemm_w4a16_preshuffle(q, s, group=32)
    x = torch.ones(2, 128, dtype=bf, device="cuda")
    with pytest.raises(gp.GemmError):
        gp.gemm_w4a16_preshuffle(q, s.float(), group=32)
    with pytest.raises(ValueError):
        gp.gemm_w4a16_preshuffle(q, s, group=64)          # two scales per row expected
    with pytest.raises(gp.GemmError):
        gp.gemm_w4a16_preshuffle(q, s, group=48)
    with pytest.raises(ValueError):
        gp.gemm_w4a16_preshuffle(q, s, zeros=s, group=32)
    with pytest.raises(ValueError):
        gp.gemm_w4a16(x.half(), w)
    with pytest.raises(ValueError):
        gp.gemm_w4a16(x[:, :64].contiguous(), w)
    with pytest.raises(ValueError):
        gp.gemm_w4a16(torch.ones(128, 2, dtype=bf, device="cuda").t(), w)
    with pytest.raises(ValueError):
        gp.gemm_w4a16(x, w, bias=torch.zeros(32, dtype=bf, device="cuda"))
    with pytest.raises(ValueError):
        gp.gemm_w4a16_gated(x, w)
    with pytest.raises(gp.GemmError):
        gp.gemm_w4a16(x[:0], w)
    with pytest.raises(KeyError):
        gp.gemm_w4a16(x, w, act="tanh")
    assert float(gp.gemm_w4a16(x, w).float().abs().sum()) == 0.0
