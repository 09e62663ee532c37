"""Infinities and NaN in the activations and scales of the 4-bit products: the formula's pattern in every
variant of the kernel, other outputs untouched, and a bounded time."""
import pytest

from tests import _ffn as F64
from tests import _w4
from tests._parity import say

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def _gen(seed):
    import torch

    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _pattern(x, weights):
    """The formula's sums in float64, elementwise products, a row at a time."""
    import torch

    return torch.stack([(r.double()[None, :] * weights).sum(1) for r in x])


# rows of every variant, column blocks enough for the wide ones, K ending inside a block
@pytest.mark.parametrize("dtype", F64.TYPES)
@pytest.mark.parametrize("M,N,K,group,zeros", [(1, 40, 416, 64, True), (1, 8209, 416, 128, False), (1, 8209, 4128, 32, True),
                                               (4, 50, 288, 128, "wide"), (3, 8241, 288, 64, True), (16, 40, 288, 32, False),
                                               (9, 16401, 288, 128, True), (32, 12305, 160, 32, True),
                                               (48, 12305, 160, 64, False), (64, 8209, 160, 128, "wide"), (40, 33, 1056, 256, True)])
def test_activations_and_scales(dtype, M, N, K, group, zeros):
    import torch

    import dense_gemm_preshuffle_amd as gp

    t, gen = F64.torch_type(dtype), _gen(M + N + K)
    x = torch.randn(M, K, device="cuda", generator=gen).to(t)
    q, v, s, z = _w4.make(gen, dtype, N, K, group, zeros)
    clean = gp.gemm_w4a16(x, gp.gemm_w4a16_preshuffle(q, s, z, group=group))
    # rows: an infinity, two of both signs, a NaN; columns: scales of inf, -inf, NaN, and 0 beside an infinite x
    bad_x, bad_s = x.clone(), s.clone()
    bad_x[0, 37] = INF
    if M > 2:
        bad_x[M // 2, 3], bad_x[M // 2, K - 1] = -INF, INF
        bad_x[M - 1, K // 2] = NAN
    bad_s[N - 1, 0], bad_s[5, -1], bad_s[17, 0] = INF, -INF, NAN
    bad_s[33 if N > 33 else 30, 37 // group] = 0.0
    w = gp.gemm_w4a16_preshuffle(q, bad_s, z, group=group)
    say(f"w4 not finite {dtype} {M}x{N}x{K} group {group} zeros {zeros}")
    y, ok = F64.guarded(M, N, t)
    gp.gemm_w4a16(bad_x, w, y=y)
    torch.cuda.synchronize()
    weights = _w4.spread(bad_s, group, K) * (v.double() - (_w4.spread(z, group, K) if z is not None else 0.0))
    want, got = _pattern(bad_x, weights), y.double()
    assert ok(), "written outside the output"
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)])
    assert torch.equal(torch.isfinite(got), torch.isfinite(want))
    rows, cols = torch.isfinite(bad_x).all(1), torch.isfinite(bad_s).all(1) & (bad_s == s).all(1)
    assert torch.equal(y[rows][:, cols], clean[rows][:, cols])


@pytest.mark.parametrize("group,zeros", [(32, "wide"), (128, False), (1 << 20, True)])
def test_results_that_come_back_into_range(group, zeros):
    """bf16 sums that pass fp32's range on the way although the results do not, beside ordinary rows."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    M, N, K, gen = 18, 70, 256, _gen(group)
    q, v, s, z = _w4.make(gen, "bf16", N, K, group, zeros)
    s = (s.float() * 2.0 ** -12).bfloat16()
    x = torch.randn(M, K, device="cuda", generator=gen)
    x[11] = x[11].sign() * 2.0 ** 122       # times 16 and 256 of them: past 2^128
    x = x.bfloat16()
    y = gp.gemm_w4a16(x, gp.gemm_w4a16_preshuffle(q, s, z, group=group))
    torch.cuda.synchronize()
    ref, err = _w4.product64("bf16", x, v, s, z, group)
    F64.within("bf16", y, ref, err, "y")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M", [1, 16, 64])
def test_time(M, gated):
    """A row, or everything, that is not finite. One output after another, each a chain of K dependent steps,
    took tens of milliseconds at least (K times the latency of a load); going over K again in the matrix
    unit stays near the clean call's 30 to 80 us. 2 ms leaves room for a slow first step on both sides."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    N, K, gen = 4096 if gated else 8192, 28672, _gen(M)
    rows = 2 * N if gated else N
    q, _ = _w4.integers(gen, rows, K)
    s = torch.full((rows, K // 128), 0.01, dtype=torch.bfloat16, device="cuda")
    w = gp.gemm_w4a16_preshuffle(q, s, group=128, gated=gated)
    run = gp.gemm_w4a16_gated if gated else gp.gemm_w4a16
    x = torch.randn(M, K, device="cuda", generator=gen).bfloat16()

    def least(x):
        times = []
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            run(x, w)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)
    clean = least(x)
    one = x.clone()
    one[M // 2, 5] = NAN
    inf = x.clone()
    inf[0, 5] = INF
    all_nan = torch.full_like(x, NAN)
    times = {"clean": clean, "nan": least(one), "inf": least(inf), "all": least(all_nan)}
    say(f"w4 M {M} gated {gated} ms", {k: round(v, 4) for k, v in times.items()})
    assert max(times.values()) < 2.0, times
