"""The tile order of the gated product keeps its cache reuse whatever the number of tiles."""
import pytest

from tests._parity import say

pytestmark = pytest.mark.gpu


def test_tiles_that_8_does_not_divide():
    """Two sizes on the same tiles, 3713 and 3760 of them: nearly the same time for each tile. Row by row, as
    they went where 8 (the XCDs) does not divide their number, the first took 1.32 times as long per tile; the
    limit lies between."""
    import torch

    import dense_gemm_preshuffle_amd as gp

    M, H = 6000, 2560
    runs, tiles = [], []
    for F in (10000, 10240):
        p = gp.gemm_gated_plan("bf16", M, F, H)
        assert p["tile_m"] * p["tile_n"] == 128 * 256 and p["ksplit"] == 1
        tiles.append(p["grid"])
        x = torch.randn(M, H, device="cuda").bfloat16()
        w = gp.gemm_gated_preshuffle((torch.randn(2 * F, H, device="cuda") * H ** -0.5).bfloat16(), "bf16")
        h = torch.empty(M, F, dtype=torch.bfloat16, device="cuda")
        runs.append(lambda x=x, w=w, h=h: gp.gemm_gated("bf16", x, w, h=h))
    assert tiles == [3713, 3760]
    times = [[], []]
    for _ in range(8):
        for t, run in zip(times, runs):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            run()
            b.record()
            torch.cuda.synchronize()
            t.append(a.elapsed_time(b))
    per_tile = [min(t[2:]) / n for t, n in zip(times, tiles)]
    say("us per tile", [round(1e3 * v, 4) for v in per_tile])
    assert per_tile[0] < 1.2 * per_tile[1]
