"""Every kernel variant that a plan of the gated, 4-bit or backward products can name is compiled, and every compiled
one is reached (host only)."""
import os
import random
import re

import pytest

import dense_gemm_preshuffle_amd as gp
from tests import _w4_variants

CSRC = os.path.join(os.path.dirname(os.path.abspath(gp.__file__)), "csrc")


def _text(name):
    return open(os.path.join(CSRC, name)).read().replace("\\\n", " ")


def _ints(pattern, text):
    return [tuple(int(v) for v in m) for m in re.findall(pattern, text)]


def _tiles(name, skip):
    """{(tile_m, tile_n, split)} of a tile list in variants.hpp; skip: what stands between tile_n and split."""
    body = re.search(rf"#define {name}\(X[^)]*\)(.*)", _text("variants.hpp")).group(1)
    return {(int(a), int(b), s == "true") for a, b, s in re.findall(rf"(\d+), (\d+),{skip} (true|false)\)", body)}


W4 = set(_ints(r"GP_W4_CASE\(DT, ZV, (\d+), (\d+), (\d+), (\d+)\)", _text("launch_w4.hpp")))
SMALL = set(_ints(r"GP_GATED_SMALL_CASE\(DT, (\d+), (\d+), (\d+), (\d+)\)", _text("launch_gated.hpp")))
GATED = _tiles("GP_TILE_GATED", "")
ROWS = _tiles("GP_TILE_ROWS", r" \d+,")


def _w4(p):
    return (p["tile_m"] // 4, p["tile_n"] // 16, p["waves"], p["tile_k"] // 128)


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def test_lists_are_read():
    assert len(W4) == 16 and len(SMALL) == 11 and len(GATED) == 7 and len(ROWS) == 8


def test_w4_plans_are_compiled_and_all_reached():
    rng, seen = random.Random(2), set()
    for _ in range(6000):
        gated = rng.random() < 0.4
        p = gp.gemm_w4a16_plan(_log(rng, 1, 300), _log(rng, 1, 40000), 32 * _log(rng, 1, 1200),
                               rng.choice([32, 64, 128, 256, 4096]), gated, rng.random() < 0.5)
        assert p["kernel"] == gp.KERNEL_SPLITK and p["threads"] == 64 * p["waves"] and p["grid"] % p["ksplit"] == 0
        assert _w4(p) in W4, p
        assert not gated or p["tile_n"] % 32 == 0          # whole pairs of gate and up
        seen.add(_w4(p))
    assert seen == W4


def test_w4_shapes_of_the_numerical_tests_cover_every_variant():
    seen = set()
    for v, M, N, K, gated in _w4_variants.shapes():
        for ws in (False, True):
            assert _w4(gp.gemm_w4a16_plan(M, N, K, 64, gated, ws)) == v, (v, M, N, K, gated)
        seen.add(v)
    assert seen == W4


def test_w4_plan_and_workspace_agree():
    for args in ((64, 392, 19520, 128), (1, 1024, 28672, 128), (40, 200, 16384, 64, True), (1, 4096, 4096, 128)):
        p = gp.gemm_w4a16_plan(*args, with_workspace=True)
        assert p["workspace_bytes"] == gp.gemm_w4a16_workspace_size(*args) and (p["ksplit"] > 1) == (p["workspace_bytes"] > 0)
        assert gp.gemm_w4a16_plan(*args)["ksplit"] == 1


def test_gated_plans_are_compiled_and_all_reached():
    rng, small, tiles = random.Random(3), set(), set()
    for _ in range(12000):
        M, F, H = _log(rng, 1, 16384), 16 * _log(rng, 1, 1200), 32 * _log(rng, 1, 512)
        try:
            p = gp.gemm_gated_plan(rng.choice(("bf16", "fp16")), M, F, H)
        except gp.GemmError:
            continue                                        # too large
        assert p["workspace_bytes"] == gp.gemm_gated_workspace_size("bf16", M, F, H)
        if p["kernel"] == gp.KERNEL_SPLITK:
            small.add((p["tile_m"] // 8, p["tile_n"] // 32, p["waves"], p["tile_k"] // 64))
        else:
            assert p["kernel"] == gp.KERNEL_TILE and p["tile_m"] <= M and p["tile_n"] <= 2 * F
            tiles.add((p["tile_m"], p["tile_n"], p["ksplit"] > 1))
    assert small == SMALL and tiles == GATED


def test_tables_of_tile_times_name_compiled_tiles():
    """choose_tile_us picks from these tables alone, and splits K where a join time stands."""
    text = _text("ffn.hip")
    for name, compiled in (("kRowsTimes", ROWS), ("kGatedTimes", GATED)):
        body = re.search(rf"{name}\[\] = \{{(.*?)\}};", text, re.S).group(1)
        rows = [[float(v) for v in m.split(",")] for m in re.findall(r"\{([^{}]*)\}", body)]
        tiles = {(int(r[0]), int(r[1]), False) for r in rows} | {(int(r[0]), int(r[1]), True) for r in rows if r[4] > 0}
        assert len(rows) == 4 and tiles == compiled, name
    assert "gemm_tile_body<DT, 16, 64, 128, 128, EPI_ROWS" in _text("gemm_tile.hpp")   # plan_pair's one tile


def test_refusals():
    for bad, status in (((0, 64, 64, 32), 1), ((4, 0, 64, 32), 1), ((4, 64, 48, 32), 2), ((4, 64, 64, 48), 2)):
        with pytest.raises(gp.GemmError) as e:
            gp.gemm_w4a16_plan(*bad)
        assert e.value.status == status
    for bad, status in ((("bf16", 0, 32, 32), 1), (("bf16", 4, 24, 32), 2), (("fp8", 4, 32, 32), 3)):
        with pytest.raises(gp.GemmError) as e:
            gp.gemm_gated_plan(*bad)
        assert e.value.status == status
    lib = gp.load_library()
    assert lib.gemm_gated_plan(gp.DTYPES["bf16"], 4, 32, 32, None) == lib.gemm_w4a16_plan(4, 32, 64, 32, 0, 0, None) == 1


# sizes at which the better of the 256 x 256 and 128 x 256 tiles took at least 6% less time, and 3% less than the next
# smaller one, timed for 12 ms at a stretch on an MI355X (type, M, F, H: us on the first, us on the second)
@pytest.mark.parametrize("dtype,M,F,H,large,small", [("fp16", 6385, 6192, 8000, 973.1, 1039.7),
                                                     ("bf16", 721, 8976, 4032, 94.0, 100.5),
                                                     ("fp16", 1935, 4096, 6848, 171.3, 184.3),
                                                     ("bf16", 5298, 10416, 7200, 1180.0, 1284.3),
                                                     ("bf16", 711, 10368, 3904, 98.4, 108.0),
                                                     ("fp16", 1121, 6560, 2912, 128.2, 83.7),
                                                     ("fp16", 517, 11792, 3776, 160.0, 108.2),
                                                     ("fp16", 2386, 6576, 1376, 107.2, 80.0),
                                                     ("bf16", 1019, 4000, 8160, 165.8, 123.8),
                                                     ("bf16", 1920, 9744, 1760, 128.8, 113.3),
                                                     ("bf16", 874, 13168, 2720, 129.5, 114.0),
                                                     ("fp16", 6725, 1632, 4896, 213.2, 188.1)])
def test_gated_tile_where_it_matters(dtype, M, F, H, large, small):
    p = gp.gemm_gated_plan(dtype, M, F, H)
    assert (p["tile_m"], p["tile_n"]) == ((256, 256) if large < small else (128, 256))
