"""Every tile that the GEMM planner picks for a gated product above 64 rows has a compiled gated form."""
import os
import random
import re

import dense_gemm_preshuffle_amd as gp

CSRC = os.path.join(os.path.dirname(os.path.abspath(gp.__file__)), "csrc")


def _list(name):
    txt = open(os.path.join(CSRC, "variants.hpp")).read().replace("\\\n", " ")
    body = re.search(rf"#define {name}\(X, DT\)(.*)", txt).group(1)
    return {tuple(int(v) for v in m) for m in re.findall(r"X\(DT, (\d+), (\d+), (\d+), (\d+), (\d+)\)", body)}


def test_gated_tiles_are_compiled():
    tiles, split = _list("GP_TILE_GATED"), _list("GP_TILE_GATED_KSPLIT")
    assert len(tiles) == 6 and len(split) == 2
    rng = random.Random(1)
    seen = set()
    for _ in range(12000):
        M = int(2 ** rng.uniform(6.03, 14))
        F = max(1, int(2 ** rng.uniform(0, 10.5))) * 16
        H = max(1, int(2 ** rng.uniform(0, 8))) * 64
        dtype = rng.choice(("bf16", "fp16"))
        try:
            p = gp.gemm_plan_ws(dtype, M, 2 * F, H)
        except gp.GemmError:
            continue
        if p["kernel"] != gp.KERNEL_TILE or p["tile_n"] < 128:
            continue      # the small kernel's
        pipe = 0 if p["pipeline"] == 1 else p["pipeline"]
        key = (p["mfma"], p["tile_m"], p["tile_n"], 2 * p["tile_k"], pipe)
        assert key in (split if p["ksplit"] > 1 else tiles), (dtype, M, F, H, p)
        seen.add((p["ksplit"] > 1, key))
    assert {k for s, k in seen if s} == split and {k for s, k in seen if not s} == tiles, seen
