"""Plans of the backward passes (host only): every product on a compiled kernel, and on the planner's own plan for
it where the operands are laid out for the preshuffled kernels."""
import random

import pytest

import dense_gemm_preshuffle_amd as gp
from tests.test_ffn_plans import ROWS, _log

# sizes (M, N, K) whose first product's preshuffled plan splits K and whose second's does not
SIZES = [(1322, 2432, 1760, False), (748, 1024, 2784, True), (1200, 1984, 1184, True), (1983, 4368, 1856, True),
         (3421, 4976, 1728, True), (1313, 3888, 4320, True), (1587, 4176, 2528, True), (1320, 2144, 4352, True)]


def _pad(k):
    unit = 1024 if k >= 16384 else 256 if k >= 4096 else 64
    return -(-k // unit) * unit


def _whole(dtype, M, N, K, gated, want_da, want_db):
    """Checks a plan; the kinds of its products."""
    da, db = gp.gemm_backward_plan(dtype, M, N, K, want_da, want_db, gated)
    assert (da is not None, db is not None) == (want_da, want_db)
    rows, k_da, k_db = (2 * N, _pad(2 * N), _pad(M)) if gated else (N, N, _pad(M))
    kinds = set()
    for p, (m, n, k) in ((da, (M, K, k_da)), (db, (rows, K, k_db))):
        if p is None:
            continue
        if p["kernel"] in (gp.KERNEL_ROWS, gp.KERNEL_PAIR):
            assert (p["tile_m"], p["tile_n"], p["ksplit"] > 1) in ROWS, p
            assert p["kernel"] == gp.KERNEL_ROWS or (p["tile_m"], p["tile_n"]) == (64, 128)
        else:
            assert p["kernel"] == gp.KERNEL_TILE
            want = gp.gemm_plan_ws(dtype, m, n, k)
            assert {f: p[f] for f in p if f != "workspace_bytes"} == {f: want[f] for f in p if f != "workspace_bytes"}, \
                (dtype, M, N, K, gated, p, want)
        kinds.add((p["kernel"], p["ksplit"] > 1))
    if want_da and want_db:
        assert (da["kernel"] == gp.KERNEL_PAIR) == (db["kernel"] == gp.KERNEL_PAIR)
    return kinds


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,N,K,gated", SIZES)
def test_second_product_has_a_plan_of_its_own(dtype, M, N, K, gated):
    _whole(dtype, M, N, K, gated, True, True)
    _whole(dtype, M, N, K, gated, False, True)


def test_no_split_no_partial_sums():
    """db alone on an unsplit preshuffled plan: a workspace of its two copies and nothing else."""
    M, F, H = 8192, 14336, 4096
    db = gp.gemm_backward_plan("bf16", M, F, H, False, True, True)[1]
    assert (db["kernel"], db["ksplit"]) == (gp.KERNEL_TILE, 1)
    assert gp.gemm_gated_backward_workspace_size("bf16", M, F, H, False, True) == M * (2 * F + H) * 2 == db["workspace_bytes"]


def test_random_sizes():
    rng, kinds = random.Random(4), set()
    for _ in range(6000):
        M, N, K = _log(rng, 1, 8192), 32 * _log(rng, 1, 512), 32 * _log(rng, 1, 512)
        da = rng.random() < 0.8
        try:
            kinds |= _whole(rng.choice(["bf16", "fp16"]), M, N, K, rng.random() < 0.5, da, not da or rng.random() < 0.8)
        except gp.GemmError:
            continue                                       # too large
    assert kinds >= {(gp.KERNEL_ROWS, False), (gp.KERNEL_ROWS, True), (gp.KERNEL_PAIR, False), (gp.KERNEL_PAIR, True),
                     (gp.KERNEL_TILE, False)}


def test_refusals():
    for bad, status in ((("bf16", 0, 32, 32), 1), (("bf16", 4, 48, 32), 2), (("fp8", 4, 32, 32), 3)):
        with pytest.raises(gp.GemmError) as e:
            gp.gemm_backward_plan(*bad)
        assert e.value.status == status
    with pytest.raises(gp.GemmError) as e:
        gp.gemm_backward_plan("bf16", 4, 32, 32, False, False)
    assert e.value.status == 1
    assert gp.load_library().gemm_backward_plan(gp.DTYPES["bf16"], 4, 32, 32, 1, 1, 0, None, None) == 1
