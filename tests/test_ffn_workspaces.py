"""Workspaces of the gated and 4-bit products: their counters are cleared, and nothing but them (host only)."""
import pytest

import dense_gemm_preshuffle_amd as gp


@pytest.fixture
def dirty(monkeypatch):
    """torch.empty gives memory that is not zero."""
    import torch

    def empty(n, dtype=None, device=None):
        return torch.full((n,), 255, dtype=dtype, device=device)
    monkeypatch.setattr(torch, "empty", empty)


def _check(ws, n):
    assert ws.numel() == n and ws.dtype.itemsize == 1
    assert not bool(ws[:65536].any()), "counters"
    # partial sums are written before they are read: clearing them cost a call that makes its own
    # workspace a pass over up to tens of megabytes
    assert bool((ws[65536:] == 255).all()), "cleared more than the counters"


def test_gated(dirty):
    n = gp.gemm_gated_workspace_size("bf16", 259, 2192, 6592)
    assert n > 1 << 22
    _check(gp.gated_workspace("bf16", 259, 2192, 6592, device="cpu"), n)
    assert gp.gated_workspace("bf16", 1, 7168, 2048, device="cpu") is None


def test_w4(dirty):
    import torch

    data = torch.full((gp.gemm_w4a16_weights_size(392, 19520, 64),), 1, dtype=torch.uint8)
    w = gp.W4Weights(data, torch.bfloat16, 392, 19520, 64, False, False)
    n = gp.gemm_w4a16_workspace_size(64, 392, 19520, 64)
    assert n > 1 << 17
    _check(gp.w4a16_workspace(64, w), n)
    assert gp.w4a16_workspace(1, gp.W4Weights(data, torch.bfloat16, 8192, 8192, 64, False, False)) is None
