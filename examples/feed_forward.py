"""A gated feed-forward block on the library: a few training steps, then the
trained block with 4-bit weights answering a few tokens.

    python examples/feed_forward.py

Training (bf16 weights, fp32 master copies, plain gradient descent):
    h, gate, up = gemm_gated(x, w)          y = gemm_bf16(h, w_down)
    dh, dw_down = gemm_backward(dy, h, w_down)
    dx, dw      = gemm_gated_backward(dh, gate, up, x, w)
Serving:
    y = gemm_w4a16(gemm_w4a16_gated(x, w4), w4_down)
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dense_gemm_preshuffle_amd as gp  # noqa: E402


class FeedForward:
    """y = (silu(x Wg^T) * (x Wu^T)) Wd^T; w holds Wg over Wu."""

    def __init__(self, hidden: int, inner: int, tokens: int, seed: int = 0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.master = [torch.randn(2 * inner, hidden, device="cuda", generator=gen) * hidden ** -0.5,
                       torch.randn(hidden, inner, device="cuda", generator=gen) * inner ** -0.5]
        # workspaces for this number of tokens, made once
        self.ws = gp.gated_workspace("bf16", tokens, inner, hidden)
        self.ws_gated = gp.gated_backward_workspace("bf16", tokens, inner, hidden)
        self.ws_down = gp.backward_workspace("bf16", tokens, hidden, inner)
        self.update()

    def update(self):
        """The bf16 weights, and their layouts for the forward products."""
        self.w, self.w_down = (m.bfloat16() for m in self.master)
        self.w_shuf = gp.gemm_gated_preshuffle(self.w, "bf16")
        self.down_shuf = gp.gemm_preshuffle_b(self.w_down, "bf16")

    def forward(self, x):
        self.x = x
        self.h, self.gate, self.up = gp.gemm_gated("bf16", x, self.w_shuf, save=True, workspace=self.ws)
        return gp.gemm_bf16(self.h, self.down_shuf)

    def backward(self, dy):
        dh, d_down = gp.gemm_backward("bf16", dy, self.h, self.w_down, workspace=self.ws_down)
        dx, dw = gp.gemm_gated_backward("bf16", dh, self.gate, self.up, self.x, self.w, workspace=self.ws_gated)
        return dx, (dw, d_down)

    def step(self, grads, rate: float):
        for m, g in zip(self.master, grads):
            m -= rate * g.float()
        self.update()


def quantize(w, group: int = 128):
    """[N, K] weights -> 4-bit integers, bf16 scales and int8 zero points per group of K."""
    N, K = w.shape
    v = w.float().view(N, K // group, group)
    lo, hi = v.amin(2), v.amax(2)
    scale = ((hi - lo) / 15).clamp(min=1e-8).bfloat16()
    zero = (-8 - lo / scale.float()).round().clamp(-128, 127)
    q = (v / scale.float()[..., None] + zero[..., None]).round().clamp(-8, 7).to(torch.int8).view(N, K)
    packed = ((q[:, 0::2] & 15) | (q[:, 1::2] << 4)).view(torch.uint8)
    return packed, scale, zero.to(torch.int8)


class Quantized:
    """The block on 4-bit weights, for a few tokens at a time."""

    def __init__(self, block: FeedForward, group: int = 128):
        self.w = gp.gemm_w4a16_preshuffle(*quantize(block.master[0], group), group=group, gated=True)
        self.down = gp.gemm_w4a16_preshuffle(*quantize(block.master[1], group), group=group)

    def forward(self, x):
        return gp.gemm_w4a16(gp.gemm_w4a16_gated(x, self.w), self.down)


def main(hidden: int = 1024, inner: int = 4096, tokens: int = 2048, steps: int = 30, rate: float = 0.4) -> dict:
    torch.manual_seed(1)
    block = FeedForward(hidden, inner, tokens)
    target = FeedForward(hidden, inner, tokens, seed=1)      # what the block is to learn
    losses = []
    for k in range(steps):
        x = torch.randn(tokens, hidden, device="cuda").bfloat16()
        diff = block.forward(x).float() - target.forward(x).float()
        losses.append(float((diff * diff).mean()))
        # gradient of the mean over tokens of half the squared distance, times the width
        _, grads = block.backward((diff * (1.0 / tokens)).bfloat16())
        block.step(grads, rate)
        if k % 5 == 0 or k == steps - 1:
            print(f"step {k:3d}  loss {losses[-1]:.4f}", flush=True)
    q = Quantized(block)
    x = torch.randn(3, hidden, device="cuda").bfloat16()
    small = FeedForward(hidden, inner, 3)
    small.master = block.master
    small.update()
    full, four = small.forward(x).float(), q.forward(x).float()
    error = float((full - four).norm() / full.norm())
    print(f"4-bit weights against bf16 ones: {100 * error:.1f}% of the answers' size", flush=True)
    return {"losses": losses, "error": error}


if __name__ == "__main__":
    main()
