"""A transformer's feed-forward sublayer on the library, trained for a few steps, and its
mixture-of-experts form answering a token.

    python examples/sublayer.py

Training (bf16 weights, fp32 master copies, plain gradient descent):
    r, n        = gemm_norm(x, residual)          h, gate, up = gemm_gated(n, w)
    y           = gemm_linear(h, w_down, bias, residual=r)
    dh, dw_down, dbias = gemm_linear_backward(dy, None, h, w_down)
    dn, dw      = gemm_gated_backward(dh, gate, up, n, w)
    dx, dresidual, ..., dw_norm = gemm_norm_backward(dn, dy, x, r)
Serving:
    r, n = gemm_norm(x, residual)      y, ids, weights = gemm_moe(n, router, experts, k, residual=r)
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dense_gemm_preshuffle_amd as gp  # noqa: E402


class Sublayer:
    """y = r + (silu(n Wg^T) * (n Wu^T)) Wd^T + b, r = residual + x, n = rms(r) * w_norm; w holds Wg over Wu."""

    def __init__(self, hidden: int, inner: int, tokens: int, seed: int = 0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def normal(*shape, scale):
            return torch.randn(*shape, device="cuda", generator=gen) * scale
        self.master = [normal(2 * inner, hidden, scale=hidden ** -0.5), normal(hidden, inner, scale=inner ** -0.5)]
        self.w_norm, self.bias = torch.ones(hidden, device="cuda"), torch.zeros(hidden, device="cuda")
        # workspaces for this number of tokens, made once
        self.ws = [gp.gated_workspace("bf16", tokens, inner, hidden), gp.linear_workspace("bf16", tokens, hidden, inner),
                   gp.linear_backward_workspace("bf16", tokens, hidden, inner, act="none"),
                   gp.gated_backward_workspace("bf16", tokens, inner, hidden), gp.norm_backward_workspace("bf16", tokens, hidden)]
        self.update()

    def update(self):
        """The bf16 weights, and their layouts for the forward products."""
        self.w, self.down = (m.bfloat16() for m in self.master)
        self.w_shuf, self.down_shuf = gp.gemm_gated_preshuffle(self.w, "bf16"), gp.gemm_linear_preshuffle(self.down, "bf16")

    def forward(self, x, residual):
        self.x = x
        self.r, self.n = gp.gemm_norm("bf16", x, residual=residual, norm_out="rms", w_out=self.w_norm)
        self.h, self.gate, self.up = gp.gemm_gated("bf16", self.n, self.w_shuf, save=True, workspace=self.ws[0])
        return gp.gemm_linear("bf16", self.h, self.down_shuf, bias=self.bias, residual=self.r, workspace=self.ws[1])

    def backward(self, dy):
        """(dx, dresidual) and the gradients of w, the down weights, the bias and the norm's weights."""
        dh, d_down, d_bias = gp.gemm_linear_backward("bf16", dy, None, self.h, self.down, workspace=self.ws[2])
        dn, dw = gp.gemm_gated_backward("bf16", dh, self.gate, self.up, self.n, self.w, workspace=self.ws[3])
        g = gp.gemm_norm_backward("bf16", dn, dy, None, self.r, norm_out="rms", w_out=self.w_norm, workspace=self.ws[4])
        return (g.dx, g.dresidual), (dw, d_down, d_bias, g.dw_out)

    def step(self, grads, rate: float):
        for p, g in zip((*self.master, self.bias, self.w_norm), grads):
            p -= rate * g.float()
        self.update()


class Experts:
    """The sublayer with `count` experts, `k` of them for each token, for a few tokens at a time."""

    def __init__(self, sublayers, router, k: int, tokens: int):
        self.w_norm, self.router, self.k = sublayers[0].w_norm, router, k
        self.experts = gp.gemm_moe_preshuffle(torch.stack([s.w for s in sublayers]), torch.stack([s.down for s in sublayers]),
                                              "bf16")
        self.ws = gp.moe_workspace(tokens, k, self.experts)

    def forward(self, x, residual):
        r, n = gp.gemm_norm("bf16", x, residual=residual, norm_out="rms", w_out=self.w_norm)
        return gp.gemm_moe("bf16", n, self.router, self.experts, self.k, residual=r, workspace=self.ws)


def main(hidden: int = 1024, inner: int = 2048, tokens: int = 2048, steps: int = 20, rate: float = 0.3) -> dict:
    torch.manual_seed(20)
    block, target = Sublayer(hidden, inner, tokens), Sublayer(hidden, inner, tokens, seed=1)
    losses = []
    for i in range(steps):
        x, residual = (torch.randn(tokens, hidden, device="cuda").bfloat16() for _ in range(2))
        diff = block.forward(x, residual).float() - target.forward(x, residual).float()
        losses.append(float((diff * diff).mean()))
        # gradient of the mean over tokens of half the squared distance, times the width
        _, grads = block.backward((diff * (1.0 / tokens)).bfloat16())
        block.step(grads, rate)
        if i % 5 == 0 or i == steps - 1:
            print(f"step {i:3d}  loss {losses[-1]:.4f}", flush=True)
    experts = Experts([block, target, Sublayer(hidden, inner, tokens, seed=2)],
                      torch.randn(3, hidden, device="cuda").mul_(hidden ** -0.5).bfloat16(), 2, 1)
    x, residual = (torch.randn(1, hidden, device="cuda").bfloat16() for _ in range(2))
    y, ids, weights = experts.forward(x, residual)
    print(f"experts {ids[0].tolist()} with weights {[round(w, 3) for w in weights[0].tolist()]}", flush=True)
    return {"losses": losses, "y": y, "ids": ids, "weights": weights}


if __name__ == "__main__":
    main()
