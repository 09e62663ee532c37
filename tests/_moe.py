"""References in 64 bits and error bounds for the mixture-of-experts layer: the router in float64 (the library's
own precision there), each pair's products as tests/_ffn.py bounds them (the weighted h is rounded to the type
between them), the sum over the choices in fp32."""
from __future__ import annotations

from tests import _ffn as F64

E32 = 2.0 ** -24


def route64(x, router, k, bias=None, score="softmax", normalize=True, scale=1.0):
    """(ids int32, weights float64): the k largest of score + bias, ties to the lowest expert."""
    import torch

    l = x.double() @ router.double().t()
    p = torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, 1)
    order = l if bias is None else p + bias.double()
    ids = torch.sort(order, dim=1, descending=True, stable=True)[1][:, :k]
    g = p.gather(1, ids)
    if normalize:
        g = g / g.sum(1, keepdim=True)
    return ids.to(torch.int32), scale * g


def experts64(dtype, x, w13, w2, ids, gates, act, residual):
    """(y, error before rounding)."""
    import torch

    M, k = ids.shape
    y = torch.zeros(M, x.shape[1], dtype=torch.float64, device=x.device)
    e, mag = torch.zeros_like(y), torch.zeros_like(y)
    for ex in range(w13.shape[0]):
        for j in range(k):
            rows = (ids[:, j] == ex).nonzero()[:, 0]
            if not len(rows):
                continue
            (h, _, _), (eh, _, _) = F64.gated64(x[rows], w13[ex], act)
            g = gates[rows, j].double()[:, None]
            h, eh = g * h, g.abs() * eh + E32 * (g * h).abs()
            o, eo = F64.product64(h, w2[ex].double(), F64.rounded(dtype, h, eh))
            y[rows] += o
            e[rows] += eo
            mag[rows] += o.abs() + eo
    if residual is not None:
        y = y + residual.double()
        mag = mag + residual.double().abs()
    return y, e + (k + 1) * E32 * mag
