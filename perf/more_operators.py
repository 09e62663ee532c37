"""Measured cases of the operators around the feed-forward products: the linear
layer with its epilogue, the norms before and after a block with the residual,
and a mixture-of-experts layer for a few tokens. Listed sizes, a draw over the
same ranges, inputs, one pass in plain torch or through the library, the work it
cannot do without, and the result in 64 bits.

Operators (activations and weights in bf16 or fp16; biases, norm weights and
gates in fp32):

  linear           y = R + act(x w^T + b); a training forward keeps z = x w^T + b
  linear_backward  dz = dy * act'(z), dx = dz w, dw = dz^T x, db = sum of dz over rows
  norm             u = norm_in(x) * w_in + b_in (or x), r = s R + gate * u,
                   y = norm_out(r) * w_out + b_out; one gate row per M / G rows
  norm_backward    from dy and dr: the gradients of x, R, the gate and the norms' parameters
  moe              l = x wr^T, p = softmax(l) or sigmoid(l), the k experts of largest
                   p (+ bias), weights p normalised and scaled;
                   y = R + sum over them of weight * ((act(x wg^T) * (x wu^T)) wd^T)
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
_EPS = 1e-5


def _l(name, dtype, act, M, N, K, bias, residual, save=False):
    return {"name": name, "op": "linear", "dtype": dtype, "act": act, "M": M, "N": N, "K": K, "bias": bias,
            "residual": residual, "save": save}


def _lb(name, dtype, act, M, N, K):
    return {"name": name, "op": "linear_backward", "dtype": dtype, "act": act, "M": M, "N": N, "K": K}


def _n(name, dtype, M, H, norm_in, norm_out, groups, affine, residual=True, backward=False):
    # groups: rows of the gate (0: no gate); affine: the norms have biases
    return {"name": name, "op": "norm_backward" if backward else "norm", "dtype": dtype, "M": M, "H": H,
            "norm_in": norm_in, "norm_out": norm_out, "groups": groups, "affine": affine, "residual": residual}


def _m(name, dtype, M, E, k, H, F, score, bias, residual):
    return {"name": name, "op": "moe", "dtype": dtype, "act": "silu", "M": M, "E": E, "k": k, "H": H, "F": F,
            "score": score, "bias": bias, "residual": residual}


def listed():
    return [
        # one generated token through a square output projection, added to the residual stream
        _l("linear_one_token", "bf16", "none", 1, 4096, 4096, False, True),
        # a decode batch of odd size down from the inner width, with a bias
        _l("linear_batch", "fp16", "none", 37, 4096, 14336, True, True),
        # a training step's down projection into the residual stream
        _l("linear_train", "bf16", "none", 8192, 4096, 14336, True, True),
        # backward of the first layer of a plain feed-forward block, ragged batch
        _lb("linear_backward_batch", "fp16", "gelu", 2000, 7168, 2048),
        # backward of a small fine-tuning batch
        _lb("linear_backward_small", "bf16", "silu", 130, 2064, 2048),
        # one generated token: residual add and the next block's norm
        _n("norm_one_token", "bf16", 1, 4096, "none", "rms", 0, False),
        # a prompt: norms after one block and before the next, a learned gate per channel
        _n("norm_prompt", "fp16", 777, 7168, "rms", "rms", 1, False),
        # a training step's forward with layer norms, a gate per sequence
        _n("norm_train", "bf16", 16384, 4096, "none", "layer", 8, True),
        # its backward pass
        _n("norm_backward_train", "bf16", 16384, 4096, "none", "layer", 8, True, backward=True),
        # backward of a small batch with both norms
        _n("norm_backward_small", "fp16", 130, 2048, "rms", "rms", 1, False, backward=True),
        # one generated token through many small experts
        _m("moe_one_token", "bf16", 1, 64, 8, 2048, 1024, "softmax", False, True),
        # a decode batch of odd size through few large experts
        _m("moe_batch", "fp16", 33, 8, 2, 4096, 14336, "sigmoid", True, False),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, int(round(v / step)) * step)


def draw(rng):
    most = {"linear": work(listed()[2]), "norm": work(listed()[7]), "moe": work(listed()[11])}
    while True:
        op = rng.choice(["linear", "linear_backward", "norm", "norm_backward", "moe"])
        dtype = rng.choice(["bf16", "fp16"])
        if op in ("linear", "linear_backward"):
            # any number of tokens; widths in steps of 16 (backward: 32), K in steps of 32
            M = _log(rng, 1, 64) if op == "linear" and rng.random() < 0.4 else _log(rng, 16, 8192)
            c = {"op": op, "dtype": dtype, "act": rng.choice(["none", "none", "silu", "gelu", "relu"]), "M": M,
                 "N": _log(rng, 256, 14336, 16 if op == "linear" else 32), "K": _log(rng, 256, 14336, 32)}
            if op == "linear":
                c.update(bias=rng.random() < 0.5, residual=rng.random() < 0.7, save=rng.random() < 0.3)
        elif op in ("norm", "norm_backward"):
            # rows of 64 to 16384 in steps of 8; no gate, one per channel, or one per sequence
            G = rng.choice([0, 0, 1, _log(rng, 2, 16)])
            rows = _log(rng, 1, 16384 // max(G, 1))
            c = {"op": op, "dtype": dtype, "M": rows * max(G, 1), "H": _log(rng, 64, 16384, 8),
                 "norm_in": rng.choice(["none", "none", "rms", "layer"]), "norm_out": rng.choice(["rms", "layer"]),
                 "groups": G, "affine": rng.random() < 0.5, "residual": rng.random() < 0.8}
        else:
            # up to 64 tokens over 4 to 128 experts
            E = _log(rng, 4, 128)
            c = {"op": op, "dtype": dtype, "act": rng.choice(["silu", "gelu"]), "M": _log(rng, 1, 64), "E": E,
                 "k": rng.randint(1, min(8, E)), "H": _log(rng, 512, 4096, 32), "F": _log(rng, 256, 14336, 16),
                 "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.4,
                 "residual": rng.random() < 0.5}
            if 6.0 * E * c["F"] * c["H"] > 2.9e9:
                continue
        w, limit = work(c), most[op.split("_")[0]]
        if w["bytes"] <= 2 * limit["bytes"] and w["flops"] <= 2 * limit["flops"] and w["bytes"] <= 2.9e9 \
                and w["flops"] <= most["linear"]["flops"]:
            return c


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t = _TYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=gen) * scale).to(t)

    def params(*shape, mean=0.0, scale=0.2):
        return torch.randn(*shape, device="cuda", generator=gen) * scale + mean

    s = {"case": case}
    if case["op"] in ("linear", "linear_backward"):
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = normal(M, K)
        s["w"] = normal(N, K, scale=K ** -0.5)
        if case["op"] == "linear":
            s["b"] = params(N) if case["bias"] else None
            s["residual"] = normal(M, N, scale=2.0) if case["residual"] else None
        else:
            s["z"], s["dy"] = normal(M, N), normal(M, N, scale=0.1)
        if own:
            import dense_gemm_preshuffle_amd as gp

            if case["op"] == "linear":
                s["w_shuf"] = gp.gemm_linear_preshuffle(s["w"], case["dtype"])
                s["ws"] = gp.linear_workspace(case["dtype"], M, N, K)
            else:
                s["ws"] = gp.linear_backward_workspace(case["dtype"], M, N, K, act=case["act"])
        return s
    if case["op"] in ("norm", "norm_backward"):
        M, H, G = case["M"], case["H"], case["groups"]
        s["x"] = normal(M, H)
        s["residual"] = normal(M, H, scale=2.0) if case["residual"] else None
        s["scale"] = 1.0
        for side in ("in", "out"):
            on = case["norm_" + side] != "none"
            s["w_" + side] = params(H, mean=1.0) if on else None
            s["b_" + side] = params(H) if on and case["affine"] else None
        s["gate"] = params(G, H, mean=0.5) if G else None
        if case["op"] == "norm_backward":
            # the gradient of the norm's output, and what reaches r past the next block; r as the forward kept it
            s["dy"], s["dr"] = normal(M, H, scale=0.1), normal(M, H, scale=0.1)
            s["r"] = normal(M, H, scale=2.0)
            if own:
                import dense_gemm_preshuffle_amd as gp

                s["ws"] = gp.norm_backward_workspace(case["dtype"], M, H, G)
        return s
    M, E, H, F = case["M"], case["E"], case["H"], case["F"]

    def weights(rows, cols):
        w = torch.empty(E, rows, cols, dtype=t, device="cuda")
        for e in range(E):
            w[e].normal_(0.0, cols ** -0.5, generator=gen)
        return w

    s["x"] = normal(M, H)
    s["router"] = normal(E, H, scale=H ** -0.5)
    s["bias"] = params(E, scale=0.05) if case["bias"] else None
    s["residual"] = normal(M, H, scale=2.0) if case["residual"] else None
    w13, w2 = weights(2 * F, H), weights(H, F)
    if own:
        import dense_gemm_preshuffle_amd as gp

        # the experts' weights are laid out once, when the model is loaded
        s["experts"] = gp.gemm_moe_preshuffle(w13, w2, case["dtype"])
        s["ws"] = gp.moe_workspace(M, case["k"], s["experts"])
    else:
        s["w13"], s["w2"] = w13, w2
    return s


def _act(act, g):
    if act == "silu":
        return g * torch.sigmoid(g)
    if act == "gelu":
        return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))
    if act == "relu":
        return torch.clamp(g, min=0)
    return g


def _slope(act, g):
    if act == "silu":
        s = torch.sigmoid(g)
        return s * (1 + g * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    if act == "relu":
        return (g > 0).to(g.dtype)
    return torch.ones_like(g)


def _normalized(kind, v):
    """(v - mean) / sqrt(var + eps), or v / rms; and the reciprocal root."""
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    rs = torch.rsqrt((v * v).mean(1, keepdim=True) + _EPS)
    return v * rs, rs


def _normalized_grad(kind, n, rs, dn):
    d = dn - n * (dn * n).mean(1, keepdim=True)
    if kind == "layer":
        d = d - dn.mean(1, keepdim=True)
    return d * rs


def _plain_norm(s):
    c = s["case"]
    t = _TYPES[c["dtype"]]
    u = s["x"].float()
    if c["norm_in"] != "none":
        u = _normalized(c["norm_in"], u)[0] * s["w_in"]
        if s["b_in"] is not None:
            u = u + s["b_in"]
    if s["gate"] is not None:
        u = u * s["gate"].repeat_interleave(c["M"] // c["groups"], dim=0)
    r = u if s["residual"] is None else s["scale"] * s["residual"].float() + u
    y = _normalized(c["norm_out"], r)[0] * s["w_out"]
    if s["b_out"] is not None:
        y = y + s["b_out"]
    return {"r": r.to(t), "y": y.to(t)}


def _plain_norm_backward(s):
    c = s["case"]
    t = _TYPES[c["dtype"]]
    out = {}
    n, rs = _normalized(c["norm_out"], s["r"].float())
    dy = s["dy"].float()
    out["dw_out"] = (dy * n).sum(0)
    if s["b_out"] is not None:
        out["db_out"] = dy.sum(0)
    g = s["dr"].float() + _normalized_grad(c["norm_out"], n, rs, dy * s["w_out"])
    if s["residual"] is not None:
        out["dresidual"] = (s["scale"] * g).to(t)
    v = s["x"].float()
    if c["norm_in"] != "none":
        v, rs = _normalized(c["norm_in"], v)
    if s["gate"] is not None:
        u = v
        if c["norm_in"] != "none":
            u = u * s["w_in"]
            if s["b_in"] is not None:
                u = u + s["b_in"]
        out["dgate"] = (g * u).view(c["groups"], -1, c["H"]).sum(1)
        g = g * s["gate"].repeat_interleave(c["M"] // c["groups"], dim=0)
    if c["norm_in"] != "none":
        out["dw_in"] = (g * v).sum(0)
        if s["b_in"] is not None:
            out["db_in"] = g.sum(0)
        g = _normalized_grad(c["norm_in"], v, rs, g * s["w_in"])
    out["dx"] = g.to(t)
    return out


def _plain_moe(s):
    c = s["case"]
    x = s["x"].float()
    # the choice of experts is made in 64 bits: scores of two experts may lie close together
    l = s["x"].double() @ s["router"].double().t()
    if c["score"] == "sigmoid":
        p = torch.sigmoid(l)
    else:
        p = torch.exp(l - l.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    chosen = l if s["bias"] is None else p + s["bias"].double()
    ids = torch.sort(chosen, dim=1, descending=True, stable=True)[1][:, :c["k"]]
    weights = p.gather(1, ids)
    weights = (weights / weights.sum(1, keepdim=True)).float()
    y = torch.zeros_like(x) if s["residual"] is None else s["residual"].float()
    F = c["F"]
    if c["M"] * c["k"] < c["E"]:
        # few pairs of token and expert: the weights of each
        for j in range(c["k"]):
            z = (s["w13"][ids[:, j]].float() @ x[:, :, None])[:, :, 0]
            h = _act(c["act"], z[:, :F]) * z[:, F:]
            y = y + weights[:, j:j + 1] * (s["w2"][ids[:, j]].float() @ h[:, :, None])[:, :, 0]
    else:
        dense = torch.zeros(c["M"], c["E"], device=x.device).scatter(1, ids, weights)
        for e in range(c["E"]):
            z = x @ s["w13"][e].float().t()
            h = _act(c["act"], z[:, :F]) * z[:, F:]
            y = y + dense[:, e:e + 1] * (h @ s["w2"][e].float().t())
    return {"y": y.to(_TYPES[c["dtype"]]), "ids": ids.to(torch.int32), "weights": weights}


def _plain(s):
    c = s["case"]
    t = _TYPES[c["dtype"]]
    if c["op"] == "linear":
        z = s["x"].float() @ s["w"].float().t()
        if s["b"] is not None:
            z = z + s["b"]
        y = _act(c["act"], z)
        if s["residual"] is not None:
            y = s["residual"].float() + y
        return {"y": y.to(t), "z": z.to(t)} if c["save"] else {"y": y.to(t)}
    if c["op"] == "linear_backward":
        dz = s["dy"].float() * _slope(c["act"], s["z"].float())
        return {"dx": (dz @ s["w"].float()).to(t), "dw": (dz.t() @ s["x"].float()).to(t), "db": dz.sum(0)}
    return {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "moe": _plain_moe}[c["op"]](s)


def _library(s):
    import dense_gemm_preshuffle_amd as gp

    c = s["case"]
    t = c["dtype"]
    if c["op"] == "linear":
        out = gp.gemm_linear(t, s["x"], s["w_shuf"], bias=s["b"], act=c["act"], residual=s["residual"],
                             save=c["save"], workspace=s["ws"])
        return {"y": out[0], "z": out[1]} if c["save"] else {"y": out}
    if c["op"] == "linear_backward":
        dx, dw, db = gp.gemm_linear_backward(t, s["dy"], s["z"], s["x"], s["w"], act=c["act"], workspace=s["ws"])
        return {"dx": dx, "dw": dw, "db": db}
    if c["op"] == "norm":
        r, y = gp.gemm_norm(t, s["x"], residual=s["residual"], scale=s["scale"], norm_in=c["norm_in"], w_in=s["w_in"],
                            b_in=s["b_in"], gate=s["gate"], norm_out=c["norm_out"], w_out=s["w_out"], b_out=s["b_out"],
                            eps=_EPS)
        return {"r": r, "y": y}
    if c["op"] == "norm_backward":
        g = gp.gemm_norm_backward(t, s["dy"], s["dr"], s["x"], s["r"], scale=s["scale"], norm_in=c["norm_in"],
                                  w_in=s["w_in"], b_in=s["b_in"], gate=s["gate"], norm_out=c["norm_out"],
                                  w_out=s["w_out"], b_out=s["b_out"], eps=_EPS,
                                  want_dresidual=s["residual"] is not None, workspace=s["ws"])
        return {k: v for k, v in g._asdict().items() if v is not None}
    y, ids, weights = gp.gemm_moe(t, s["x"], s["router"], s["experts"], c["k"], bias=s["bias"], score=c["score"],
                                  act=c["act"], residual=s["residual"], workspace=s["ws"])
    return {"y": y, "ids": ids, "weights": weights}


def run(state):
    return _library(state) if own else _plain(state)


def work(case):
    M = case["M"]
    if case["op"] == "linear":
        N, K = case["N"], case["K"]
        outs = 1 + case["residual"] + case["save"]
        return {"bytes": 2 * (M * K + N * K + outs * M * N) + 4 * N * case["bias"], "flops": 2.0 * M * N * K}
    if case["op"] == "linear_backward":
        N, K = case["N"], case["K"]
        # without an activation the gradient is dy itself and z is not read
        reads = 1 if case["act"] == "none" else 2
        return {"bytes": 2 * (reads * M * N + 2 * M * K + 2 * N * K) + 4 * N, "flops": 4.0 * M * N * K}
    if case["op"] in ("norm", "norm_backward"):
        H, norms = case["H"], 1 + (case["norm_in"] != "none")
        vectors = norms * (1 + case["affine"]) + case["groups"]
        if case["op"] == "norm":
            # x and R read, r and y written
            return {"bytes": 2 * M * H * (3 + case["residual"]) + 4 * H * vectors, "flops": 10.0 * M * H * norms}
        # dy, dr and r read, x where its norm or the gate needs it; dx and dR written
        values = 4 + case["residual"] + (case["norm_in"] != "none" or case["groups"] > 0)
        return {"bytes": 2 * M * H * values + 8 * H * vectors, "flops": 20.0 * M * H * norms}
    E, k, H, F = case["E"], case["k"], case["H"], case["F"]
    # experts that are expected to be chosen by at least one token
    chosen = E * (1 - (1 - k / E) ** M)
    return {"bytes": 2 * (3 * F * H * chosen + E * H + M * H * (2 + case["residual"])) + 8 * M * k,
            "flops": 6.0 * M * k * F * H + 2.0 * M * E * H}


def _exact_gate(act, g):
    """act(g) and its derivative in 64 bits."""
    one = torch.ones_like(g)
    if act == "silu":
        e = torch.exp(-g.abs())
        p = torch.where(g >= 0, one, e) / (1 + e)          # 1 / (1 + exp(-g)), no overflow
        m = torch.where(g >= 0, e, one) / (1 + e)          # 1 - p
        return g * p, p + g * p * m
    if act == "gelu":
        p = 0.5 * torch.special.erfc(-g / 2.0 ** 0.5)      # the normal distribution function
        return g * p, p + g * torch.exp(-g.square() / 2) / (2 * math.pi) ** 0.5
    if act == "relu":
        return torch.where(g > 0, g, 0 * one), torch.where(g > 0, one, 0 * one)
    return g, one


def _exact_norm(kind, v):
    """Normalised rows, and a function that takes a gradient of them back to the rows."""
    H = v.shape[1]
    if kind == "none":
        return v, lambda d: d
    centred = v - v.sum(1, keepdim=True) / H if kind == "layer" else v
    sigma = (centred.square().sum(1, keepdim=True) / H + _EPS).sqrt()
    n = centred / sigma

    def back(d):
        along = (d * n).sum(1, keepdim=True) / H
        d = (d - along * n) / sigma
        return d - d.sum(1, keepdim=True) / H if kind == "layer" else d

    return n, back


def _exact_norms(case, s):
    H, G = case["H"], case["groups"]
    one, zero = torch.ones(H, dtype=torch.float64, device="cuda"), torch.zeros(H, dtype=torch.float64, device="cuda")

    def vec(v, other):
        return other if v is None else v.double()

    w_in, b_in, w_out, b_out = (vec(s[k], o) for k, o in (("w_in", one), ("b_in", zero), ("w_out", one),
                                                          ("b_out", zero)))
    gate = one.view(1, H) if s["gate"] is None else s["gate"].double()
    G = gate.shape[0]
    m, back_in = _exact_norm(case["norm_in"], s["x"].double())
    u = m * w_in + b_in
    if case["op"] == "norm":
        r = (u.view(G, -1, H) * gate.view(G, 1, H)).view(-1, H)
        if s["residual"] is not None:
            r = r + s["residual"].double() * s["scale"]
        return {"r": r, "y": _exact_norm(case["norm_out"], r)[0] * w_out + b_out}
    n, back_out = _exact_norm(case["norm_out"], s["r"].double())
    dy = s["dy"].double()
    t = s["dr"].double() + back_out(dy * w_out)
    du = (t.view(G, -1, H) * gate.view(G, 1, H)).view(-1, H)
    out = {"dx": back_in(du * w_in), "dw_out": (dy * n).sum(0)}
    if s["b_out"] is not None:
        out["db_out"] = dy.sum(0)
    if s["residual"] is not None:
        out["dresidual"] = t * s["scale"]
    if s["gate"] is not None:
        out["dgate"] = (t * u).view(G, -1, H).sum(1)
    if s["w_in"] is not None:
        out["dw_in"] = (du * m).sum(0)
    if s["b_in"] is not None:
        out["db_in"] = du.sum(0)
    return out


def _exact_moe(case, seed):
    global own
    was, own = own, False            # the weights as they were given
    try:
        s = prepare(case, seed)
    finally:
        own = was
    F = case["F"]
    x = s["x"].double()
    l = torch.mm(x, s["router"].double().t())
    if case["score"] == "sigmoid":
        e = torch.exp(-l.abs())
        p = torch.where(l >= 0, torch.ones_like(e), e) / (1 + e)
    else:
        p = torch.exp(l - l.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    order = l if s["bias"] is None else p + s["bias"].double()
    order = order.clone()
    ids, weights = [], []
    for _ in range(case["k"]):
        best = order.argmax(1)
        ids.append(best)
        weights.append(p.gather(1, best[:, None])[:, 0])
        order.scatter_(1, best[:, None], -math.inf)
    ids, weights = torch.stack(ids, 1), torch.stack(weights, 1)
    weights = weights / weights.sum(1, keepdim=True)
    y = torch.zeros_like(x) if s["residual"] is None else s["residual"].double()
    for e in range(case["E"]):
        token, slot = torch.nonzero(ids == e, as_tuple=True)
        if not len(token):
            continue
        w = s["w13"][e].double()
        h = _exact_gate(case["act"], torch.mm(x[token], w[:F].t()))[0] * torch.mm(x[token], w[F:].t())
        y.index_add_(0, token, torch.mm(h, s["w2"][e].double().t()) * weights[token, slot][:, None])
    return {"y": y, "ids": ids.to(torch.int32), "weights": weights}


def exact(case, seed):
    if case["op"] == "moe":
        return _exact_moe(case, seed)
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_backward"):
        return _exact_norms(case, s)
    x = s["x"].double()
    if case["op"] == "linear":
        z = torch.mm(x, s["w"].double().t())
        if s["b"] is not None:
            z += s["b"].double()
        y = _exact_gate(case["act"], z)[0]
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return {"y": y, "z": z} if case["save"] else {"y": y}
    dz = s["dy"].double() * _exact_gate(case["act"], s["z"].double())[1]
    return {"dx": torch.mm(dz, s["w"].double()), "dw": torch.mm(dz.t(), x), "db": dz.sum(0)}
