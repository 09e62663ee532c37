"""Measured cases of the gated feed-forward operators and of the products with
4-bit weights: listed sizes, a draw over the same ranges, inputs, one pass in
plain torch or through the library, the work it cannot do without, and the
result in 64 bits.

Operators (x [M, H] and w [2F, H] in bf16 or fp16; w holds the F gate rows,
then the F up rows):

  gated           g = x w[:F]^T, u = x w[F:]^T, h = act(g) * u; a training
                  forward also keeps g and u in the input type
  gated_backward  from dh and the kept g, u:
                  dg = dh * u * act'(g), du = dh * act(g),
                  dx = [dg du] w, dw = [dg du]^T x
  w4a16           y = x W^T + bias with W[n, k] = s[n, k/G] (q[n, k] - z[n, k/G]),
                  q a 4-bit integer, s (and optionally z) per group of G
                  consecutive k
  w4a16_gated     the gated form on such weights (gate rows, then up rows)
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _g(name, dtype, act, M, H, F, save=False):
    return {"name": name, "op": "gated", "dtype": dtype, "act": act, "M": M, "H": H, "F": F, "save": save}


def _b(name, dtype, act, M, H, F):
    return {"name": name, "op": "gated_backward", "dtype": dtype, "act": act, "M": M, "H": H, "F": F}


def _q(name, dtype, M, N, K, group, zeros, bias=False):
    return {"name": name, "op": "w4a16", "dtype": dtype, "M": M, "N": N, "K": K, "group": group, "zeros": zeros,
            "bias": bias}


def _qg(name, dtype, act, M, F, K, group, zeros):
    return {"name": name, "op": "w4a16_gated", "dtype": dtype, "act": act, "M": M, "F": F, "K": K, "group": group,
            "zeros": zeros}


def listed():
    return [
        # one generated token: bound by reading the weights
        _g("gated_one_token", "bf16", "silu", 1, 2048, 7168),
        # a decode batch of odd size, columns that no tile divides
        _g("gated_batch", "fp16", "gelu", 37, 4096, 7184),
        # a chunk of a prompt, of odd length
        _g("gated_chunk", "bf16", "silu", 509, 4096, 7168),
        # a training step's forward: the pre-activations are kept
        _g("gated_train", "bf16", "silu", 8192, 4096, 14336, True),
        # backward of a small ragged batch (fine tuning)
        _b("backward_small", "fp16", "gelu", 130, 2048, 2064),
        # backward of an ordinary batch
        _b("backward_batch", "fp16", "silu", 2000, 4096, 7168),
        # backward of a training step, the largest case
        _b("backward_train", "bf16", "silu", 8192, 4096, 14336),
        # one token through a square projection: latency
        _q("w4_square", "bf16", 1, 4096, 4096, 128, False),
        # one token, small groups with zero points
        _q("w4_small_groups", "fp16", 1, 7168, 2048, 32, True),
        # one token through the largest down projection: weight bandwidth
        _q("w4_down", "bf16", 1, 8192, 28672, 128, True, True),
        # a batch of sequences, an odd number of output columns
        _q("w4_batch", "fp16", 16, 4091, 7168, 64, False),
        # a few tokens (speculative decoding) through gate and up
        _qg("w4_gated", "bf16", "silu", 3, 14336, 4096, 128, True),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, int(round(v / step)) * step)


def draw(rng):
    most = {"flops": 8.0 * 8192 * 4096 * 14336, "bytes": 2e9}
    while True:
        op = rng.choice(["gated", "gated_backward", "w4a16", "w4a16_gated"])
        dtype, act = rng.choice(["bf16", "fp16"]), rng.choice(["silu", "silu", "gelu", "relu", "none"])
        if op in ("gated", "gated_backward"):
            # hidden sizes in steps of 32, feed-forward sizes in steps of 16, any number of tokens
            c = {"op": op, "dtype": dtype, "act": act, "M": _log(rng, 1 if op == "gated" else 32, 8192),
                 "H": _log(rng, 256, 8192, 32), "F": _log(rng, 256, 16384, 16)}
            if op == "gated":
                c["save"] = rng.random() < 0.4
        else:
            # 4-bit weights: one token in half of the cases, up to 64 otherwise; odd output sizes
            M = 1 if rng.random() < 0.5 else _log(rng, 1, 64)
            group = rng.choice([32, 64, 128, 128, 256])
            c = {"op": op, "dtype": dtype, "M": M, "K": _log(rng, 256, 28672, 32), "group": group,
                 "zeros": rng.random() < 0.5}
            if op == "w4a16":
                c["N"], c["bias"] = _log(rng, 64, 32768), rng.random() < 0.3
            else:
                c["F"], c["act"] = _log(rng, 64, 16384), act
        w = work(c)
        if w["flops"] <= most["flops"] and w["bytes"] <= most["bytes"]:
            return c


def _int4(gen, rows, cols):
    """Normal weights rounded to 4-bit integers, two per byte, the even k in the low nibble."""
    q = (torch.randn(rows, cols, device="cuda", generator=gen) * 2.5).round_().clamp_(-8, 7).to(torch.int8)
    return ((q[:, 0::2] & 15) | (q[:, 1::2] << 4)).view(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t = _TYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=gen) * scale).to(t)

    s = {"case": case}
    if case["op"] in ("gated", "gated_backward"):
        M, H, F = case["M"], case["H"], case["F"]
        s["x"] = normal(M, H)                              # a normalised hidden state
        s["w"] = normal(2 * F, H, scale=H ** -0.5)
        if case["op"] == "gated_backward":
            s["gate"], s["up"] = normal(M, F), normal(M, F)
            s["dh"] = normal(M, F, scale=0.1)
        if own:
            import dense_gemm_preshuffle_amd as gp

            if case["op"] == "gated":
                # inference weights are laid out once, when the model is loaded
                s["w_shuf"] = gp.gemm_gated_preshuffle(s["w"], case["dtype"])
                s["ws"] = gp.gated_workspace(case["dtype"], M, F, H)
            else:
                s["ws"] = gp.gated_backward_workspace(case["dtype"], M, F, H)
        return s
    gated = case["op"] == "w4a16_gated"
    M, K, G = case["M"], case["K"], case["group"]
    N = 2 * case["F"] if gated else case["N"]
    groups = -(-K // G)
    s["x"] = normal(M, K)
    s["q"] = _int4(gen, N, K)
    s["scales"] = ((torch.rand(N, groups, device="cuda", generator=gen) + 0.5) * (0.4 * K ** -0.5)).to(t)
    s["zeros"] = None
    if case["zeros"]:
        s["zeros"] = torch.randint(-3, 4, (N, groups), device="cuda", generator=gen, dtype=torch.int8)
    s["bias"] = None
    if case.get("bias"):
        s["bias"] = torch.randn(N, device="cuda", generator=gen)
    if own:
        import dense_gemm_preshuffle_amd as gp

        s["weights"] = gp.gemm_w4a16_preshuffle(s["q"], s["scales"], s["zeros"], group=G, gated=gated)
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


def _dequantize(q, scales, zeros, group):
    """float32 [N, K] weights of packed 4-bit integers."""
    b = q.to(torch.int32)
    v = torch.stack((b & 15, b >> 4), dim=2).flatten(1)
    v = v - 16 * (v >= 8).to(torch.int32)
    K = v.shape[1]
    s = scales.float().repeat_interleave(group, dim=1)[:, :K]
    v = v.float()
    if zeros is not None:
        v = v - zeros.float().repeat_interleave(group, dim=1)[:, :K]
    return v * s


def _plain(s):
    c = s["case"]
    t = _TYPES[c["dtype"]]
    if c["op"] == "gated":
        F = c["F"]
        z = s["x"].float() @ s["w"].float().t()
        g, u = z[:, :F], z[:, F:]
        h = (_act(c["act"], g) * u).to(t)
        return {"h": h, "gate": g.to(t), "up": u.to(t)} if c["save"] else {"h": h}
    if c["op"] == "gated_backward":
        g, u, dh = s["gate"].float(), s["up"].float(), s["dh"].float()
        d = torch.cat((dh * u * _slope(c["act"], g), dh * _act(c["act"], g)), dim=1)
        return {"dx": (d @ s["w"].float()).to(t), "dw": (d.t() @ s["x"].float()).to(t)}
    w = _dequantize(s["q"], s["scales"], s["zeros"], c["group"])
    y = s["x"].float() @ w.t()
    if c["op"] == "w4a16_gated":
        F = c["F"]
        return {"h": (_act(c["act"], y[:, :F]) * y[:, F:]).to(t)}
    if s["bias"] is not None:
        y = y + s["bias"]
    return {"y": y.to(t)}


def _library(s):
    import dense_gemm_preshuffle_amd as gp

    c = s["case"]
    if c["op"] == "gated":
        if c["save"]:
            h, gate, up = gp.gemm_gated(c["dtype"], s["x"], s["w_shuf"], act=c["act"], save=True, workspace=s["ws"])
            return {"h": h, "gate": gate, "up": up}
        return {"h": gp.gemm_gated(c["dtype"], s["x"], s["w_shuf"], act=c["act"], workspace=s["ws"])}
    if c["op"] == "gated_backward":
        # the weights change every step: they are taken as they are, row-major
        dx, dw = gp.gemm_gated_backward(c["dtype"], s["dh"], s["gate"], s["up"], s["x"], s["w"], act=c["act"],
                                        workspace=s["ws"])
        return {"dx": dx, "dw": dw}
    if c["op"] == "w4a16_gated":
        return {"h": gp.gemm_w4a16_gated(s["x"], s["weights"], act=c["act"])}
    return {"y": gp.gemm_w4a16(s["x"], s["weights"], bias=s["bias"])}


def run(state):
    return _library(state) if own else _plain(state)


def work(case):
    if case["op"] in ("gated", "gated_backward"):
        M, H, F = case["M"], case["H"], case["F"]
        if case["op"] == "gated":
            values = M * H + 2 * F * H + M * F * (3 if case["save"] else 1)
            return {"bytes": 2 * values, "flops": 4.0 * M * H * F}
        # dh, gate, up, x, w read; dx, dw written
        return {"bytes": 2 * (3 * M * F + 2 * M * H + 4 * F * H), "flops": 8.0 * M * H * F}
    gated = case["op"] == "w4a16_gated"
    M, K = case["M"], case["K"]
    N = 2 * case["F"] if gated else case["N"]
    groups = N * -(-K // case["group"])
    weights = N * K / 2 + groups * (3 if case["zeros"] else 2) + (4 * N if case.get("bias") else 0)
    return {"bytes": weights + 2 * M * K + 2 * M * (N // 2 if gated else N), "flops": 2.0 * M * N * K}


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


def _exact_weights(s, N, K, G):
    lo, hi = s["q"].bitwise_and(15).double(), s["q"].div(16, rounding_mode="floor").double()
    w = torch.empty(N, K, dtype=torch.float64, device=s["q"].device)
    w[:, 0::2] = torch.where(lo > 7.5, lo - 16, lo)
    w[:, 1::2] = torch.where(hi > 7.5, hi - 16, hi)
    at = torch.arange(K, device=w.device) // G
    if s["zeros"] is not None:
        w -= s["zeros"].double()[:, at]
    return w.mul_(s["scales"].double()[:, at])


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if case["op"] == "gated":
        F = case["F"]
        g = torch.mm(x, s["w"][:F].double().t())
        u = torch.mm(x, s["w"][F:].double().t())
        h = _exact_gate(case["act"], g)[0] * u
        return {"h": h, "gate": g, "up": u} if case["save"] else {"h": h}
    if case["op"] == "gated_backward":
        F = case["F"]
        value, slope = _exact_gate(case["act"], s["gate"].double())
        dh = s["dh"].double()
        du, dg = dh * value, dh * s["up"].double() * slope
        dx = torch.mm(dg, s["w"][:F].double()) + torch.mm(du, s["w"][F:].double())
        return {"dx": dx, "dw": torch.cat((torch.mm(dg.t(), x), torch.mm(du.t(), x)))}
    gated = case["op"] == "w4a16_gated"
    N = 2 * case["F"] if gated else case["N"]
    y = torch.mm(x, _exact_weights(s, N, case["K"], case["group"]).t())
    if gated:
        F = case["F"]
        return {"h": _exact_gate(case["act"], y[:, :F])[0] * y[:, F:]}
    return {"y": y if s["bias"] is None else y + s["bias"].double()}
