"""Measured cases of the operators around the experts' products: the router, a whole mixture-of-experts layer for a
few tokens, and the FP8 product with bias, activation and residual in its epilogue, forward and backward.

`run` computes a case with elementary torch operations in 32 bits, or, with `own` set, through the package's calls.

Definitions (sums over a 128-wide scaling block; e4m3 codes; s = FP32 block scale; value = code * s):

  quantise   s = max(amax, 1e-4) / 448 over 1x128 values, code = e4m3(v / s), to nearest, ties to even; both quotients are
             rounded to FP32 (BF16 inputs often meet the ties exactly, so the rounding belongs to the definition)
  route      ids = the k largest selection values of a row, ties to the lowest index (selection value: the logit, or,
             with a bias, sigmoid(logit) + bias); weight = scale * softmax or sigmoid score, renormalised over the k
             if asked; a logit of -inf cannot be selected, and a slot without an expert gets id -1 and weight 0
  moe        out[t] = residual[t] + sum_j weights[t, j] * W2[e] . Q(act(g) * u), (g; u) = W13[e] . Q(x[t]), e = ids[t, j];
             an id outside [0, E) adds nothing
  gemm       Z = A . B^T + bias, D = act(Z) + residual
  backward   dZ = dD * act'(Z), given as codes along its rows (for dX = dZ . B), as codes along its columns (the transpose,
             tokens padded to 128 with zeros, for dB = dZ^T . A), and dbias = the sum of dZ's rows
"""
import math

import torch

own = False

DEV = "cuda"
FLOOR, TOP = 1e-4, 448.0
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def listed():
    return [
        # one decode step of one sequence: a row of router logits
        {"name": "route_one_token", "op": "route", "T": 1, "E": 64, "k": 6, "scoring": "softmax", "bias": False, "renorm": True, "half": False, "masked": 0.0},
        # prefill of a long batch: sigmoid scores with a balancing bias, BF16 logits, a few experts switched off
        {"name": "route_prefill", "op": "route", "T": 32749, "E": 256, "k": 8, "scoring": "sigmoid", "bias": True, "renorm": True, "half": True, "masked": 0.02},
        # training step: the weights' gradient back to every logit (softmax without renormalisation is dense)
        {"name": "route_gradient", "op": "route_backward", "T": 16384, "E": 128, "k": 8, "scoring": "softmax", "bias": False, "renorm": False, "half": False, "masked": 0.0},
        # one decode step of one sequence through the workload's expert shapes (4096 x 7168 and 7168 x 2048)
        {"name": "moe_one_token", "op": "moe", "T": 1, "k": 8, "E": 16, "H": 7168, "I": 2048, "act": "silu", "residual": True, "dropped": 0.0},
        # a small model's layer: few, narrow experts, where the call's latency counts
        {"name": "moe_small_layer", "op": "moe", "T": 5, "k": 2, "E": 8, "H": 1024, "I": 384, "act": "silu", "residual": False, "dropped": 0.0},
        # one rank of an expert-parallel group: most of a token's experts live elsewhere (id -1)
        {"name": "moe_local_experts", "op": "moe", "T": 33, "k": 8, "E": 16, "H": 7168, "I": 2048, "act": "silu", "residual": False, "dropped": 0.75},
        # a full decode batch: every expert is met by many tokens
        {"name": "moe_64_tokens", "op": "moe", "T": 64, "k": 8, "E": 16, "H": 7168, "I": 2048, "act": "gelu_tanh", "residual": True, "dropped": 0.0},
        # the dense (shared) layer of one decode step
        {"name": "gemm_one_token", "op": "gemm", "M": 1, "N": 4096, "K": 7168, "act": "gelu", "bias": True, "residual": False, "keep": False},
        # ragged rows, the workload's odd width
        {"name": "gemm_ragged", "op": "gemm", "M": 333, "N": 2112, "K": 7168, "act": "relu", "bias": True, "residual": True, "keep": False},
        # training forward: the pre-activation is kept for the backward pass
        {"name": "gemm_training", "op": "gemm", "M": 4096, "N": 7168, "K": 2048, "act": "silu", "bias": True, "residual": True, "keep": True},
        # its backward pass
        {"name": "backward_training", "op": "backward", "M": 4096, "N": 7168, "act": "silu"},
        # a ragged micro-batch
        {"name": "backward_ragged", "op": "backward", "M": 333, "N": 2048, "act": "gelu_tanh"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "route_backward", "moe", "moe", "gemm", "gemm", "backward"))
    if op in ("route", "route_backward"):
        E = rng.choice((rng.randint(2, 31), rng.randint(32, 512)))
        sig = rng.random() < 0.5
        return {"op": op, "T": _log(rng, 1, 32768), "E": E, "k": rng.randint(1, min(E, 10)), "scoring": "sigmoid" if sig else "softmax",
                "bias": sig and rng.random() < 0.6, "renorm": rng.random() < 0.6, "half": rng.random() < 0.5, "masked": rng.choice((0.0, 0.3))}
    if op == "moe":
        E = _log(rng, 2, 16)
        return {"op": op, "T": _log(rng, 1, 64), "k": rng.randint(1, min(E, 8)), "E": E, "H": 128 * rng.randint(4, 56), "I": 128 * rng.randint(1, 16),
                "act": rng.choice(("silu", "silu", "gelu_tanh", "gelu", "relu")), "residual": rng.random() < 0.5, "dropped": rng.choice((0.0, 0.5, 0.9))}
    if op == "gemm":
        M, N, K = _log(rng, 1, 4096), 8 * _log(rng, 8, 1024), 128 * _log(rng, 1, 64)
        M = max(1, min(M, int(6.0e10 / (N * K))))
        return {"op": op, "M": M, "N": N, "K": K, "act": rng.choice(ACTS), "bias": rng.random() < 0.7, "residual": rng.random() < 0.6, "keep": rng.random() < 0.4}
    return {"op": op, "M": _log(rng, 1, 4096), "N": 128 * _log(rng, 1, 56), "act": rng.choice(ACTS)}


def work(case):
    c = case
    if c["op"] == "route":
        return {"bytes": c["T"] * (c["E"] * (2 if c["half"] else 4) + 8 * c["k"]) + (4 * c["E"] if c["bias"] else 0), "flops": 0}
    if c["op"] == "route_backward":
        # without renormalised weights of a softmax only the selected logits are needed
        dense = c["scoring"] == "softmax" and not c["renorm"]
        size = 2 if c["half"] else 4
        return {"bytes": c["T"] * (c["E"] * size * (2 if dense else 1) + c["k"] * (8 if dense else 8 + size)), "flops": 0}
    if c["op"] == "moe":
        kept = c["k"] * (1.0 - c["dropped"])
        met = c["E"] * (1.0 - (1.0 - kept / c["E"]) ** c["T"])   # experts that at least one token meets, on average
        weights = 3 * c["H"] * c["I"] * (1.0 + 4.0 / 128 ** 2)
        return {"bytes": met * weights + c["T"] * (c["H"] * (6 if c["residual"] else 4) + 8 * c["k"]), "flops": 6.0 * c["T"] * kept * c["H"] * c["I"]}
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        outs = 1 + int(c["residual"]) + int(c["keep"])
        return {"bytes": (M + N) * K + M * K / 32 + N * K / 4096 + 2 * M * N * outs + (4 * N if c["bias"] else 0), "flops": 2.0 * M * N * K}
    M, N = c["M"], c["N"]
    Mp = (M + 127) // 128 * 128
    return {"bytes": M * N * (2 if c["act"] == "none" else 4) + (M + Mp) * N * (1 + 1 / 32) + 4 * N, "flops": 0}


def _rng(seed, stream):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 1009 + stream)


def _normal(seed, stream, *shape):
    return torch.randn(*shape, generator=_rng(seed, stream), device=DEV)


def _codes(v):
    return v.clamp(-TOP, TOP).to(torch.float8_e4m3fn)


def _quantise(v):
    """1x128 blocks of the last axis: e4m3 codes as values, and scales."""
    b = v.unflatten(-1, (-1, 128))
    s = b.abs().amax(-1).clamp_min(FLOOR)
    s = s / torch.full_like(s, TOP)      # by a tensor: a division by a number would be a product with its reciprocal
    return _codes(b / s.unsqueeze(-1)).flatten(-2), s


def _quantise_blocks(v):
    """128x128 blocks of [N, K] (the last row block may be short)."""
    N, K = v.shape
    p = torch.nn.functional.pad(v, (0, 0, 0, -N % 128)).view(-1, 128, K // 128, 128)
    s = p.abs().amax((1, 3)).clamp_min(FLOOR)
    s = s / torch.full_like(s, TOP)
    return _codes(p / s[:, None, :, None]).view(-1, K)[:N].contiguous(), s


def prepare(case, seed):
    c, s = case, {"case": case}
    if c["op"] in ("route", "route_backward"):
        logits = _normal(seed, 1, c["T"], c["E"]) * 2.0
        if c["masked"]:
            off = torch.rand(c["E"], generator=_rng(seed, 2), device=DEV) < c["masked"]
            logits[:, off] = -math.inf
        s["logits"] = logits.to(torch.bfloat16) if c["half"] else logits
        s["bias"] = _normal(seed, 3, c["E"]) * 0.05 if c["bias"] else None
        s["scale"] = 2.5 if c["scoring"] == "sigmoid" else 1.0
        if c["op"] == "route":
            s["ids"] = torch.empty(c["T"], c["k"], dtype=torch.int32, device=DEV)
            s["weights"] = torch.empty(c["T"], c["k"], device=DEV)
        else:
            s["ids"] = _route(c, s["logits"], s["bias"], s["scale"])[0]
            s["dweights"] = _normal(seed, 4, c["T"], c["k"]) * 0.01
            s["dlogits"] = torch.empty_like(s["logits"])
    elif c["op"] == "moe":
        T, k, E, H, I = c["T"], c["k"], c["E"], c["H"], c["I"]
        s["x"] = _normal(seed, 1, T, H).to(torch.bfloat16)
        logits = _normal(seed, 2, T, E)
        top, ids = logits.topk(k, dim=1)
        lost = torch.rand(T, k, generator=_rng(seed, 3), device=DEV) < c["dropped"]
        s["ids"] = torch.where(lost, -1, ids).to(torch.int32)
        s["weights"] = torch.softmax(top, 1)
        s["residual"] = _normal(seed, 4, T, H).to(torch.bfloat16) if c["residual"] else None
        w13 = [_quantise_blocks(_normal(seed, 10 + 2 * e, 2 * I, H) / math.sqrt(H)) for e in range(E)]
        s["W13"], s["s13"] = torch.stack([w for w, _ in w13]), torch.stack([q for _, q in w13])
        del w13
        w2 = [_quantise_blocks(_normal(seed, 11 + 2 * e, H, I) / math.sqrt(I)) for e in range(E)]
        s["W2"], s["s2"] = torch.stack([w for w, _ in w2]), torch.stack([q for _, q in w2])
        s["out"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        s["A"], s["sfa"] = _quantise(_normal(seed, 1, M, K))
        s["B"], s["sfb"] = _quantise_blocks(_normal(seed, 2, N, K) / math.sqrt(K))
        s["bias"] = _normal(seed, 3, N) * 0.5 if c["bias"] else None
        s["residual"] = _normal(seed, 4, M, N).to(torch.bfloat16) if c["residual"] else None
        s["D"] = torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
        s["Z"] = torch.empty_like(s["D"]) if c["keep"] else None
    else:
        M, N = c["M"], c["N"]
        Mp = (M + 127) // 128 * 128
        s["dD"] = (_normal(seed, 1, M, N) * 1e-2).to(torch.bfloat16)
        s["Z"] = _normal(seed, 2, M, N).to(torch.bfloat16) if c["act"] != "none" else None
        s["q"] = torch.empty(M, N, dtype=torch.float8_e4m3fn, device=DEV)
        s["sf"] = torch.empty(M, N // 128, device=DEV)
        s["qt"] = torch.empty(N, Mp, dtype=torch.float8_e4m3fn, device=DEV)
        s["sft"] = torch.empty(N, Mp // 128, device=DEV)
        s["dbias"] = torch.empty(N, device=DEV)
    if own:
        # the workspaces that a program keeps beside its weights
        import moe_grouped_gemm_tma_gb300 as dg
        if c["op"] == "moe":
            s["workspace"] = dg.moe_layer_workspace(c["T"], c["k"], c["E"], c["H"], c["I"])
        elif c["op"] == "backward":
            s["workspace"] = dg.epilogue_backward_workspace(c["M"], c["N"])
    return s


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return torch.ones_like(z)


def _route(c, logits, bias, scale):
    l = logits.float()
    score = 1.0 / (1.0 + torch.exp(-l))
    pick = l if bias is None else torch.where(l == -math.inf, l, score + bias)
    top, at = torch.sort(pick, dim=1, descending=True, stable=True)
    top, at = top[:, :c["k"]], at[:, :c["k"]]
    open_ = top != -math.inf
    if c["scoring"] == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True).clamp_min(torch.finfo(torch.float32).min))
        score = e / e.sum(1, keepdim=True).clamp_min(torch.finfo(torch.float32).tiny)
    w = torch.where(open_, score.gather(1, at), 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return torch.where(open_, at, -1).to(torch.int32), w * scale


def _route_backward(c, logits, ids, dw, scale):
    l = logits.float()
    at, open_ = ids.clamp_min(0).long(), ids >= 0
    dw = torch.where(open_, dw * scale, 0.0)
    if c["scoring"] == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True).clamp_min(torch.finfo(torch.float32).min))
        p = e / e.sum(1, keepdim=True).clamp_min(torch.finfo(torch.float32).tiny)
        w = torch.where(open_, p.gather(1, at), 0.0)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp_min(torch.finfo(torch.float32).tiny)
            grad = w * (dw - (w * dw).sum(1, keepdim=True))
            return torch.zeros_like(l).scatter_add_(1, at, torch.where(open_, grad, 0.0)).to(logits.dtype)
        grad = torch.zeros_like(l).scatter_add_(1, at, w * dw) - p * (w * dw).sum(1, keepdim=True)
        return grad.to(logits.dtype)
    p = torch.where(open_, 1.0 / (1.0 + torch.exp(-l.gather(1, at))), 0.0)
    if c["renorm"]:
        r = p / p.sum(1, keepdim=True).clamp_min(torch.finfo(torch.float32).tiny)
        grad = (1.0 - p) * r * (dw - (r * dw).sum(1, keepdim=True))
    else:
        grad = dw * p * (1.0 - p)
    return torch.zeros_like(l).scatter_add_(1, at, torch.where(open_, grad, 0.0)).to(logits.dtype)


def _values(q, s):
    """The values of 1x128-scaled codes."""
    return (q.float().unflatten(-1, (-1, 128)) * s.unsqueeze(-1)).flatten(-2)


def _block_values(q, s):
    """The values of 128x128-scaled codes [..., N, K]."""
    rows = s.repeat_interleave(128, -2)[..., :q.shape[-2], :]
    return (q.float().unflatten(-1, (-1, 128)) * rows.unsqueeze(-1)).flatten(-2)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "route":
        ids, weights = _route(c, s["logits"], s["bias"], s["scale"])
        return {"ids": ids, "weights": weights}
    if c["op"] == "route_backward":
        return {"dlogits": _route_backward(c, s["logits"], s["ids"], s["dweights"], s["scale"])}
    if c["op"] == "moe":
        x = _values(*_quantise(s["x"].float()))
        g, u = torch.matmul(x, _block_values(s["W13"], s["s13"]).transpose(1, 2)).chunk(2, -1)   # [E, T, I]
        h = _values(*_quantise(_act(g, c["act"]) * u))
        y = torch.matmul(h, _block_values(s["W2"], s["s2"]).transpose(1, 2))                     # [E, T, H]
        met = s["ids"].unsqueeze(2) == torch.arange(c["E"], device=DEV)
        share = torch.where(met, s["weights"].unsqueeze(2), 0.0).sum(1)                          # [T, E]
        out = (share.t().unsqueeze(2) * y).sum(0)
        return {"out": (out if s["residual"] is None else out + s["residual"].float()).to(torch.bfloat16)}
    if c["op"] == "gemm":
        z = torch.matmul(_values(s["A"], s["sfa"]), _block_values(s["B"], s["sfb"]).t())
        z = z if s["bias"] is None else z + s["bias"]
        d = _act(z, c["act"])
        d = d if s["residual"] is None else d + s["residual"].float()
        return {"D": d.to(torch.bfloat16), **({"Z": z.to(torch.bfloat16)} if c["keep"] else {})}
    dz = s["dD"].float()
    dz = dz if s["Z"] is None else dz * _act_slope(s["Z"].float(), c["act"])
    q, sf = _quantise(dz)
    qt, sft = _quantise(torch.nn.functional.pad(dz, (0, 0, 0, -c["M"] % 128)).t().contiguous())
    return {"q": q, "sf": sf, "qt": qt, "sft": sft, "dbias": dz.sum(0)}


def _run_own(s):
    import moe_grouped_gemm_tma_gb300 as dg
    c = s["case"]
    if c["op"] == "route":
        dg.dg_moe_route(s["logits"], s["ids"], s["weights"], bias=s["bias"], scoring=c["scoring"], renormalize=c["renorm"], scale=s["scale"])
        return {"ids": s["ids"], "weights": s["weights"]}
    if c["op"] == "route_backward":
        dg.dg_moe_route_backward(s["logits"], s["ids"], s["dweights"], s["dlogits"], scoring=c["scoring"], renormalize=c["renorm"], scale=s["scale"])
        return {"dlogits": s["dlogits"]}
    if c["op"] == "moe":
        dg.dg_moe_layer(s["x"], s["ids"], s["weights"], s["W13"], s["s13"], s["W2"], s["s2"], s["out"], s["workspace"], act=c["act"], residual=s["residual"])
        return {"out": s["out"]}
    if c["op"] == "gemm":
        dg.dg_gemm_fp8_nt_epilogue(s["A"], s["sfa"], s["B"], s["sfb"], s["D"], bias=s["bias"], act=c["act"], residual=s["residual"], Z=s["Z"])
        return {"D": s["D"], **({"Z": s["Z"]} if c["keep"] else {})}
    dg.dg_epilogue_backward(s["dD"], s["Z"], s["q"], s["sf"], s["qt"], s["sft"], s["dbias"], s["workspace"], act=c["act"])
    return {"q": s["q"], "sf": s["sf"], "qt": s["qt"], "sft": s["sft"], "dbias": s["dbias"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _round_e4m3(v):
    """The e4m3 value nearest to each 64-bit value, ties to even: 3 fraction bits, lowest exponent -6, largest value 448."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(-6) - 3)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def _exact_codes(v):
    b = v.reshape(*v.shape[:-1], -1, 128)
    s = (torch.clamp(b.abs().max(-1).values, min=FLOOR) / TOP).float().double()
    return _round_e4m3((b / s[..., None]).float().double()).reshape(v.shape), s


def _exact_act(z, act):
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp_min(0), (z > 0).double()
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    a, b = math.sqrt(2 / math.pi), 0.044715
    p = torch.sigmoid(2 * a * (z + b * z ** 3))        # (1 + tanh(y)) / 2 = sigmoid(2 y)
    return z * p, p + 2 * a * z * p * (1 - p) * (1 + 3 * b * z ** 2)


def _exact_weight(q, s):
    n, k = q.shape
    grid = s.double()[torch.arange(n, device=DEV) // 128][:, torch.arange(k, device=DEV) // 128]
    return q.double() * grid


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] in ("route", "route_backward"):
        l = s["logits"].double()
        ids = _route(c, s["logits"], s["bias"], s["scale"])[0].long() if c["op"] == "route" else s["ids"].long()
        open_ = (ids >= 0).double()
        if c["scoring"] == "softmax":
            score = torch.nan_to_num(torch.softmax(l, 1), nan=0.0)
        else:
            score = torch.sigmoid(l)
        p = torch.gather(score, 1, ids.clamp_min(0)) * open_
        total = p.sum(1, keepdim=True)
        if c["op"] == "route":
            w = torch.nan_to_num(p / total, nan=0.0) if c["renorm"] else p
            return {"ids": None, "weights": w * s["scale"]}
        dw = s["dweights"].double() * s["scale"] * open_
        # the gradient with respect to the selected scores, then through the score
        dp = torch.nan_to_num(dw / total - (dw * p).sum(1, keepdim=True) / total ** 2, nan=0.0) * open_ if c["renorm"] else dw
        dscore = torch.zeros_like(l).scatter_add_(1, ids.clamp_min(0), dp)
        if c["scoring"] == "softmax":
            return {"dlogits": score * (dscore - (dscore * score).sum(1, keepdim=True))}
        return {"dlogits": dscore * score * (1 - score)}
    if c["op"] == "moe":
        q, sx = _exact_codes(s["x"].double())
        x = (q.reshape(c["T"], -1, 128) * sx[..., None]).reshape(c["T"], -1)
        out = torch.zeros(c["T"], c["H"], dtype=torch.float64, device=DEV) if s["residual"] is None else s["residual"].double()
        for e in range(c["E"]):
            t, j = (s["ids"] == e).nonzero(as_tuple=True)
            if not len(t):
                continue
            gu = x[t] @ _exact_weight(s["W13"][e], s["s13"][e]).T
            h = _exact_act(gu[:, :c["I"]], c["act"])[0] * gu[:, c["I"]:]
            q, sh = _exact_codes(h)
            h = (q.reshape(len(t), -1, 128) * sh[..., None]).reshape(len(t), -1)
            out.index_add_(0, t, s["weights"][t, j].double()[:, None] * (h @ _exact_weight(s["W2"][e], s["s2"][e]).T))
        return {"out": out}
    if c["op"] == "gemm":
        a = (s["A"].double().reshape(c["M"], -1, 128) * s["sfa"].double()[..., None]).reshape(c["M"], -1)
        z = a @ _exact_weight(s["B"], s["sfb"]).T
        if s["bias"] is not None:
            z += s["bias"].double()
        d = _exact_act(z, c["act"])[0]
        if s["residual"] is not None:
            d = d + s["residual"].double()
        return {"D": d, **({"Z": z} if c["keep"] else {})}
    dz = s["dD"].double()
    if s["Z"] is not None:
        dz = dz * _exact_act(s["Z"].double(), c["act"])[1]
    q, sf = _exact_codes(dz)
    rows = torch.zeros(-c["M"] % 128, c["N"], dtype=torch.float64, device=DEV)
    qt, sft = _exact_codes(torch.cat([dz, rows]).T.contiguous())
    return {"q": q, "sf": sf, "qt": qt, "sft": sft, "dbias": dz.sum(0)}
