"""Measured cases of the operators that a mixture-of-experts block needs between its grouped products, in prefill and in
training: tokens sorted by expert and back, the norm before the block, the gated activation between its two products, and
the activations that are kept in 8 bits for the backward pass.

`run` computes a case with elementary torch operations in 32 bits, or, with `own` set, through the package's calls.

Definitions (e4m3 codes, one FP32 scale s for each 1x128 block, value = code * s):

  quantise   s = max(amax, 1e-4) / 448 over 128 values of a row, with pow2 the power of two above it (2^e for s = m 2^e,
             1/2 <= m < 1); code = e4m3(v / s), to nearest, ties to even; both quotients are rounded to FP32
  sort       rows[t, j] = where slot (t, j) goes: the rows of expert e = ids[t, j] are in the order of the slots, from
             row base[e] on. Contiguous layout: the bases are the sums of the counts before, each rounded up to 128;
             m_indices has the expert of every row, -1 where there is none. Masked layout: base[e] = e * max_m, slots past
             max_m have no row. An id outside [0, E) has no row: -1
  gather     A[rows[t, j]] = x[t] (e4m3 codes and scales, or BF16); contiguous layout: the rows between an expert's last and the
             end of its block of 128 are zeros (of scale 1e-4 / 448); all others stay as they were
  combine    out[t] = residual[t] + sum_j weights[t, j] * y[rows[t, j]]
  combine_backward  dy[rows[t, j]] = weights[t, j] * dout[t], zeros as in gather; dweights[t, j] = sum_h y[rows[t, j], h] * dout[t, h]
  norm       s = bf16(x + residual), y = s * rsqrt(mean(s^2) + eps) * g; given as BF16, or quantised
  norm_backward     with r = rsqrt(mean(s^2) + eps): dx = r * (g * dy - s * r^2 * mean(g * dy * s)) + dsum, dg = sum_t dy * s * r
  glu        h = act(g) * u for (g, u) = the halves of a row of Z, quantised; Z's own codes are kept for the backward pass on request. Rows
             without an expert's token (behind the last block, or past an expert's count) are not computed
  glu_backward      dg = dh * u * act'(g), du = dh * act(g), from BF16 (g, u) or from the kept codes: (dg, du) quantised along its rows
             and along its columns (the transpose, rows padded to 128 with zeros), and h quantised along its columns
  transpose  the values of codes with scales along the rows, quantised along the columns (as above)
"""
import math

import torch

own = False

DEV = "cuda"
FLOOR, TOP = 1e-4, 448.0
EPS = 1e-6
ACTS = ("silu", "silu", "gelu_tanh", "gelu", "relu")


def listed():
    return [
        # a decode step of a few sequences through the masked layout: latency counts
        {"name": "dispatch_decode", "op": "dispatch", "T": 5, "k": 2, "E": 8, "H": 1024, "half": False, "max_m": 16, "dropped": 0.0},
        # prefill of a long batch: FP8 tokens to 256 experts, the grouped product's padded segments
        {"name": "dispatch_prefill", "op": "dispatch", "T": 8189, "k": 8, "E": 256, "H": 7168, "half": False, "max_m": 0, "dropped": 0.0},
        # the way back, on one rank of an expert-parallel group: most of a token's experts live elsewhere
        {"name": "combine_local_experts", "op": "combine", "T": 4099, "k": 8, "E": 32, "H": 7168, "weighted": True, "residual": True, "dropped": 0.75},
        # training: the gradient of the weighted sum, to the experts' rows and to the router's weights
        {"name": "combine_gradient", "op": "combine_backward", "T": 4096, "k": 8, "E": 64, "H": 7168, "dropped": 0.0},
        # one decode step of one sequence, output for the block-scaled product
        {"name": "norm_one_token", "op": "norm", "T": 1, "H": 7168, "residual": True, "keep": True, "out": "fp8", "pow2": True, "half": True},
        # prefill: sum of the residual stream kept, FP8 rows for the dispatch, BF16 rows for the router
        {"name": "norm_prefill", "op": "norm", "T": 16381, "H": 7168, "residual": True, "keep": True, "out": "both", "pow2": False, "half": False},
        # its gradient in a training step, with what comes down the residual stream
        {"name": "norm_gradient", "op": "norm_backward", "T": 8192, "H": 7168, "dsum": True, "half": False},
        # a small model's decode step: one expert's few rows at a time
        {"name": "glu_decode", "op": "glu", "T": 24, "E": 8, "max_m": 16, "layout": "masked", "I": 384, "act": "silu", "keep": False, "pow2": False},
        # training forward in the padded segments, the pre-activations kept in 8 bits
        {"name": "glu_training", "op": "glu", "T": 32768, "E": 64, "max_m": 0, "layout": "contiguous", "I": 2048, "act": "silu", "keep": True, "pow2": False},
        # its backward pass from them
        {"name": "glu_gradient", "op": "glu_backward", "M": 16384, "I": 2048, "act": "silu", "kept": True},
        # the operand of a weight gradient from the codes that the forward product read: a ragged micro-batch
        {"name": "transpose_ragged", "op": "transpose", "M": 333, "N": 2048},
        # and a whole batch's tokens
        {"name": "transpose_training", "op": "transpose", "M": 32768, "N": 7168},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("dispatch", "dispatch", "combine", "combine_backward", "norm", "norm", "norm_backward", "glu", "glu", "glu_backward", "transpose"))
    if op in ("dispatch", "combine", "combine_backward"):
        E, H = _log(rng, 2, 256), 128 * _log(rng, 1, 56)
        k = rng.randint(1, min(E, 8))
        T = min(_log(rng, 1, 8192), int(2.2e8 / (k * H)))
        c = {"op": op, "T": T, "k": k, "E": E, "H": H, "dropped": rng.choice((0.0, 0.0, 0.5, 0.9)) if T * k > 100 else 0.0}
        if op == "dispatch":
            masked = rng.random() < 0.4
            return {**c, "half": rng.random() < 0.3, "max_m": max(1, min(2 * T * k // E + rng.randint(1, 40), 100000 // E)) if masked else 0}
        if op == "combine":
            return {**c, "weighted": rng.random() < 0.7, "residual": rng.random() < 0.5}
        return c
    if op in ("norm", "norm_backward"):
        T, half = _log(rng, 1, 16384), rng.random() < 0.5
        if op == "norm_backward":
            T = min(T, 8192)
            return {"op": op, "T": T, "H": 8 * _log(rng, 16, 896), "dsum": rng.random() < 0.7, "half": half}
        out = rng.choice(("bf16", "fp8", "both"))
        residual = rng.random() < 0.6
        return {"op": op, "T": T, "H": 8 * _log(rng, 16, 896) if out == "bf16" else 128 * _log(rng, 1, 56), "residual": residual, "keep": residual and rng.random() < 0.8,
                "out": out, "pow2": out != "bf16" and rng.random() < 0.4, "half": half}
    I = 128 * _log(rng, 1, 16)
    if op == "glu":
        layout = rng.choice(("dense", "contiguous", "masked"))
        T, E = _log(rng, 1, 32768), _log(rng, 1, 64) if layout != "dense" else 1
        return {"op": op, "T": T, "E": E, "max_m": 2 * T // E + rng.randint(1, 40) if layout == "masked" else 0, "layout": layout, "I": I, "act": rng.choice(ACTS),
                "keep": rng.random() < 0.5, "pow2": rng.random() < 0.3}
    if op == "glu_backward":
        return {"op": op, "M": _log(rng, 1, 16384), "I": I, "act": rng.choice(ACTS), "kept": rng.random() < 0.5}
    return {"op": op, "M": _log(rng, 1, 32768), "N": 128 * _log(rng, 1, 56)}


def _up(v):
    return (v + 127) // 128 * 128


def _rows_needed(T, k, E):
    """Rows that the contiguous layout of T * k slots never exceeds."""
    return (T * k + 127 * min(E, T * k)) // 128 * 128


def work(case):
    c = case
    if c["op"] in ("dispatch", "combine", "combine_backward"):
        T, k, H = c["T"], c["k"], c["H"]
        rows = T * k * (1.0 - c["dropped"])
        pads = 63.5 * min(c["E"], rows)
        if c["op"] == "dispatch":
            token = 2 * H if c["half"] else H + H / 32
            some = T * (1.0 - c["dropped"] ** k)                      # tokens with a row at all
            lists = 8 * T * k + 4 * c["E"] + (0 if c["max_m"] else 4 * _rows_needed(T, k, c["E"]))
            return {"bytes": lists + (some + rows + (0 if c["max_m"] else pads)) * token, "flops": 0}
        if c["op"] == "combine":
            return {"bytes": 2 * H * (rows + T * (2 if c["residual"] else 1)) + T * k * (8 if c["weighted"] else 4), "flops": 0}
        return {"bytes": 2 * H * (T + 2 * rows + pads) + 12 * T * k + 4 * _rows_needed(T, k, c["E"]), "flops": 0}
    if c["op"] == "norm":
        outs = {"bf16": 2, "fp8": 1 + 1 / 32, "both": 3 + 1 / 32}[c["out"]]
        return {"bytes": c["T"] * c["H"] * (2 + 2 * c["residual"] + 2 * c["keep"] + outs) + c["H"] * (2 if c["half"] else 4), "flops": 0}
    if c["op"] == "norm_backward":
        return {"bytes": c["T"] * c["H"] * (6 + 2 * c["dsum"]) + c["H"] * (6 if c["half"] else 8), "flops": 0}
    code = 1 + 1 / 32
    if c["op"] == "glu":
        rows = c["T"]
        if c["layout"] == "contiguous":
            rows += 63.5 * min(c["E"], c["T"])
        return {"bytes": rows * c["I"] * (4 + code + (2 * code if c["keep"] else 0)), "flops": 0}
    if c["op"] == "glu_backward":
        M, I = c["M"], c["I"]
        return {"bytes": M * I * (2 + (2 * code if c["kept"] else 4) + 2 * code) + _up(M) * I * 3 * code, "flops": 0}
    return {"bytes": (c["M"] + _up(c["M"])) * c["N"] * code, "flops": 0}


def _rng(seed, stream):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 1009 + stream)


def _normal(seed, stream, *shape):
    return torch.randn(*shape, generator=_rng(seed, stream), device=DEV)


def _codes(v):
    return v.clamp(-TOP, TOP).to(torch.float8_e4m3fn)


def _quantise(v, pow2=False):
    """1x128 blocks of the last axis: e4m3 codes, and scales."""
    b = v.unflatten(-1, (-1, 128))
    s = b.abs().amax(-1).clamp_min(FLOOR)
    s = s / torch.full_like(s, TOP)      # by a tensor: a division by a number would be a product with its reciprocal
    if pow2:
        s = torch.ldexp(torch.ones_like(s), torch.frexp(s).exponent)
    return _codes(b / s.unsqueeze(-1)).flatten(-2), s


def _quantise_columns(v):
    """The transpose of [M, N] in 1x128 blocks along M, padded to 128 with zeros."""
    return _quantise(torch.nn.functional.pad(v, (0, 0, 0, -v.shape[0] % 128)).t().contiguous())


def _values(q, s):
    """The values of 1x128-scaled codes."""
    return (q.float().unflatten(-1, (-1, 128)) * s.unsqueeze(-1)).flatten(-2)


def _ids(seed, T, k, E, dropped):
    """The experts of each token, some met more often than others; -1: the expert lives elsewhere."""
    liked = _normal(seed, 40, T, E) + 0.5 * _normal(seed, 41, E)
    ids = liked.topk(k, dim=1).indices
    lost = torch.rand(T, k, generator=_rng(seed, 42), device=DEV) < dropped
    return torch.where(lost, -1, ids).to(torch.int32)


def _sort(ids, E, Mt, max_m):
    """rows [T, k], counts [E], and m_indices [Mt] of the contiguous layout (max_m = 0)."""
    flat = ids.reshape(-1).long()
    open_ = (flat >= 0) & (flat < E)
    key = torch.where(open_, flat, E)
    order = torch.sort(key, stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.long, device=DEV).scatter_add_(0, key, torch.ones_like(key))
    at = torch.arange(key.numel(), device=DEV)
    rank = torch.empty_like(order).scatter_(0, order, at)              # a slot's place among all slots, by expert
    within = rank - (counts.cumsum(0) - counts)[key]
    if max_m:
        base = torch.arange(E + 1, device=DEV) * max_m
        open_ = open_ & (within < max_m)
    else:
        room = (counts + 127) // 128 * 128
        base = room.cumsum(0) - room
    rows = torch.where(open_, base[key] + within, -1)
    m_indices = None
    if not max_m:
        m_indices = torch.full((Mt + 1,), -1, device=DEV).scatter_(0, torch.where(open_, rows, Mt), torch.where(open_, key, -1))[:Mt].to(torch.int32)
    return rows.view(ids.shape).to(torch.int32), counts[:E].to(torch.int32), m_indices


def _pads(m_indices):
    """Rows without a token in blocks that have some."""
    b = m_indices.view(-1, 128)
    return ((b < 0) & (b[:, :1] >= 0)).view(-1)


def _scatter_rows(v, rows, like):
    """`like` zeroed, with row rows[t, j] = v[t, j] (v [T, k, ...]), where that is a row."""
    n = like.shape[0]
    out = torch.zeros(n + 1, *like.shape[1:], dtype=v.dtype, device=DEV)
    out[torch.where(rows >= 0, rows.long(), n).reshape(-1)] = v.reshape(-1, *v.shape[2:])
    return out[:n]


def prepare(case, seed):
    c, s = case, {"case": case}
    if c["op"] in ("dispatch", "combine", "combine_backward"):
        T, k, E, H = c["T"], c["k"], c["E"], c["H"]
        max_m = c.get("max_m", 0)
        Mt = E * max_m if max_m else _rows_needed(T, k, E)
        ids = _ids(seed, T, k, E, c["dropped"])
        x = _normal(seed, 1, T, H)
        if c["op"] == "dispatch":
            s["ids"] = ids
            if c["half"]:
                s["x"], s["sf"] = x.to(torch.bfloat16), None
            else:
                s["x"], s["sf"] = _quantise(x)
            s["rows"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
            s["counts"] = torch.empty(E, dtype=torch.int32, device=DEV)
            s["m_indices"] = None if max_m else torch.empty(Mt, dtype=torch.int32, device=DEV)
            s["A"] = torch.zeros(Mt, H, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) if not c["half"] else torch.zeros(Mt, H, dtype=torch.bfloat16, device=DEV)
            s["sfa"] = None if c["half"] else torch.zeros(Mt, H // 128, device=DEV)
        else:
            s["rows"], _, s["m_indices"] = _sort(ids, E, Mt, 0)
            s["y"] = _normal(seed, 2, Mt, H).to(torch.bfloat16)
            s["weights"] = torch.softmax(_normal(seed, 3, T, k), 1) if c.get("weighted", True) else None
            if c["op"] == "combine":
                s["residual"] = x.to(torch.bfloat16) if c["residual"] else None
                s["out"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
            else:
                s["dout"] = (x * 1e-2).to(torch.bfloat16)
                s["dy"] = torch.zeros(Mt, H, dtype=torch.bfloat16, device=DEV)
                s["dweights"] = torch.empty(T, k, device=DEV)
    elif c["op"] in ("norm", "norm_backward"):
        T, H = c["T"], c["H"]
        g = 1.0 + 0.2 * _normal(seed, 3, H)
        s["g"] = g.to(torch.bfloat16) if c["half"] else g
        s["x"] = (_normal(seed, 1, T, H) * 1.5).to(torch.bfloat16)
        if c["op"] == "norm":
            s["residual"] = (_normal(seed, 2, T, H) * 4.0).to(torch.bfloat16) if c["residual"] else None
            s["sum"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV) if c["keep"] else None
            s["y"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV) if c["out"] != "fp8" else None
            s["q"] = torch.empty(T, H, dtype=torch.float8_e4m3fn, device=DEV) if c["out"] != "bf16" else None
            s["sf"] = torch.empty(T, H // 128, device=DEV) if c["out"] != "bf16" else None
        else:
            s["dy"] = (_normal(seed, 2, T, H) * 1e-2).to(torch.bfloat16)
            s["dsum"] = (_normal(seed, 4, T, H) * 1e-2).to(torch.bfloat16) if c["dsum"] else None
            s["dx"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
            s["dg"] = torch.empty(H, device=DEV)
    elif c["op"] == "glu":
        T, E, I = c["T"], c["E"], c["I"]
        s["m_indices"] = s["masked_m"] = None
        if c["layout"] == "dense":
            M = T
        else:
            ids = torch.randint(0, E, (T, 1), generator=_rng(seed, 2), device=DEV).to(torch.int32)
            M = E * c["max_m"] if c["max_m"] else _rows_needed(T, 1, E)
            rows, counts, s["m_indices"] = _sort(ids, E, M, c["max_m"])
            s["masked_m"] = counts if c["max_m"] else None
        s["Z"] = _normal(seed, 1, M, 2 * I).to(torch.bfloat16)
        if s["m_indices"] is not None:
            s["Z"][_pads(s["m_indices"])] = 0.0                   # what the product of zero rows is
        s["q"] = torch.zeros(M, I, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
        s["sf"] = torch.zeros(M, I // 128, device=DEV)
        s["kept"] = torch.zeros(M, 2 * I, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) if c["keep"] else None
        s["kept_sf"] = torch.zeros(M, 2 * I // 128, device=DEV) if c["keep"] else None
    elif c["op"] == "glu_backward":
        M, I = c["M"], c["I"]
        Z = _normal(seed, 1, M, 2 * I).to(torch.bfloat16)
        s["Z"], s["kept"], s["kept_sf"] = (None, *_quantise(Z.float())) if c["kept"] else (Z, None, None)
        s["dH"] = (_normal(seed, 2, M, I) * 1e-2).to(torch.bfloat16)
        for name, n, m in (("q", M, 2 * I), ("qt", 2 * I, _up(M)), ("ht", I, _up(M))):
            s[name] = torch.empty(n, m, dtype=torch.float8_e4m3fn, device=DEV)
            s[name + "_sf"] = torch.empty(n, m // 128, device=DEV)
    else:
        M, N = c["M"], c["N"]
        # (rows of unlike size, as a batch's tokens are)
        s["q"], s["sf"] = _quantise(_normal(seed, 1, M, N) * torch.exp(0.5 * _normal(seed, 2, M, 1)))
        s["qt"] = torch.empty(N, _up(M), dtype=torch.float8_e4m3fn, device=DEV)
        s["sft"] = torch.empty(N, _up(M) // 128, device=DEV)
    if own and c["op"] in ("dispatch", "norm_backward"):
        # the workspaces that a program keeps beside its weights
        import moe_grouped_gemm_tma_gb300 as dg
        s["workspace"] = dg.moe_sort_workspace(c["T"], c["k"], c["E"]) if c["op"] == "dispatch" else dg.rmsnorm_backward_workspace(c["T"], c["H"])
    return s


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1.0 + torch.exp(-z))


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)
    p = 1.0 / (1.0 + torch.exp(-z))
    return p * (1.0 + z * (1.0 - p))


def _computed(s, M):
    """Rows of the gated activation that are computed; None: all."""
    if s["m_indices"] is not None:
        return (s["m_indices"].view(-1, 128)[:, :1] >= 0).expand(-1, 128).reshape(M, 1)
    if s["masked_m"] is not None:
        max_m = M // s["masked_m"].numel()
        return (torch.arange(max_m, device=DEV) < s["masked_m"][:, None]).view(M, 1)
    return None


def _only(q, sf, rows):
    """Zeros in the rows that are not computed."""
    if rows is None:
        return q, sf
    return torch.where(rows, q.view(torch.uint8), 0).view(torch.float8_e4m3fn), torch.where(rows, sf, 0.0)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "dispatch":
        Mt, k = s["A"].shape[0], c["k"]
        rows, counts, m_indices = _sort(s["ids"], c["E"], Mt, c["max_m"])
        out = {"rows": rows, "counts": counts, **({} if m_indices is None else {"m_indices": m_indices})}
        if c["half"]:
            return {**out, "A": _scatter_rows(s["x"].unsqueeze(1).expand(-1, k, -1), rows, s["A"])}
        A = _scatter_rows(s["x"].view(torch.uint8).unsqueeze(1).expand(-1, k, -1), rows, s["A"]).view(torch.float8_e4m3fn)
        sfa = _scatter_rows(s["sf"].unsqueeze(1).expand(-1, k, -1), rows, s["sfa"])
        if m_indices is not None:
            lowest = torch.full((1, 1), FLOOR, device=DEV) / torch.full((1, 1), TOP, device=DEV)
            sfa = torch.where(_pads(m_indices).unsqueeze(1), lowest, sfa)
        return {**out, "A": A, "sfa": sfa}
    if c["op"] in ("combine", "combine_backward"):
        open_ = (s["rows"] >= 0).unsqueeze(2)
        y = torch.where(open_, s["y"][s["rows"].clamp_min(0).long()].float(), 0.0)             # [T, k, H]
        if c["op"] == "combine":
            out = (y if s["weights"] is None else y * s["weights"].unsqueeze(2)).sum(1)
            return {"out": (out if s["residual"] is None else out + s["residual"].float()).to(torch.bfloat16)}
        dout = s["dout"].float().unsqueeze(1)
        dy = _scatter_rows((s["weights"].unsqueeze(2) * dout).to(torch.bfloat16), s["rows"], s["dy"])
        return {"dy": dy, "dweights": (y * dout).sum(2)}
    if c["op"] == "norm":
        t = s["x"].float()
        t = t if s["residual"] is None else (t + s["residual"].float()).to(torch.bfloat16).float()
        y = t * torch.rsqrt((t * t).mean(1, keepdim=True) + EPS) * s["g"].float()
        out = {"sum": t.to(torch.bfloat16)} if c["keep"] else {}
        if c["out"] != "fp8":
            out["y"] = y.to(torch.bfloat16)
        if c["out"] != "bf16":
            out["q"], out["sf"] = _quantise(y, c["pow2"])
        return out
    if c["op"] == "norm_backward":
        t, dy = s["x"].float(), s["dy"].float()
        r = torch.rsqrt((t * t).mean(1, keepdim=True) + EPS)
        gdy = dy * s["g"].float()
        dx = r * (gdy - t * (r * r * (gdy * t).mean(1, keepdim=True)))
        dx = dx if s["dsum"] is None else dx + s["dsum"].float()
        return {"dx": dx.to(torch.bfloat16), "dg": (dy * t * r).sum(0)}
    if c["op"] == "glu":
        M = s["Z"].shape[0]
        rows = _computed(s, M)
        Z = s["Z"].float()
        g, u = Z.chunk(2, 1)
        q, sf = _only(*_quantise(_act(g, c["act"]) * u, c["pow2"]), rows)
        if not c["keep"]:
            return {"q": q, "sf": sf}
        kept, kept_sf = _only(*_quantise(Z), rows)
        return {"q": q, "sf": sf, "kept": kept, "kept_sf": kept_sf}
    if c["op"] == "glu_backward":
        g, u = (s["Z"].float() if s["Z"] is not None else _values(s["kept"], s["kept_sf"])).chunk(2, 1)
        dh, a = s["dH"].float(), _act(g, c["act"])
        dz = torch.cat((dh * u * _act_slope(g, c["act"]), dh * a), 1)
        out = {"q": _quantise(dz), "qt": _quantise_columns(dz), "ht": _quantise_columns(a * u)}
        return {name + end: v for name, pair in out.items() for end, v in zip(("", "_sf"), pair)}
    qt, sft = _quantise_columns(_values(s["q"], s["sf"]))
    return {"qt": qt, "sft": sft}


def _run_own(s):
    import moe_grouped_gemm_tma_gb300 as dg
    c = s["case"]
    if c["op"] == "dispatch":
        if c["max_m"]:
            dg.dg_moe_sort_masked(s["ids"], s["rows"], s["counts"], c["max_m"], s["workspace"])
        else:
            dg.dg_moe_sort_contiguous(s["ids"], s["rows"], s["counts"], s["m_indices"], s["workspace"])
        dg.dg_moe_gather(s["x"], s["sf"], s["rows"], s["A"], s["sfa"], m_indices=s["m_indices"])
        return {n: s[n] for n in ("rows", "counts", "m_indices", "A", "sfa") if s[n] is not None}
    if c["op"] == "combine":
        dg.dg_moe_combine(s["y"], s["rows"], s["out"], weights=s["weights"], residual=s["residual"])
        return {"out": s["out"]}
    if c["op"] == "combine_backward":
        dg.dg_moe_combine_backward(s["dout"], s["rows"], s["dy"], weights=s["weights"], y=s["y"], dweights=s["dweights"], m_indices=s["m_indices"])
        return {"dy": s["dy"], "dweights": s["dweights"]}
    if c["op"] == "norm":
        dg.dg_rmsnorm(s["x"], s["g"], y=s["y"], q=s["q"], sf=s["sf"], residual=s["residual"], sum=s["sum"], eps=EPS, pow2=c["pow2"])
        return {n: s[n] for n in ("sum", "y", "q", "sf") if s[n] is not None}
    if c["op"] == "norm_backward":
        dg.dg_rmsnorm_backward(s["dy"], s["x"], s["g"], s["dx"], s["dg"], s["workspace"], dsum=s["dsum"], eps=EPS)
        return {"dx": s["dx"], "dg": s["dg"]}
    if c["op"] == "glu":
        dg.dg_glu(s["Z"], s["q"], s["sf"], kept=s["kept"], kept_sf=s["kept_sf"], m_indices=s["m_indices"], masked_m=s["masked_m"], act=c["act"], pow2=c["pow2"])
        return {n: s[n] for n in ("q", "sf", "kept", "kept_sf") if s[n] is not None}
    if c["op"] == "glu_backward":
        dg.dg_glu_backward(s["dH"], s["q"], s["q_sf"], s["qt"], s["qt_sf"], s["ht"], s["ht_sf"], Z=s["Z"], kept=s["kept"], kept_sf=s["kept_sf"], act=c["act"])
        return {n: s[n] for n in ("q", "q_sf", "qt", "qt_sf", "ht", "ht_sf")}
    dg.dg_transpose_fp8(s["q"], s["sf"], s["qt"], s["sft"])
    return {"qt": s["qt"], "sft": s["sft"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _round_e4m3(v):
    """The e4m3 value nearest to each 64-bit value, ties to even: 3 fraction bits, lowest exponent -6, largest value 448."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(-6) - 3)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def _exact_codes(v, pow2=False):
    b = v.reshape(*v.shape[:-1], -1, 128)
    s = (torch.clamp(b.abs().max(-1).values, min=FLOOR) / TOP).float().double()
    if pow2:
        s = 2.0 ** (torch.floor(torch.log2(s)) + 1)
    return _round_e4m3((b / s[..., None]).float().double()).reshape(v.shape), s


def _exact_columns(v):
    rows = torch.zeros(-v.shape[0] % 128, v.shape[1], dtype=torch.float64, device=DEV)
    return _exact_codes(torch.cat([v, rows]).T.contiguous())


def _exact_act(z, act):
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


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "dispatch":
        # slots in the order of their experts, one expert after the other
        Mt = s["A"].shape[0]
        A = torch.zeros(Mt, c["H"], dtype=torch.float64, device=DEV)
        sfa = None if c["half"] else torch.zeros(Mt, c["H"] // 128, dtype=torch.float64, device=DEV)
        first = 0
        for e in range(c["E"]):
            t = (s["ids"] == e).nonzero()[:, 0]
            if c["max_m"]:
                first, t = e * c["max_m"], t[:c["max_m"]]
            n = len(t)
            A[first:first + n] = s["x"][t].double()
            if sfa is not None:
                sfa[first:first + n] = s["sf"][t].double()
                if not c["max_m"]:
                    sfa[first + n:first + _up(n)] = FLOOR / TOP
            first += _up(n)
        return {"rows": None, "counts": None, **({} if c["max_m"] else {"m_indices": None}), "A": A, **({} if sfa is None else {"sfa": sfa})}
    if c["op"] == "combine":
        out = torch.zeros(c["T"], c["H"], dtype=torch.float64, device=DEV) if s["residual"] is None else s["residual"].double()
        for j in range(c["k"]):
            t = (s["rows"][:, j] >= 0).nonzero()[:, 0]
            w = 1.0 if s["weights"] is None else s["weights"][t, j, None].double()
            out[t] += w * s["y"][s["rows"][t, j].long()].double()
        return {"out": out}
    if c["op"] == "combine_backward":
        dy = torch.zeros(*s["dy"].shape, dtype=torch.float64, device=DEV)
        dw = torch.zeros(c["T"], c["k"], dtype=torch.float64, device=DEV)
        for j in range(c["k"]):
            t = (s["rows"][:, j] >= 0).nonzero()[:, 0]
            r, d = s["rows"][t, j].long(), s["dout"][t].double()
            dy[r] = s["weights"][t, j, None].double() * d
            dw[t, j] = torch.einsum("th,th->t", s["y"][r].double(), d)
        return {"dy": dy, "dweights": dw}
    if c["op"] in ("norm", "norm_backward"):
        t, g = s["x"].double(), s["g"].double()
        if c["op"] == "norm":
            if s["residual"] is not None:
                t = (t + s["residual"].double()).to(torch.bfloat16).double()
            y = t / torch.sqrt(t.square().mean(1, keepdim=True) + EPS) * g
            out = {"sum": t} if c["keep"] else {}
            if c["out"] != "fp8":
                out["y"] = y
            if c["out"] != "bf16":
                out["q"], out["sf"] = _exact_codes(y, c["pow2"])
            return out
        n = torch.sqrt(t.square().mean(1, keepdim=True) + EPS)
        h = t / n                                          # the normalised row; the gradient loses its share along it
        d = s["dy"].double()
        dx = (d * g - h * (d * g * h).mean(1, keepdim=True)) / n
        return {"dx": dx if s["dsum"] is None else dx + s["dsum"].double(), "dg": (d * h).sum(0)}
    if c["op"] == "glu":
        M, I = s["Z"].shape[0], c["I"]
        at = torch.ones(M, 1, dtype=torch.bool, device=DEV)
        if s["m_indices"] is not None:
            at = (s["m_indices"][::128] >= 0).repeat_interleave(128)[:, None]
        elif s["masked_m"] is not None:
            r = torch.arange(M, device=DEV)
            at = (r % c["max_m"] < s["masked_m"][r // c["max_m"]])[:, None]
        Z = s["Z"].double()
        pairs = {"q": _exact_codes(_exact_act(Z[:, :I], c["act"])[0] * Z[:, I:], c["pow2"])}
        names = {"q": ("q", "sf"), "kept": ("kept", "kept_sf")}
        if c["keep"]:
            pairs["kept"] = _exact_codes(Z)
        return {n: v * at for p, pair in pairs.items() for n, v in zip(names[p], pair)}
    if c["op"] == "glu_backward":
        I = c["I"]
        if s["Z"] is not None:
            Z = s["Z"].double()
        else:
            Z = (s["kept"].double().reshape(c["M"], -1, 128) * s["kept_sf"].double()[..., None]).reshape(c["M"], -1)
        a, slope = _exact_act(Z[:, :I], c["act"])
        d = s["dH"].double()
        dz = torch.empty_like(Z)
        dz[:, :I] = d * Z[:, I:] * slope
        dz[:, I:] = d * a
        out = {}
        out["q"], out["q_sf"] = _exact_codes(dz)
        out["qt"], out["qt_sf"] = _exact_columns(dz)
        out["ht"], out["ht_sf"] = _exact_columns(a * Z[:, I:])
        return out
    v = (s["q"].double().reshape(c["M"], -1, 128) * s["sf"].double()[..., None]).reshape(c["M"], -1)
    qt, sft = _exact_columns(v)
    return {"qt": qt, "sft": sft}
