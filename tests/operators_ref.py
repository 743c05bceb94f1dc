"""Plain 64-bit (CPU) forms of the operators around the products, written from their definitions."""
import math

import numpy as np
import torch

TOP, FLOOR = 448.0, 1e-4


def e4m3_nearest(v):
    """The e4m3 value nearest to each float64, ties to even, saturating; NaN stays."""
    v = np.asarray(v, dtype=np.float64)
    _, e = np.frexp(np.where(np.isfinite(v), v, 1.0))
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    with np.errstate(invalid="ignore"):
        return np.clip(np.rint(v / step) * step, -TOP, TOP)


def quantise(v):
    """1x128 blocks of the last axis -> (codes as values, scales); the quotients are rounded to FP32, the scale
    floor is the FP32 number nearest to 1e-4."""
    v = np.asarray(v, dtype=np.float64)
    b = v.reshape(*v.shape[:-1], -1, 128)
    amax = np.abs(b).max(-1)
    with np.errstate(invalid="ignore", divide="ignore"):
        s = np.float32(np.where(amax < np.float32(FLOOR), np.float32(FLOOR), amax) / TOP).astype(np.float64)
        q = np.float32(b / s[..., None]).astype(np.float64)
    return e4m3_nearest(q).reshape(v.shape), s


def values(q, s):
    return (q.reshape(*s.shape, 128) * s[..., None]).reshape(q.shape)


def block_values(codes, s):
    """float64 values of 128x128-scaled codes [N, K] (uint8 torch tensor) with scales [ceil(N/128), K/128]."""
    q = codes.view(torch.float8_e4m3fn).double().numpy()
    n, k = q.shape
    return q * s.double().numpy()[np.arange(n) // 128][:, np.arange(k) // 128]


def row_values(codes, s):
    q = codes.view(torch.float8_e4m3fn).double().numpy()
    return values(q, s.double().numpy())


_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(z, name):
    with np.errstate(over="ignore"):
        if name == "relu":
            return np.where(z < 0, 0.0, z)
        if name == "gelu":
            return 0.5 * z * (1 + _erf(z / math.sqrt(2)))
        if name == "gelu_tanh":
            return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
        if name == "silu":
            return z / (1 + np.exp(-z))
    return z


def act_slope(z, name):
    with np.errstate(over="ignore"):
        if name == "relu":
            return (z > 0).astype(np.float64)
        if name == "gelu":
            return 0.5 * (1 + _erf(z / math.sqrt(2))) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        if name == "gelu_tanh":
            a = math.sqrt(2 / math.pi)
            t = np.tanh(a * (z + 0.044715 * z ** 3))
            return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)
        if name == "silu":
            p = 1 / (1 + np.exp(-z))
            return p * (1 + z * (1 - p))
    return np.ones_like(z)


def route(logits, k, scoring, renorm, scale, bias=None):
    """(ids, weights) of float64 logits [T, E]; selection values are compared as FP32 numbers (with a bias
    they are FP32 sums of an FP32 sigmoid)."""
    T, E = logits.shape
    ids = np.full((T, k), -1, dtype=np.int64)
    w = np.zeros((T, k))
    top_finite = float(np.finfo(np.float32).max)
    for t in range(T):
        l = np.minimum(logits[t], top_finite)
        ok = ~np.isnan(l) & (l > -np.inf)
        pick = l.astype(np.float64)
        with np.errstate(over="ignore"):
            sig = 1 / (1 + np.exp(-np.where(ok, l, 0.0)))
        if bias is not None:
            pick = (sig.astype(np.float32) + bias[:E].astype(np.float32)).astype(np.float64)
            ok = ok & ~np.isnan(pick) & (pick > -np.inf)
        order = sorted((e for e in range(E) if ok[e]), key=lambda e: (-pick[e], e))[:k]
        if not order:
            continue
        if scoring == "softmax":
            ex = np.where(ok, np.exp(np.where(ok, l, 0.0) - l[ok].max()), 0.0)
            score = ex / ex.sum()
        else:
            score = sig
        got = score[order]
        if renorm:
            total = got.sum()
            got = got / total if total > 0 else np.zeros_like(got)
        ids[t, :len(order)] = order
        w[t, :len(order)] = got * scale
    return ids, w


def route_weights(logits, ids, scoring, renorm, scale):
    """The weights of given ids, for differences."""
    T, E = logits.shape
    w = np.zeros(ids.shape)
    for t in range(T):
        l = logits[t]
        ok = l > -np.inf
        if scoring == "softmax":
            ex = np.where(ok, np.exp(np.where(ok, l, 0.0) - l[ok].max()), 0.0)
            score = ex / ex.sum()
        else:
            score = np.where(ok, 1 / (1 + np.exp(-np.where(ok, l, 0.0))), 0.0)
        sel = [(j, e) for j, e in enumerate(ids[t]) if 0 <= e < E]
        total = sum(score[e] for _, e in sel) if renorm else 1.0
        for j, e in sel:
            w[t, j] = scale * score[e] / total if total > 0 else 0.0
    return w


def route_backward(logits, ids, dw, scoring, renorm, scale):
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        l = np.minimum(logits[t], float(np.finfo(np.float32).max))        # as the forward pass takes +inf
        ok = l > -np.inf
        if not ok.any():
            continue
        if scoring == "softmax":
            ex = np.where(ok, np.exp(np.where(ok, l, 0.0) - l[ok].max()), 0.0)
            p = ex / ex.sum()
        else:
            p = np.where(ok, 1 / (1 + np.exp(-np.where(ok, l, 0.0))), 0.0)
        sel = [(j, e) for j, e in enumerate(ids[t]) if 0 <= e < E]
        dp = np.zeros(E)
        total = sum(p[e] for _, e in sel)
        dot = sum(dw[t, j] * p[e] for j, e in sel)
        for j, e in sel:
            dp[e] += scale * (dw[t, j] / total - dot / total ** 2 if renorm else dw[t, j])
        out[t] = p * (dp - (dp * p).sum()) if scoring == "softmax" else dp * p * (1 - p)
    return out


def moe(x, ids, weights, W13, s13, W2, s2, name, residual=None):
    """float64 output of the layer: x [T, H] float64, ids, weights, codes and scales as torch CPU tensors."""
    T, H = x.shape
    E, I2, _ = W13.shape
    I = I2 // 2
    xv = values(*quantise(x))
    out = np.zeros((T, H)) if residual is None else residual.astype(np.float64).copy()
    for e in range(E):
        rows = [(t, j) for t in range(T) for j in range(ids.shape[1]) if ids[t, j] == e]
        if not rows:
            continue
        w13, w2 = block_values(W13[e], s13[e]), block_values(W2[e], s2[e])
        xs = xv[[t for t, _ in rows]]
        gu = xs @ w13.T
        h = act(gu[:, :I], name) * gu[:, I:]
        y = values(*quantise(h)) @ w2.T
        for (t, j), v in zip(rows, y):
            out[t] += float(weights[t, j]) * v
    return out
