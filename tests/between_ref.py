"""Plain forms of the operators between the grouped products, from their definitions, in 64 bits (torch, on any device), and
the checks of quantised outputs that the tests share."""
import math

import torch

TOP, FLOOR = 448.0, 1e-4


def up(v):
    return (v + 127) // 128 * 128


def sort(ids, E, Mt=0, max_m=0):
    """rows [T][k], counts [E] and m_indices [Mt] as lists: slot by slot."""
    counts = [0] * E
    for row in ids:
        for e in row:
            if 0 <= e < E:
                counts[e] += 1
    base, at = [], 0
    for e in range(E):
        base.append(e * max_m if max_m else at)
        at += up(counts[e])
    seen, rows = [0] * E, []
    for row in ids:
        out = []
        for e in row:
            r = -1
            if 0 <= e < E:
                if not max_m or seen[e] < max_m:
                    r = base[e] + seen[e]
                seen[e] += 1
            out.append(r)
        rows.append(out)
    m_indices = [-1] * Mt
    for e in range(E):
        for i in range(counts[e] if not max_m else 0):
            m_indices[base[e] + i] = e
    return rows, counts, m_indices


def pads(m_indices):
    b = m_indices.view(-1, 128)
    return ((b < 0) & (b[:, :1] >= 0)).view(-1)


def combine(y, rows, weights, residual):
    """(sum, sum of the terms' magnitudes), float64."""
    T, k = rows.shape
    out = torch.zeros(T, y.shape[1], dtype=torch.float64, device=y.device) if residual is None else residual.double()
    mag = out.abs()
    for j in range(k):
        t = ((rows[:, j] >= 0) & (rows[:, j] < y.shape[0])).nonzero()[:, 0]
        term = y[rows[t, j].long()].double() * (1.0 if weights is None else weights[t, j, None].double())
        out[t] += term
        mag[t] += term.abs()
    return out, mag


def rmsnorm(s, weight, eps):
    s = s.double()
    return s / torch.sqrt(s.square().mean(1, keepdim=True) + eps) * weight.double()


def rmsnorm_backward(dy, s, weight, eps, dsum=None):
    """dx, dweight by the chain rule through the row's norm."""
    s, dy, w = s.double(), dy.double(), weight.double()
    n = torch.sqrt(s.square().mean(1, keepdim=True) + eps)
    d = dy * w
    dx = d / n - s * (d * s).mean(1, keepdim=True) / n ** 3
    return dx if dsum is None else dx + dsum.double(), (dy * s / n).sum(0)


def act(z, name):
    if name == "relu":
        return torch.where(z < 0, 0.0, z)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        a, b = math.sqrt(2 / math.pi), 0.044715
        p = torch.sigmoid(2 * a * (z + b * z ** 3))
        return p + z * p * (1 - p) * 2 * a * (1 + 3 * b * z * z)
    if name == "silu":
        p = torch.sigmoid(z)
        return p + z * p * (1 - p)
    return torch.ones_like(z)


def values(q, s):
    """Codes (float8 or uint8) times their 1x128 scales, float64."""
    q = q.view(torch.float8_e4m3fn).double()
    return (q.unflatten(-1, (-1, 128)) * s.double().unsqueeze(-1)).flatten(-2)


def pow2(e):
    """2^e in float64, from its bits (a power function may be off by a last place)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def e4m3(v):
    """The nearest e4m3 value of each float64, ties to even, saturating."""
    _, e = torch.frexp(v)
    step = pow2((e - 1).clamp_min(-6) - 3)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def next_pow2(s):
    """2^e for s = m 2^e, 1/2 <= m < 1."""
    return pow2(torch.frexp(s)[1])


def _half_step(v):
    return pow2((torch.frexp(v)[1] - 1).clamp_min(-6) - 4)


def quantise(v, above=False):
    """(codes as values, scales), float64, of 1x128 blocks of the last axis: both quotients rounded to FP32. above: the
    scale is the power of two above that."""
    b = v.double().unflatten(-1, (-1, 128))
    floor = torch.tensor(FLOOR, dtype=torch.float32, device=v.device).double()
    s = (torch.maximum(b.abs().amax(-1), floor) / TOP).float().double()
    if above:
        s = next_pow2(s)
    return e4m3((b / s.unsqueeze(-1)).float().double()).flatten(-2), s


def columns(v):
    """[M, N] -> [N, Mp], zeros past M."""
    return torch.nn.functional.pad(v, (0, 0, 0, -v.shape[0] % 128)).t().contiguous()


def check_codes(q, s, v, err, above=False, what=""):
    """Codes and scales against float64 values v that the kernel has, before quantisation, within err (elementwise).
    The scale is max(amax, floor) / 448 of values off by at most the block's largest err, with two roundings (the floor's, the
    quotient's) of 2^-24 each. A code is within half a step of v over the scale (2^(e-4) in [2^e, 2^(e+1)), 2^-10 below 2^-6),
    which v's error and the quotient's own rounding, another 2^-24 of it, may move."""
    b, e = v.unflatten(-1, (-1, 128)), err.unflatten(-1, (-1, 128))
    s = s.double()
    most, off = b.abs().amax(-1).clamp_min(FLOOR), e.amax(-1)
    low, high = (most - off).clamp_min(FLOOR) / TOP * (1 - 2.0 ** -23), (most + off) / TOP * (1 + 2.0 ** -23)
    if above:
        low, high = next_pow2(low), next_pow2(high)
        assert (torch.frexp(s)[0] == 0.5).all(), what
    assert ((s >= low) & (s <= high)).all(), f"{what}: scale off by {((s - low) / low).abs().max()}"
    t = b / s.unsqueeze(-1)
    got = q.view(torch.float8_e4m3fn).double().unflatten(-1, (-1, 128))
    moved = e / s.unsqueeze(-1) + t.abs() * 2.0 ** -23
    half = _half_step(t.abs() + moved)
    bound = half + moved
    worst = (got - t.clamp(-TOP, TOP)).abs() - bound
    assert (worst <= 0).all(), f"{what}: {int((worst > 0).sum())} codes off, worst by {worst.max()}"
