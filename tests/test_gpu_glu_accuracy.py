"""How good the gated activation's values and slopes are, gate by gate: where one value of a scaling block is not 0, the block's
scale is that value over 448, rounded to FP32, so that it shows all 24 bits. Every BF16 gate is looked at, each with a factor that
brings its product to about 1.

The bounds count roundings of 2^-24. The base-2 exponential is good to two last places, 4 of them; the reciprocal with its
Newton step to 2."""
import pytest
import torch

import moe_grouped_gemm_tma_gb300 as dg
from tests import between_ref as B
from tests.test_gpu_glu import DEV, run_backward

pytestmark = pytest.mark.gpu
UNIT = 2.0 ** -24
FLOOR = (torch.tensor(1e-4) / torch.tensor(448.0)).double().item()
ACTS = ["silu", "gelu_tanh", "gelu", "relu", "none"]


def gates():
    """Every finite BF16 number but those whose square is not one (and the zeros)."""
    g = torch.arange(-2 ** 15, 2 ** 15, device=DEV, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    return g[torch.isfinite(g) & (g.abs() < 2.0 ** 60) & (g.abs() > 2.0 ** -60)]


def diagonal(v):
    """[n padded to 128, 128] of zeros, with v[r] in column r % 128 of row r."""
    n = len(v)
    out = torch.zeros(B.up(n), 128, dtype=torch.bfloat16, device=DEV)
    r = torch.arange(n, device=DEV)
    out[r, r % 128] = v.bfloat16()
    return out


def to_one(v):
    """The powers of two that bring v to [1, 2), as far as BF16 has them."""
    return B.pow2((1 - torch.frexp(v.abs())[1]).clamp(-126, 127))


def sigmoid_and_argument(g, act):
    y = g if act == "silu" else 2 * 0.7978845608028654 * (g + 0.044715 * g ** 3)
    return torch.sigmoid(y), y


def forward_units(g, act):
    """How far a value may be off, in units of itself."""
    m = g.abs()
    if act == "silu":
        # the exponential, its two-part argument (of which (z times the rest of log2 e)^2 / 2 is left out), a rounding of it; then
        # the reciprocal and the product
        p, _ = sigmoid_and_argument(g, act)
        return (1 - p) * (4 + 1 + 1 + (4.9e-6 * m.clamp_max(90)) ** 2 / 2 / UNIT) + 2 + 1
    if act == "gelu_tanh":
        # y by constants and two operations, three roundings, which its exponential makes |y| times as large; the exponential; a sum, its
        # approximate reciprocal (a last place), the product
        p, y = sigmoid_and_argument(g, act)
        return (1 - p) * (4 + 3 * y.abs().clamp_max(200)) + 1 + 2 + 1
    if act == "gelu":
        # below zero: the tail's polynomial (3.4e-7) and its argument (five roundings), the exponential, and what its argument m^2 / 2 is
        # off, by a constant's rounding and its own; above zero that is of what is taken from z, which has a rounding
        tail = 5.7 + 5 + 4 + 2 + 0.75 * m.clamp_max(14) ** 2
        part = torch.special.ndtr(-m)
        return torch.where(g < 0, tail, tail * part + 1)
    return torch.zeros_like(m)


@pytest.mark.parametrize("act", ACTS)
def test_forward_values(act):
    g = gates()
    gd = g.double()
    a = B.act(gd, act)
    ok = a.abs() >= 2.0 ** -119
    u = torch.where(ok, to_one(a), 1.0)
    n = len(g)
    Z = torch.cat((diagonal(g), diagonal(u)), 1)
    M = Z.shape[0]
    q, sf = torch.empty(M, 128, dtype=torch.uint8, device=DEV), torch.empty(M, 1, device=DEV)
    dg.dg_glu(Z, q, sf, act=act)
    h = (a * u).abs().clamp_min(1e-4)
    off = (sf[:n, 0].double() * 448 / h - 1).abs()[ok] / UNIT
    bound = (forward_units(gd, act) + 2)[ok]              # (and the two roundings of a scale)
    assert (off <= bound).all(), f"{(off / bound).max()} times the bound at {g[ok][(off / bound).argmax()]}: {off.max()}"


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu"])
def test_activations_that_vanish_are_nothing_times_anything(act):
    g = gates()
    gd = g.double()
    small = (gd < 0) & (B.act(gd, act).abs() < 2.0 ** -119) & (gd < -1)
    assert small.sum() > 5000
    g, gd = g[small], gd[small]
    n = len(g)
    u = torch.full((n,), 2.0 ** 127, device=DEV)
    Z = torch.cat((diagonal(g), diagonal(u)), 1)
    M = Z.shape[0]
    q, sf = torch.empty(M, 128, dtype=torch.uint8, device=DEV), torch.empty(M, 1, device=DEV)
    dg.dg_glu(Z, q, sf, act=act)
    back = run_backward(diagonal(torch.full((n,), 2.0 ** 60, device=DEV)), Z=Z, act=act)
    h = sf[:n, 0].double()
    r = torch.arange(n, device=DEV)
    du, ht = back["q"][1][:n, 1].double(), back["ht"][1].double()[r % 128, r // 128]
    assert (h <= 2.0 ** 8 / 448 * 1.001).all() and (ht <= 2.0 ** 8 / 448 * 1.001).all() and (du <= FLOOR).all()
    gone = gd <= -88
    assert (h[gone] == FLOOR).all() and (ht[gone] == FLOOR).all()
    assert (q[:n][gone] & 0x7F == 0).all()
    # 2^60 2^127 is past FP32, and so is the slope's product with it where it has one; times 1 and 1 it is nothing
    Z[:, 128:] = (Z[:, 128:] != 0).bfloat16()
    back = run_backward(diagonal(torch.ones(n, device=DEV)), Z=Z, act=act)
    assert (back["q"][1][:n] == FLOOR).all() and (back["q"][0] & 0x7F == 0).all()


@pytest.mark.parametrize("act", ACTS)
def test_backward_values_and_slopes(act):
    g = gates()
    gd = g.double()
    n = len(g)
    a, slope = B.act(gd, act), B.slope(gd, act)
    ok = a.abs() >= 2.0 ** -119
    k = torch.where(ok, to_one(a), 1.0)
    r = torch.arange(n, device=DEV)

    def run(dh, u):
        out = run_backward(diagonal(dh), Z=torch.cat((diagonal(g), diagonal(u)), 1), act=act)
        rows = out["q"][1][:n].double() * 448
        columns = out["qt"][1].double() * 448
        # a row's one value is a column's one value too
        assert torch.equal(rows[:, 0], columns[r % 128, r // 128]) and torch.equal(rows[:, 1], columns[128 + r % 128, r // 128])
        return rows[:, 0], rows[:, 1], out["ht"][1].double()[r % 128, r // 128] * 448

    # du = dh act(g) and h = act(g) u at about 1, the slope times 1
    _, du, _ = run(k, torch.ones_like(k))
    _, _, h = run(torch.ones_like(k), k)
    want = (a * k).abs().clamp_min(1e-4)
    if act == "gelu":
        # Phi to 8e-8, its exponential and the product, of z
        m = gd.abs().clamp_max(14)
        off = gd.abs() * (8e-8 + (torch.special.ndtr(-m) * (4 + 0.75 * m * m) + 2) * UNIT) * k + 2 * UNIT * want
        off = torch.where(gd < -1, off + want * (4e-6 + (4 + 0.75 * m * m) * UNIT), off)
    else:
        units = forward_units(gd, act) + 2 + (0 if act in ("relu", "none") else 1)
        if act == "gelu_tanh":
            # the exponential, two roundings of its argument and itself, y by two constants and two operations; reciprocal, two products
            p, y = sigmoid_and_argument(gd, act)
            units = (1 - p) * (4 + 2 + 4 * y.abs().clamp_max(200)) + 2 + 1 + 1 + 2
        off = units * UNIT * want
    for name, got in (("du", du), ("h", h)):
        bad = ((got - want).abs() - off)[ok]
        assert (bad <= 0).all(), f"{name}: {((got - want).abs() / off)[ok].max()} times the bound at {g[ok][bad.argmax()]}"
    # slopes: to a few roundings of 1 (2^-21), seen where they pass the scale's floor
    one = torch.ones_like(k)
    dz, _, _ = run(1024 * one, one)
    assert ((dz - (1024 * slope).abs().clamp_min(1e-4)).abs() <= 1024 * 2.0 ** -21 * (1 + slope.abs())).all()
