"""The gated activation, the codes that it keeps, its backward pass and the transposition of codes, against their 64-bit forms."""
import pytest
import torch

import moe_grouped_gemm_tma_gb300 as dg
from tests import between_ref as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
ACTS = ["silu", "gelu", "gelu_tanh", "relu", "none"]
E4M3 = torch.float8_e4m3fn


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def make_z(M, I, seed=0, spread=2.0):
    return (torch.randn(M, 2 * I, device=DEV, generator=gen(seed + M + I)) * spread).bfloat16()


def value_error(g, h, u):
    """How far an activation times u may be off. Relative: 2^-18 for the exponential's and the reciprocal's approximations, and the
    rounding of the exponent's argument, 2^-24 of up to 0.8 (|g| + 0.05 |g|^3) log2(e), which the sigmoid's relative error
    carries over; absolute: the sigmoid is held at 2^-63 and more (5e-18 of |u|)."""
    return h.abs() * (2.0 ** -18 + 2.0 ** -23 * (g.abs() + 0.1 * g.abs() ** 3)) + 1e-17 * u.abs()


def alloc(M, I, keep, fill=0x55):
    q = torch.full((M, I), fill, dtype=torch.uint8, device=DEV)
    sf = torch.full((M, I // 128), -3.0, device=DEV)
    kept = torch.full((M, 2 * I), fill, dtype=torch.uint8, device=DEV) if keep else None
    ksf = torch.full((M, 2 * I // 128), -3.0, device=DEV) if keep else None
    return q, sf, kept, ksf


def check_glu(Z, I, act, pow2, rows, q, sf, kept, ksf):
    g, u = Z[rows].double().split(I, 1)
    h = B.act(g, act) * u
    B.check_codes(q[rows], sf[rows], h, value_error(g, h, u), pow2, act)
    if kept is not None:
        want, s = B.quantise(Z[rows])
        assert torch.equal(kept[rows].view(E4M3).double(), want) and torch.equal(ksf[rows].double(), s)
    if len(rows) < Z.shape[0]:
        other = torch.ones(Z.shape[0], dtype=torch.bool, device=DEV)
        other[rows] = False
        assert (q[other] == 0x55).all() and (sf[other] == -3.0).all()
        assert kept is None or ((kept[other] == 0x55).all() and (ksf[other] == -3.0).all())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M,I", [(1, 128), (3, 256), (5, 2048), (31, 384), (129, 128), (333, 640)])
def test_glu(M, I, act, pow2):
    Z = make_z(M, I)
    out = alloc(M, I, True)
    dg.dg_glu(Z, *out, act=act, pow2=pow2)
    check_glu(Z, I, act, pow2, torch.arange(M, device=DEV), *out)
    q, sf, _, _ = alloc(M, I, False)
    dg.dg_glu(Z, q, sf, act=act, pow2=pow2)
    assert torch.equal(q, out[0]) and torch.equal(sf, out[1])


def test_glu_over_the_whole_range():
    # every BF16 gate within 60, with u = 1: activations that vanish, and those that are the gate itself
    g = torch.arange(-2 ** 15, 2 ** 15, device=DEV, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    g = g[torch.isfinite(g) & (g.abs() < 60)]
    n = len(g) // 128
    Z = torch.ones(n, 256, dtype=torch.bfloat16, device=DEV)
    Z[:, :128] = g[: n * 128].view(n, 128)
    for act in ACTS:
        out = alloc(n, 128, True)
        dg.dg_glu(Z, *out, act=act)
        check_glu(Z, 128, act, False, torch.arange(n, device=DEV), *out)


@pytest.mark.parametrize("keep", [False, True])
def test_glu_of_the_contiguous_layout(keep):
    I = 384
    first = torch.tensor([3, -1, 0, 7, -1, -1, 2], dtype=torch.int32, device=DEV)         # the experts of seven blocks
    m_indices = first.repeat_interleave(128)
    m_indices[2 * 128 + 5:3 * 128] = -1           # a block with five rows: all of it is computed
    M = len(m_indices)
    Z = make_z(M, I)
    out = alloc(M, I, keep)
    dg.dg_glu(Z, *out, m_indices=m_indices)
    rows = torch.cat([torch.arange(b * 128, (b + 1) * 128, device=DEV) for b in (0, 2, 3, 6)])
    check_glu(Z, I, "silu", False, rows, *out)


@pytest.mark.parametrize("max_m", [1, 3, 16, 37, 200])
def test_glu_of_the_masked_layout(max_m):
    I, counts = 256, [0, 1, max_m, 5 * max_m + 7, 2, 0, -3]
    G = len(counts)
    masked_m = torch.tensor(counts, dtype=torch.int32, device=DEV)
    Z = make_z(G * max_m, I)
    out = alloc(G * max_m, I, True)
    shaped = lambda t: t.view(G, max_m, -1)  # noqa: E731
    dg.dg_glu(shaped(Z), *(shaped(t) for t in out), masked_m=masked_m, act="gelu")
    rows = torch.cat([torch.arange(g * max_m, g * max_m + max(0, min(c, max_m)), device=DEV) for g, c in enumerate(counts)])
    check_glu(Z, I, "gelu", False, rows, *out)


def test_nan_and_infinity_stay_in_their_blocks():
    M, I = 40, 512
    Z = make_z(M, I)
    want = alloc(M, I, True)
    dg.dg_glu(Z, *want)
    Z[7, 130], Z[20, I + 400], Z[33, 5] = float("nan"), float("inf"), float("nan")
    got = alloc(M, I, True)
    dg.dg_glu(Z, *got)
    spoilt = torch.zeros(M, 2 * I // 128, dtype=torch.bool, device=DEV)
    for r, c in ((7, 130), (20, I + 400), (33, 5)):
        spoilt[r, c // 128] = True
    same = lambda a, b, m: torch.equal(a.unflatten(1, (m.shape[1], -1))[~m], b.unflatten(1, (m.shape[1], -1))[~m])  # noqa: E731
    assert same(got[2], want[2], spoilt) and same(got[3], want[3], spoilt)
    h = spoilt[:, : I // 128] | spoilt[:, I // 128:]
    assert same(got[0], want[0], h) and same(got[1], want[1], h)
    assert not torch.isfinite(got[1][h]).any() and not torch.isfinite(got[3][spoilt]).any()


# ---------------------------------------------------------------- backward
def slope_error(g):
    """The slopes are right to a few roundings of 1: 2^-21."""
    return torch.full_like(g, 2.0 ** -21)


def run_backward(dH, Z=None, kept=None, ksf=None, act="silu", parts=("q", "qt", "ht")):
    M, I = dH.shape
    Mp = B.up(M)
    out = {}
    for name, n, m in (("q", M, 2 * I), ("qt", 2 * I, Mp), ("ht", I, Mp)):
        out[name] = (torch.full((n, m), 0x7F, dtype=torch.uint8, device=DEV), torch.full((n, m // 128), -3.0, device=DEV)) if name in parts else (None, None)
    dg.dg_glu_backward(dH, *out["q"], *out["qt"], *out["ht"], Z=Z, kept=kept, kept_sf=ksf, act=act)
    return out


def check_backward(dH, g, u, act, out, input_error):
    """input_error: how far the kernel's g and u may be from these, relative (codes times scales are rounded to FP32)."""
    d = dH.double()
    a, s = B.act(g, act), B.slope(g, act)
    ae = value_error(g, a, torch.ones_like(g)) + input_error * (g * s).abs() * 1.01
    # the slope's own slope is below 1.2 everywhere
    se = slope_error(g) + 1.2 * input_error * g.abs()
    few = 3 * 2.0 ** -24 + input_error
    dg_, du, h = d * u * s, d * a, a * u
    err = torch.cat(((d * u).abs() * se + few * dg_.abs(), d.abs() * ae + few * du.abs()), 1)
    dz = torch.cat((dg_, du), 1)
    if out["q"][0] is not None:
        B.check_codes(*out["q"], dz, err, what="rows")
    if out["qt"][0] is not None:
        B.check_codes(*out["qt"], B.columns(dz), B.columns(err), what="columns")
    if out["ht"][0] is not None:
        B.check_codes(*out["ht"], B.columns(h), B.columns(u.abs() * ae + few * h.abs()), what="h")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("M,I", [(1, 128), (5, 256), (128, 128), (129, 384), (300, 640), (1000, 2048)])
def test_backward(M, I, act, kept):
    Z = make_z(M, I, seed=3)
    dH = (torch.randn(M, I, device=DEV, generator=gen(M)) * 0.05).bfloat16()
    if kept:
        q, sf, codes, ksf = alloc(M, I, True)
        dg.dg_glu(Z, q, sf, codes, ksf, act=act)
        out = run_backward(dH, kept=codes, ksf=ksf, act=act)
        g, u = B.values(codes, ksf).split(I, 1)
    else:
        out = run_backward(dH, Z=Z, act=act)
        g, u = Z.double().split(I, 1)
    check_backward(dH, g, u, act, out, 2.0 ** -24 if kept else 0.0)
    if M % 128:
        for name in ("qt", "ht"):
            assert (out[name][0][:, M:] == 0).all()
    # a part alone gives the same bits
    for name in ("q", "qt", "ht"):
        some = run_backward(dH, Z=None if kept else Z, kept=codes if kept else None, ksf=ksf if kept else None, act=act, parts=(name,))
        assert torch.equal(some[name][0], out[name][0]) and torch.equal(some[name][1], out[name][1]), name


def test_backward_over_the_whole_range():
    g = torch.arange(-2 ** 15, 2 ** 15, device=DEV, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    g = g[torch.isfinite(g) & (g.abs() < 60)]
    n = len(g) // 128
    Z = torch.ones(n, 256, dtype=torch.bfloat16, device=DEV)
    Z[:, :128] = g[: n * 128].view(n, 128)
    dH = torch.ones(n, 128, dtype=torch.bfloat16, device=DEV)
    for act in ACTS:
        out = run_backward(dH, Z=Z, act=act)
        check_backward(dH, Z[:, :128].double(), Z[:, 128:].double(), act, out, 0.0)


@pytest.mark.parametrize("act", ACTS)
def test_very_large_gates(act):
    # beyond where any exponential of them is finite: the activation is the gate or nothing, its slope 1 or 0
    big = torch.tensor([60.0, 86.0, 87.0, 88.0, 90.0, 100.0, 126.0, 150.0, 1000.0, 65536.0, 2.0 ** 60, 2.0 ** 100, 2.0 ** 126], device=DEV)
    g = torch.cat((big, -big)).repeat(5)[:128].bfloat16()
    Z = torch.ones(3, 256, dtype=torch.bfloat16, device=DEV)
    Z[1, :128] = g.abs().neg()
    Z[0, :128], Z[2, :128] = g.abs(), 0.5
    Z[:, 128:] = 2.0 ** -30
    out = alloc(3, 128, True)
    dg.dg_glu(Z, *out, act=act)
    back = run_backward(torch.ones(3, 128, dtype=torch.bfloat16, device=DEV), Z=Z, act=act)
    gd, u = Z.double().split(128, 1)
    value = torch.where(gd > 1, gd, B.act(gd.clamp(-80, 1), act) if act != "none" else gd)
    slope = torch.where(gd > 1, 1.0, B.slope(gd.clamp(-80, 1), act) if act != "none" else 1.0)
    err = lambda v: v.abs() * 2.0 ** -17 + 1e-17  # noqa: E731
    B.check_codes(out[0], out[1], value * u, err(value * u), what="h")
    dz = torch.cat((u * slope, value), 1)
    B.check_codes(*back["q"], dz, err(dz), what="rows")
    B.check_codes(*back["qt"], B.columns(dz), B.columns(err(dz)), what="columns")
    B.check_codes(*back["ht"], B.columns(value * u), B.columns(err(value * u)), what="h")


def test_backward_nan_stays_in_its_blocks():
    M, I = 256, 256
    Z, dH = make_z(M, I), torch.randn(M, I, device=DEV, generator=gen(1)).bfloat16()
    want = run_backward(dH, Z=Z)
    dH[140, 7] = float("nan")
    got = run_backward(dH, Z=Z)
    rows = torch.zeros(M, 4, dtype=torch.bool, device=DEV)
    rows[140, 0] = rows[140, 2] = True
    assert torch.equal(got["q"][1].isnan(), rows)
    cols = torch.zeros(2 * I, 2, dtype=torch.bool, device=DEV)
    cols[7, 1] = cols[I + 7, 1] = True
    assert torch.equal(got["qt"][1].isnan(), cols)
    keep = ~cols.repeat_interleave(128, 1)
    assert torch.equal(got["qt"][0][keep], want["qt"][0][keep]) and torch.equal(got["ht"][0], want["ht"][0])


def test_backward_against_differences():
    # the gradients' values along random directions, against differences of the 64-bit form at the kept values
    M, I = 128, 256
    Z = make_z(M, I, spread=1.0)
    q, sf, codes, ksf = alloc(M, I, True)
    dg.dg_glu(Z, q, sf, codes, ksf, act="silu")
    dH = torch.randn(M, I, device=DEV, generator=gen(2)).bfloat16()
    out = run_backward(dH, kept=codes, ksf=ksf)
    z = B.values(codes, ksf)
    f = lambda z: float((B.act(z[:, :I], "silu") * z[:, I:] * dH.double()).sum())  # noqa: E731
    got = B.values(*out["q"])
    for i in range(4):
        v = torch.randn(M, 2 * I, device=DEV, generator=gen(10 + i), dtype=torch.float64)
        along = (f(z + 1e-6 * v) - f(z - 1e-6 * v)) / 2e-6
        # each code is off by 2^-4 of itself, or half the smallest step of its block
        off = (2.0 ** -4 * got.abs() + 2.0 ** -10 * out["q"][1].double().repeat_interleave(128, 1)) * v.abs() * 1.1
        assert abs(float((got * v).sum()) - along) <= float(off.sum())


# ---------------------------------------------------------------- transposition
@pytest.mark.parametrize("M,N", [(1, 128), (3, 256), (127, 128), (128, 384), (129, 128), (333, 2048), (1000, 640)])
def test_transpose(M, N):
    x = torch.randn(M, N, device=DEV, generator=gen(M)) * torch.exp(2 * torch.randn(M, 1, device=DEV, generator=gen(N)))
    q = torch.randint(0, 256, (M, N), dtype=torch.uint8, device=DEV, generator=gen(5))
    q[(q & 0x7F) == 0x7F] = 0                     # (no NaN)
    for codes in (q, (x / x.abs().amax(1, keepdim=True) * 448).to(E4M3).view(torch.uint8)):
        sf = x.abs().unflatten(1, (-1, 128)).amax(2) / 448
        qt, sft = torch.full((N, B.up(M)), 0x7F, dtype=torch.uint8, device=DEV), torch.full((N, B.up(M) // 128), -1.0, device=DEV)
        dg.dg_transpose_fp8(codes, sf, qt, sft)
        v = B.values(codes, sf).float()           # the product's one rounding
        want, s = B.quantise(B.columns(v))
        assert torch.equal(sft.double(), s) and torch.equal(qt.view(E4M3).double(), want)


def test_transpose_every_code_and_special_scales():
    q = torch.arange(256, device=DEV).to(torch.uint8).repeat(128, 1)[:, :256].contiguous()
    q[(q & 0x7F) == 0x7F] = 1
    sf = torch.ones(128, 2, device=DEV)
    sf[5], sf[9], sf[11, 1] = 0.0, 2.0 ** -30, 3.0e4
    qt, sft = torch.empty(256, 128, dtype=torch.uint8, device=DEV), torch.empty(256, 1, device=DEV)
    dg.dg_transpose_fp8(q, sf, qt, sft)
    want, s = B.quantise(B.columns(B.values(q, sf).float()))
    assert torch.equal(sft.double(), s) and torch.equal(qt.view(E4M3).double(), want)
    q[17, 3] = 0x7F                               # NaN
    sf[40, 1] = float("inf")
    dg.dg_transpose_fp8(q, sf, qt, sft)
    assert sft[3].isnan().all() and torch.equal(sft[:128].isnan().view(-1), torch.arange(128, device=DEV) == 3)
    assert not torch.isfinite(sft[128:]).any()    # (0 times the infinity is NaN)


def test_offsets_past_32_bits():
    M, N = 2 ** 18 + 5, 16384                     # 4.3 GB of codes
    q = torch.zeros(M, N, dtype=torch.uint8, device=DEV)
    sf = torch.ones(M, N // 128, device=DEV)
    q[-5:] = torch.randint(0, 0x7F, (5, N), dtype=torch.uint8, device=DEV, generator=gen(1))
    qt, sft = torch.empty(N, B.up(M), dtype=torch.uint8, device=DEV), torch.empty(N, B.up(M) // 128, device=DEV)
    dg.dg_transpose_fp8(q, sf, qt, sft)
    want, s = B.quantise(B.columns(B.values(q[-5:], sf[-5:]).float()))
    assert torch.equal(qt[:, -128:].view(E4M3).double(), want) and torch.equal(sft[:, -1:].double(), s)
    assert (qt[:, :-128] == 0).all()
    del q, qt
    M, I = 2 ** 17 + 5, 8192
    Z = torch.zeros(M, 2 * I, dtype=torch.bfloat16, device=DEV)
    Z[-5:] = make_z(5, I)
    out = alloc(M, I, True)
    dg.dg_glu(Z, *out)
    check_glu(Z[-5:], I, "silu", False, torch.arange(5, device=DEV), *(t[-5:] for t in out))
    dH = torch.zeros(M, I, dtype=torch.bfloat16, device=DEV)
    dH[-5:] = 1.0
    back = run_backward(dH, kept=out[2], ksf=out[3])
    last = {n: (c[-5:], s[-5:]) if n == "q" else (c[:, -128:], s[:, -1:]) for n, (c, s) in back.items()}
    check_backward(dH[-5:], *B.values(out[2][-5:], out[3][-5:]).split(I, 1), "silu", last, 2.0 ** -24)
