"""The norm with the residual's addition and its gradient, against their 64-bit forms.

The kernel's FP32 chain of a row: squares of up to 32 values a thread in two halves, 5 exchanges, 16 warps, the mean's product,
eps' sum, a rounded reciprocal square root (which halves the errors before it), two products: under 24 roundings of 2^-24."""
import pytest
import torch

import moe_grouped_gemm_tma_gb300 as dg
from tests import between_ref as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL = 24 * 2.0 ** -24


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def make(T, H, half, seed=0, residual=True):
    g = gen(seed + T + H)
    x = (torch.randn(T, H, device=DEV, generator=g) * 2).bfloat16()
    r = (torch.randn(T, H, device=DEV, generator=g) * 3).bfloat16() if residual else None
    w = 1 + 0.3 * torch.randn(H, device=DEV, generator=g)
    return x, r, w.bfloat16() if half else w


def run(x, r, w, y=True, q=True, keep=True, eps=1e-6, pow2=False):
    T, H = x.shape
    out = {"sum": torch.full_like(x, float("nan")) if keep else None, "y": torch.full_like(x, float("nan")) if y else None,
           "q": torch.full((T, H), 0x7F, dtype=torch.uint8, device=DEV) if q else None, "sf": torch.full((T, H // 128), -1.0, device=DEV) if q else None}
    dg.dg_rmsnorm(x, w, y=out["y"], q=out["q"], sf=out["sf"], residual=r, sum=out["sum"], eps=eps, pow2=pow2)
    return out


def check(x, r, w, out, eps, pow2=False):
    eps = float(torch.tensor(eps, dtype=torch.float32))
    s = x if r is None else (x.float() + r.float()).bfloat16()         # one FP32 addition, one rounding
    if out["sum"] is not None:
        assert torch.equal(out["sum"], s)
    want = B.rmsnorm(s, w, eps)
    if out["y"] is not None:
        assert ((out["y"].double() - want).abs() <= (2.0 ** -8 + 2 * REL) * want.abs() + 2.0 ** -133).all()
    if out["q"] is not None:
        B.check_codes(out["q"], out["sf"], want, REL * want.abs(), pow2)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("T,H", [(1, 128), (1, 7168), (3, 256), (5, 384), (4, 512), (33, 1024), (7, 1152), (130, 2048), (9, 4096), (1, 16384), (40, 7168), (2, 8320)])
def test_norm(T, H, half, pow2):
    x, r, w = make(T, H, half)
    out = run(x, r, w, pow2=pow2)
    check(x, r, w, out, 1e-6, pow2)
    plain = run(x, None, w, pow2=pow2)
    check(x, None, w, plain, 1e-6, pow2)
    # the same bits with fewer outputs, and in place
    for kw in (dict(y=False, keep=False), dict(q=False, keep=False), dict(y=False, q=False)):
        some = run(x, r, w, pow2=pow2, **kw)
        for n, v in some.items():
            assert v is None or torch.equal(v.view(torch.uint8), out[n].view(torch.uint8)), n
    a, b = x.clone(), r.clone()
    dg.dg_rmsnorm(a, w, y=a, residual=b, sum=b)
    assert torch.equal(a, out["y"]) and torch.equal(b, out["sum"])
    a = x.clone()
    dg.dg_rmsnorm(a, w, residual=r, sum=a)
    assert torch.equal(a, out["sum"])


@pytest.mark.parametrize("H", [8, 40, 264, 520, 1000, 1032, 2104, 5000, 16376])
def test_norm_of_odd_widths(H):
    x, r, w = make(21, H, False)
    check(x, r, w, run(x, r, w, q=False), 1e-6)


def test_zero_rows_and_eps():
    x, r, w = make(6, 2048, False)
    x[2], r[2] = 0, 0
    x[3], r[3] = 1e-6, 0
    x[4], r[4] = 2.0 ** -120, 0
    out = run(x, r, w, eps=1e-5)
    assert (out["y"][2] == 0).all() and (out["q"][2] == 0).all()
    assert torch.equal(out["sf"][2].cpu(), (torch.tensor(1e-4) / torch.tensor(448.0)).expand(16))
    check(x, r, w, out, 1e-5)
    big, _, w = make(3, 1024, False)
    check(big, None, w, run(big, None, w, eps=0.0), 0.0)
    check(big, None, w, run(big, None, w, eps=3.0), 3.0)


def test_nan_and_infinity_stay_in_their_row():
    x, r, w = make(9, 1536, False)
    want = run(x, r, w)
    x[4, 77], x[6, 1000] = float("nan"), float("inf")
    got = run(x, r, w)
    ok = [i for i in range(9) if i not in (4, 6)]
    for n in ("sum", "y", "q", "sf"):
        assert torch.equal(got[n][ok].view(torch.uint8), want[n][ok].view(torch.uint8)), n
    assert got["y"][4].isnan().all() and got["sf"][4].isnan().all() and got["y"][6, 1000].isnan()
    assert (got["y"][6, :999] == 0).all()         # over an infinite norm


def test_weights_of_both_signs_and_zero():
    x, r, w = make(5, 256, False)
    w[:128] = 0
    w[200] = -5.0
    check(x, r, w, run(x, r, w), 1e-6)


# ---------------------------------------------------------------- gradient
def backward(dy, s, w, dsum=None, eps=1e-6, dweight=True, ws=None):
    T, H = s.shape
    dx = torch.full_like(s, float("nan"))
    dw = torch.full((H,), float("nan"), device=DEV) if dweight else None
    ws = dg.rmsnorm_backward_workspace(T, H).fill_(0xFF) if ws is None else ws
    dg.dg_rmsnorm_backward(dy, s, w, dx, dw, ws if dweight else None, dsum=dsum, eps=eps)
    return dx, dw


def check_backward(dy, s, w, dsum, eps, dx, dw):
    eps = float(torch.tensor(eps, dtype=torch.float32))
    want, want_dw = B.rmsnorm_backward(dy, s, w, eps, dsum)
    sd, d, wd = s.double(), dy.double(), w.double()
    r = 1 / torch.sqrt(sd.square().mean(1, keepdim=True) + eps)
    # terms' magnitudes: both parts of dx and dsum are off by the row's chain (3 r's and a sum of products, whose error is
    # relative to the products' magnitudes), then one rounding to BF16
    mag = r * (d * wd).abs() + sd.abs() * r ** 3 * (d * wd * sd).abs().mean(1, keepdim=True) + (0 if dsum is None else dsum.double().abs())
    assert ((dx.double() - want).abs() <= 2.0 ** -8 * want.abs() + 4 * REL * mag + 2.0 ** -133).all()
    if dw is not None:
        # a product, r's chain, and the sum: a CTA's rows (up to 8 warps'), ctas / 16, 16 warps
        T, H = s.shape
        ctas = dg.load().dg_rmsnorm_backward_workspace(T, H) // (4 * H)
        chain = 24 + 3 + -(-T // ctas) + 8 + -(-ctas // 16) + 16
        assert ((dw.double() - want_dw).abs() <= chain * 2.0 ** -24 * (d * sd * r).abs().sum(0)).all()


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("T,H", [(1, 8), (1, 7168), (3, 256), (70, 384), (1300, 512), (33, 1024), (700, 1152), (330, 2048), (1, 16384), (610, 7168), (2, 1000), (5, 5000), (2500, 136), (5000, 1000), (9, 2048), (1250, 3000), (200, 12000)])
def test_backward(T, H, half):
    s, dsum, w = make(T, H, half)
    dy = torch.randn(T, H, device=DEV, generator=gen(9)).bfloat16()
    dx, dw = backward(dy, s, w, dsum)
    check_backward(dy, s, w, dsum, 1e-6, dx, dw)
    plain, dw2 = backward(dy, s, w)
    check_backward(dy, s, w, None, 1e-6, plain, dw2)
    assert torch.equal(dw, dw2)
    alone, _ = backward(dy, s, w, dsum, dweight=False)
    assert torch.equal(alone, dx)
    for name in ("dy", "x", "dsum"):              # in place
        a = {"dy": dy.clone(), "x": s.clone(), "dsum": dsum.clone()}
        dg.dg_rmsnorm_backward(a["dy"], a["x"], w, a[name], dsum=a["dsum"])
        assert torch.equal(a[name], dx), name


def test_backward_of_no_rows_is_zero():
    dw = torch.full((256,), 7.0, device=DEV)
    e = torch.empty(0, 256, dtype=torch.bfloat16, device=DEV)
    dg.dg_rmsnorm_backward(e, e, torch.ones(256, device=DEV), e, dw)
    assert (dw == 0).all()


def test_backward_of_zero_rows():
    s, _, w = make(4, 512, False)
    s[1] = 0
    dy = torch.randn(4, 512, device=DEV, generator=gen(9)).bfloat16()
    dx, dw = backward(dy, s, w, eps=1e-2)
    check_backward(dy, s, w, None, 1e-2, dx, dw)


def test_backward_against_differences():
    # the kernel's own forward in BF16 is too coarse for differences: its 64-bit form, whose gradient test_between_refusals.py
    # holds to differences, is differenced here at the kernel's inputs along random directions
    s, _, w = make(6, 640, False)
    dy = torch.randn(6, 640, device=DEV, generator=gen(3)).bfloat16()
    dx, dw = backward(dy, s, w)
    for i in range(4):
        v = torch.randn(6, 640, device=DEV, generator=gen(20 + i), dtype=torch.float64)
        u = torch.randn(640, device=DEV, generator=gen(30 + i), dtype=torch.float64)
        h = 1e-6
        f = lambda a, b: float((B.rmsnorm(a, b, 1e-6) * dy.double()).sum())  # noqa: E731
        sd, wd = s.double(), w.double()
        along = (f(sd + h * v, wd) - f(sd - h * v, wd)) / (2 * h)
        # each dx is off by 2^-8 of itself
        assert abs(float((dx.double() * v).sum()) - along) <= 1.1 * 2.0 ** -8 * float((dx.double() * v).abs().sum())
        along = (f(sd, wd + h * u) - f(sd, wd - h * u)) / (2 * h)
        assert abs(float((dw.double() * u).sum()) - along) <= 2.0 ** -18 * float((dw.double() * u).abs().sum()) + 1e-4


def test_many_rows_past_32_bits():
    T, H = 2 ** 17 + 3, 16384                     # 4.3 GB
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    x[-2:] = torch.randn(2, H, device=DEV, generator=gen(1)).bfloat16()
    w = torch.ones(H, device=DEV)
    q, sf = torch.empty(T, H, dtype=torch.uint8, device=DEV), torch.empty(T, H // 128, device=DEV)
    dg.dg_rmsnorm(x, w, q=q, sf=sf)
    want = B.rmsnorm(x[-2:], w, float(torch.tensor(1e-6)))
    B.check_codes(q[-2:], sf[-2:], want, REL * want.abs())
    dx, dw = torch.empty_like(x), torch.empty(H, device=DEV)
    dg.dg_rmsnorm_backward(x, x, w, dx, dw, dg.rmsnorm_backward_workspace(T, H))
    check_backward(x[-2:], x[-2:], w, None, 1e-6, dx[-2:], None)
    assert torch.isfinite(dw).all() and (dx[:-2] == 0).all()
