"""What the operators between the grouped products refuse, before any CUDA work (no GPU needed), their sizes, and their plain
forms' own checks (gradients against differences in 64 bits)."""
import ctypes
import random

import pytest
import torch

import moe_grouped_gemm_tma_gb300 as dg
from tests import between_ref as B


def _p(addr):
    return ctypes.c_void_p(addr)


OK, ODD8, ODD4, ODD2 = _p(0x10000), _p(0x10008), _p(0x10004), _p(0x10002)
INVALID, SHAPE, MISALIGNED = 1, 2, 3


def calls(f, base):
    return lambda **kw: f(*{**base, **kw}.values(), None)


def test_sort_refusals():
    L = dg.load()
    base = dict(ids=OK, rows=OK, counts=OK, m=OK, ws=OK, size=1 << 30, T=4, k=2, E=4, Mt=1024)
    call = calls(L.dg_moe_sort_contiguous, base)
    assert call(T=-1) == INVALID and call(k=-1) == INVALID and call(E=0) == INVALID and call(Mt=-128) == INVALID
    assert call(k=33) == SHAPE and call(E=1025) == SHAPE and call(T=1 << 23) == SHAPE
    assert call(Mt=1000) == SHAPE and call(Mt=384) == SHAPE          # 8 slots of 4 experts: up to 4 blocks
    for name in ("ids", "rows", "counts", "m"):
        assert call(**{name: None}) == INVALID, name
    for name in ("ids", "rows", "counts"):
        assert call(**{name: ODD2}) == MISALIGNED, name
    assert call(m=ODD8) == MISALIGNED and call(ws=ODD8) == MISALIGNED
    assert call(T=8193, ws=None, Mt=1 << 15) == INVALID and call(T=8193, size=16, Mt=1 << 15) == INVALID
    base = dict(ids=OK, rows=OK, counts=OK, ws=OK, size=1 << 30, T=4, k=2, E=4, max_m=16)
    call = calls(L.dg_moe_sort_masked, base)
    assert call(T=-1) == INVALID and call(k=-1) == INVALID and call(E=0) == INVALID and call(max_m=0) == INVALID and call(max_m=-1) == INVALID
    assert call(k=33) == SHAPE and call(E=1025) == SHAPE and call(max_m=1 << 29) == SHAPE
    for name in ("ids", "rows", "counts"):
        assert call(**{name: None}) == INVALID and call(**{name: ODD2}) == MISALIGNED, name


def test_sort_sizes():
    L = dg.load()
    rng = random.Random(3)
    for _ in range(200):
        T, k, E = rng.randint(0, 300), rng.randint(0, 8), rng.randint(1, 40)
        rows = L.dg_moe_sort_rows(T, k, E)
        # the worst routing: as many experts as possible with one slot more than whole blocks
        met = min(E, T * k)
        spare = T * k - met
        assert rows == 128 * (met + spare // 128), (T, k, E)
    assert L.dg_moe_sort_workspace(16384, 1, 8) == 0 and L.dg_moe_sort_workspace(1 << 20, 8, 8) == (608 + 1) * 8 * 4 and L.dg_moe_sort_workspace(16385, 1, 8) == (33 + 1) * 8 * 4
    for bad in ((-1, 1, 1), (1, -1, 1), (1, 1, 0), (1, 33, 64), (1, 1, 1025), (1 << 22, 8, 64)):
        assert L.dg_moe_sort_rows(*bad) == -1 and L.dg_moe_sort_workspace(*bad) == -1
    sizes = [L.dg_moe_sort_workspace(n, 1, 64) for n in range(16000, 1 << 20, 497)]
    assert sizes == sorted(sizes)                  # one for many tokens serves fewer
    with pytest.raises(dg.DGError):
        dg.moe_sort_rows(1, 33, 64)
    with pytest.raises(dg.DGError):
        dg.moe_sort_workspace(1, 33, 64)
    assert dg.moe_sort_rows(5, 2, 8) == 1024 and dg.moe_sort_rows(0, 2, 8) == 0


def test_gather_refusals():
    base = dict(x=OK, sf=OK, type=2, rows=OK, m=OK, out=OK, osf=OK, T=4, k=2, H=256, Mt=256)
    call = calls(dg.load().dg_moe_gather, base)
    bf16 = dict(type=0, sf=None, osf=None)
    assert call(type=1) == INVALID and call(type=3) == INVALID
    for name in ("T", "k", "H", "Mt"):
        assert call(**{name: -1}) == INVALID, name
    assert call(k=33) == SHAPE and call(H=200) == SHAPE and call(H=204, **bf16) == SHAPE and call(Mt=200) == SHAPE
    assert call(T=1 << 30, H=1 << 16) == SHAPE and call(T=2 ** 31 - 1, H=128) == SHAPE and call(Mt=2 ** 31 - 128) == SHAPE
    for name in ("x", "sf", "rows", "out", "osf"):
        assert call(**{name: None}) == INVALID, name
    assert call(type=0) == INVALID and call(type=0, sf=None) == INVALID          # scales go with codes
    for name in ("x", "out"):
        assert call(**{name: ODD8}) == MISALIGNED and call(**{name: ODD8}, **bf16) == MISALIGNED, name
    for name in ("sf", "osf", "rows", "m"):
        assert call(**{name: ODD2}) == MISALIGNED, name
    assert call(H=0) == 0 and call(Mt=0) == 0 and call(T=0, m=None) == 0 and call(k=0, m=None) == 0


def test_combine_refusals():
    base = dict(y=OK, rows=OK, w=OK, res=OK, out=OK, T=4, k=2, H=256, Mt=256)
    call = calls(dg.load().dg_moe_combine, base)
    for name in ("T", "k", "H", "Mt"):
        assert call(**{name: -1}) == INVALID, name
    assert call(k=33) == SHAPE and call(H=100) == SHAPE and call(T=2 ** 31 - 1, H=8) == SHAPE
    for name in ("y", "rows", "out"):
        assert call(**{name: None}) == INVALID, name
    for name in ("y", "res", "out"):
        assert call(**{name: ODD8}) == MISALIGNED, name
    for name in ("w", "rows"):
        assert call(**{name: ODD2}) == MISALIGNED, name
    assert call(T=0) == 0 and call(H=0) == 0
    base = dict(dout=OK, y=OK, rows=OK, w=OK, m=OK, dy=OK, dw=OK, T=4, k=2, H=256, Mt=256)
    call = calls(dg.load().dg_moe_combine_backward, base)
    for name in ("T", "k", "H", "Mt"):
        assert call(**{name: -1}) == INVALID, name
    assert call(k=33) == SHAPE and call(H=100) == SHAPE and call(Mt=200) == SHAPE and call(T=2 ** 31 - 1, H=8) == SHAPE
    for name in ("dout", "y", "rows"):
        assert call(**{name: None}) == INVALID, name
    for name in ("dout", "y", "dy"):
        assert call(**{name: ODD8}) == MISALIGNED, name
    for name in ("w", "rows", "dw", "m"):
        assert call(**{name: ODD2}) == MISALIGNED, name
    assert call(dy=None, dw=None) == 0 and call(T=0, m=None) == 0 and call(k=0, m=None) == 0


def test_rmsnorm_refusals():
    L = dg.load()
    base = dict(x=OK, res=OK, w=OK, type=1, sum=OK, y=OK, q=OK, sf=OK, pow2=0, T=4, H=256, eps=1e-6)
    call = calls(L.dg_rmsnorm, base)
    assert call(T=-1) == INVALID and call(H=-8) == INVALID and call(type=2) == INVALID and call(type=-1) == INVALID
    assert call(eps=-1.0) == INVALID and call(eps=float("nan")) == INVALID
    assert call(q=None) == INVALID and call(sf=None) == INVALID
    assert call(H=100) == SHAPE and call(H=16392) == SHAPE and call(H=200) == SHAPE and call(T=2 ** 31 - 1) == SHAPE
    assert call(x=None) == INVALID and call(w=None) == INVALID
    for name in ("x", "res", "w", "sum", "y", "q"):
        assert call(**{name: ODD8}) == MISALIGNED, name
    assert call(sf=ODD2) == MISALIGNED
    assert call(T=0) == 0 and call(H=0) == 0 and call(sum=None, y=None, q=None, sf=None) == 0
    base = dict(dy=OK, x=OK, w=OK, type=1, dsum=OK, dx=OK, dw=OK, ws=OK, size=1 << 30, T=4, H=256, eps=1e-6)
    call = calls(L.dg_rmsnorm_backward, base)
    assert call(T=-1) == INVALID and call(H=-8) == INVALID and call(type=2) == INVALID and call(eps=-1.0) == INVALID
    assert call(H=100) == SHAPE and call(H=16392) == SHAPE and call(T=2 ** 31 - 1) == SHAPE
    for name in ("dy", "x", "w", "dx"):
        assert call(**{name: None}) == INVALID, name
    assert call(ws=None) == INVALID and call(size=256 * 4 - 1) == INVALID and call(T=9, size=2 * 256 * 4 - 1) == INVALID
    for name in ("dy", "x", "w", "dsum", "dx", "ws"):
        assert call(**{name: ODD8}) == MISALIGNED, name
    assert call(dw=ODD2) == MISALIGNED
    assert call(H=0) == 0 and call(T=0, dw=None) == 0
    assert L.dg_rmsnorm_backward_workspace(4, 256) == 256 * 4 and L.dg_rmsnorm_backward_workspace(4, 2048) == 4 * 2048 * 4 and L.dg_rmsnorm_backward_workspace(1, 100) == -1
    assert L.dg_rmsnorm_backward_workspace(1 << 20, 7168) == 304 * 7168 * 4 and L.dg_rmsnorm_backward_workspace(1, 16392) == -1
    for H in (8, 1024, 1032, 2048, 4096, 7168, 16384):
        sizes = [L.dg_rmsnorm_backward_workspace(T, H) for T in range(0, 9000)]
        assert sizes == sorted(sizes)              # one for many rows serves fewer
    with pytest.raises(dg.DGError):
        dg.rmsnorm_backward_workspace(1, 100)


def test_glu_refusals():
    L = dg.load()
    base = dict(Z=OK, q=OK, sf=OK, kept=OK, ksf=OK, mi=None, mm=None, G=1, act=4, pow2=0, M=256, I=256)
    call = calls(L.dg_glu, base)
    assert call(M=-1) == INVALID and call(I=-1) == INVALID and call(G=-1) == INVALID and call(act=5) == INVALID and call(act=-1) == INVALID
    assert call(kept=None) == INVALID and call(ksf=None) == INVALID and call(mi=OK, mm=OK) == INVALID
    assert call(I=200) == SHAPE and call(mi=OK, M=200) == SHAPE and call(M=2 ** 31 - 1) == SHAPE and call(M=2 ** 30, I=1 << 20) == SHAPE
    assert call(mm=OK, G=0) == INVALID and call(mm=OK, G=3) == INVALID
    for name in ("Z", "q", "sf"):
        assert call(**{name: None}) == INVALID, name
    for name in ("Z", "q", "kept"):
        assert call(**{name: ODD8}) == MISALIGNED, name
    assert call(sf=ODD2) == MISALIGNED and call(ksf=ODD2) == MISALIGNED and call(mi=ODD2) == MISALIGNED and call(mm=ODD2) == MISALIGNED
    assert call(M=0) == 0 and call(I=0) == 0
    base = dict(dH=OK, Z=OK, kept=None, ksf=None, act=4, q=OK, sf=OK, qt=OK, sft=OK, ht=OK, hsft=OK, M=256, I=256)
    call = calls(L.dg_glu_backward, base)
    assert call(M=-1) == INVALID and call(I=-1) == INVALID and call(act=5) == INVALID
    for name in ("sf", "q", "sft", "qt", "hsft", "ht", "dH", "Z"):
        assert call(**{name: None}) == INVALID, name
    assert call(kept=OK) == INVALID and call(kept=OK, ksf=OK) == INVALID and call(ksf=OK) == INVALID      # one of Z and the codes
    assert call(I=200) == SHAPE and call(M=2 ** 31 - 1) == SHAPE and call(M=2 ** 30, I=1 << 22) == SHAPE
    for name in ("dH", "Z", "q", "qt", "ht"):
        assert call(**{name: ODD8}) == MISALIGNED, name
    assert call(Z=None, kept=ODD8, ksf=OK) == MISALIGNED and call(Z=None, kept=OK, ksf=ODD2) == MISALIGNED
    for name in ("sf", "sft", "hsft"):
        assert call(**{name: ODD2}) == MISALIGNED, name
    assert call(M=0) == 0 and call(I=0) == 0 and call(q=None, sf=None, qt=None, sft=None, ht=None, hsft=None) == 0


def test_transpose_refusals():
    call = calls(dg.load().dg_transpose_fp8, dict(q=OK, sf=OK, qt=OK, sft=OK, M=256, N=256))
    assert call(M=-1) == INVALID and call(N=-1) == INVALID and call(N=200) == SHAPE
    assert call(M=2 ** 31 - 1) == SHAPE and call(M=2 ** 30, N=1 << 22) == SHAPE
    for name in ("q", "sf", "qt", "sft"):
        assert call(**{name: None}) == INVALID, name
    assert call(q=ODD8) == MISALIGNED and call(qt=ODD8) == MISALIGNED and call(sf=ODD2) == MISALIGNED and call(sft=ODD2) == MISALIGNED
    assert call(M=0) == 0 and call(N=0) == 0


def e(*s, dtype=torch.float32):
    return torch.empty(*s, dtype=dtype)


def test_binding_refuses_host_tensors_types_and_shapes():
    b, i, u, h = torch.bfloat16, torch.int32, torch.uint8, torch.float16
    with pytest.raises(ValueError, match="CUDA tensor"):
        dg.dg_moe_sort_contiguous(e(2, 2, dtype=i), e(2, 2, dtype=i), e(4, dtype=i), e(512, dtype=i))
    with pytest.raises(TypeError, match="ids must be int32"):
        dg.dg_moe_sort_masked(e(2, 2, dtype=torch.int64), e(2, 2, dtype=i), e(4, dtype=i), 8)
    with pytest.raises(TypeError, match="x must be"):
        dg.dg_moe_gather(e(2, 128, dtype=h), None, e(2, 1, dtype=i), e(4, 128, dtype=h))
    with pytest.raises(ValueError, match="CUDA tensor"):
        dg.dg_moe_gather(e(2, 128, dtype=u), e(2, 1), e(2, 1, dtype=i), e(4, 128, dtype=u), e(4, 1))
    with pytest.raises(TypeError, match="y must be bfloat16"):
        dg.dg_moe_combine(e(4, 128), e(2, 1, dtype=i), e(2, 128, dtype=b))
    with pytest.raises(ValueError, match="dweights with y"):
        dg.dg_moe_combine_backward(e(2, 128, dtype=b), e(2, 1, dtype=i), None)
    with pytest.raises(TypeError, match="dout must be bfloat16"):
        dg.dg_moe_combine_backward(e(2, 128), e(2, 1, dtype=i), e(4, 128, dtype=b))
    with pytest.raises(TypeError, match="x must be bfloat16"):
        dg.dg_rmsnorm(e(2, 128), e(128))
    with pytest.raises(ValueError, match="CUDA tensor"):
        dg.dg_rmsnorm(e(2, 128, dtype=b), e(128))
    with pytest.raises(TypeError, match="x must be bfloat16"):
        dg.dg_rmsnorm_backward(e(2, 128, dtype=b), e(2, 128), e(128), e(2, 128, dtype=b))
    with pytest.raises(TypeError, match="Z must be bfloat16"):
        dg.dg_glu(e(2, 256), e(2, 128, dtype=u), e(2, 1))
    with pytest.raises(ValueError, match="one of Z and kept"):
        dg.dg_glu_backward(e(2, 128, dtype=b), *[None] * 6)
    with pytest.raises(TypeError, match="e4m3 codes"):
        dg.dg_transpose_fp8(e(2, 128), e(2, 1), e(128, 128, dtype=u), e(128, 1))


class _Cuda:
    """A host tensor that says it is on a GPU: it gets past the device check to the one under test."""

    def __init__(self, t, device=0):
        self._t, self._device, self.is_cuda, self.device = t, device, True, f"cuda:{device}"

    def get_device(self):
        return self._device

    def __getattr__(self, name):
        return getattr(self._t, name)


def c(*s, dtype=torch.float32, device=0):
    return _Cuda(e(*s, dtype=dtype), device)


def test_binding_refuses_shapes_layouts_and_devices():
    b, i, u = torch.bfloat16, torch.int32, torch.uint8
    with pytest.raises(ValueError, match="rows must have shape"):
        dg.dg_moe_sort_masked(c(2, 2, dtype=i), c(2, 3, dtype=i), c(4, dtype=i), 8)
    with pytest.raises(ValueError, match="rows is on cuda:1"):
        dg.dg_moe_sort_masked(c(2, 2, dtype=i), c(2, 2, dtype=i, device=1), c(4, dtype=i), 8)
    with pytest.raises(ValueError, match="sf and out_sf go with"):
        dg.dg_moe_gather(c(2, 128, dtype=u), None, c(2, 1, dtype=i), c(4, 128, dtype=u))
    with pytest.raises(ValueError, match="sf and out_sf go with"):
        dg.dg_moe_gather(c(2, 128, dtype=b), c(2, 1), c(2, 1, dtype=i), c(4, 128, dtype=b), c(4, 1))
    with pytest.raises(ValueError, match="rows must have shape"):
        dg.dg_moe_gather(c(2, 128, dtype=b), None, c(3, 1, dtype=i), c(4, 128, dtype=b))
    with pytest.raises(ValueError, match="m_indices must have shape"):
        dg.dg_moe_gather(c(2, 128, dtype=b), None, c(2, 1, dtype=i), c(128, 128, dtype=b), m_indices=c(4, dtype=i))
    with pytest.raises(ValueError, match="contiguous"):
        dg.dg_moe_combine(_Cuda(e(128, 4, dtype=b).t()), c(2, 1, dtype=i), c(2, 128, dtype=b))
    with pytest.raises(ValueError, match="weights must have shape"):
        dg.dg_moe_combine(c(4, 128, dtype=b), c(2, 1, dtype=i), c(2, 128, dtype=b), weights=c(2, 2))
    with pytest.raises(ValueError, match="y must have shape"):
        dg.dg_moe_combine_backward(c(2, 128, dtype=b), c(2, 1, dtype=i), c(4, 128, dtype=b), y=c(5, 128, dtype=b), dweights=c(2, 1))
    with pytest.raises(ValueError, match="weight must have shape"):
        dg.dg_rmsnorm(c(2, 128, dtype=b), c(64))
    with pytest.raises(ValueError, match="dx must have shape"):
        dg.dg_rmsnorm_backward(c(2, 128, dtype=b), c(2, 128, dtype=b), c(128), c(2, 64, dtype=b))
    with pytest.raises(ValueError, match="sf must have shape"):
        dg.dg_glu(c(2, 256, dtype=b), c(2, 128, dtype=u), c(2, 2))
    with pytest.raises(ValueError, match="even number of columns"):
        dg.dg_glu(c(2, 257, dtype=b), c(2, 128, dtype=u), c(2, 1))
    with pytest.raises(ValueError, match="masked_m must have shape"):
        dg.dg_glu(c(2, 4, 256, dtype=b), c(2, 4, 128, dtype=u), c(2, 4, 1), masked_m=c(4, dtype=i))
    with pytest.raises(ValueError, match="qt must have shape"):
        dg.dg_glu_backward(c(2, 128, dtype=b), None, None, c(256, 2, dtype=u), c(256, 1), None, None, Z=c(2, 256, dtype=b))
    with pytest.raises(ValueError, match="sft must have shape"):
        dg.dg_transpose_fp8(c(2, 128, dtype=u), c(2, 1), c(128, 128, dtype=u), c(128, 2))


@pytest.mark.parametrize("name", ["relu", "gelu", "gelu_tanh", "silu", "none"])
def test_reference_slopes_are_the_activations_differences(name):
    z, h = torch.linspace(-7, 7, 280, dtype=torch.float64), 1e-5
    torch.testing.assert_close(B.slope(z, name), (B.act(z + h, name) - B.act(z - h, name)) / (2 * h), atol=1e-9, rtol=0)


def test_reference_norm_gradient_is_its_differences():
    g = torch.Generator().manual_seed(2)
    s, w, dy = (torch.randn(*n, generator=g, dtype=torch.float64) for n in ((3, 16), (16,), (3, 16)))
    dx, dw = B.rmsnorm_backward(dy, s, w, 0.01)
    loss = lambda s, w: float((B.rmsnorm(s, w, 0.01) * dy).sum())  # noqa: E731
    h = 1e-6
    for i in range(16):
        d = torch.zeros(16, dtype=torch.float64)
        d[i] = h
        assert abs((loss(s, w + d) - loss(s, w - d)) / (2 * h) - float(dw[i])) < 1e-8
        for t in range(3):
            d = torch.zeros_like(s)
            d[t, i] = h
            assert abs((loss(s + d, w) - loss(s - d, w)) / (2 * h) - float(dx[t, i])) < 1e-8


@pytest.mark.parametrize("pow2", [False, True])
def test_reference_quantisation_is_the_input_recipe(pow2):
    from moe_grouped_gemm_tma_gb300 import inputs as I
    x = torch.randn(16, 384, generator=torch.Generator().manual_seed(3))
    x[4] *= 1e-7
    q, s = B.quantise(x.double(), pow2)
    want_q, want_s = I.quantize_1x128(x, pow2)
    assert torch.equal(s, want_s.double()) and torch.equal(q, want_q.view(torch.float8_e4m3fn).double())
    B.check_codes(want_q, want_s, x.double(), torch.zeros_like(x).double(), pow2)


def test_the_check_of_codes_sees_a_wrong_one():
    x = torch.randn(4, 256, generator=torch.Generator().manual_seed(5), dtype=torch.float64)
    q, s = B.quantise(x)
    q8 = q.float().to(torch.float8_e4m3fn)
    B.check_codes(q8, s, x, torch.zeros_like(x))
    bad = q8.view(torch.uint8).clone()
    bad[2, 77] += 1
    with pytest.raises(AssertionError):
        B.check_codes(bad, s, x, torch.zeros_like(x))
    with pytest.raises(AssertionError):
        B.check_codes(q8, s * (1 + 1e-5), x, torch.zeros_like(x))
