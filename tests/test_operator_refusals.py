"""What the operators around the products refuse, before any CUDA work (no GPU needed), and their definitions' own
checks (gradients against differences in 64 bits)."""
import ctypes

import numpy as np
import pytest
import torch

import moe_grouped_gemm_tma_gb300 as dg
from tests import operators_ref as R


def _p(addr):
    return ctypes.c_void_p(addr)


OK, ODD8, ODD2, ODD1 = _p(0x10000), _p(0x10008), _p(0x10002), _p(0x10001)


def test_gemm_epilogue_refusals():
    f = dg.load().dg_gemm_fp8_nt_epilogue          # A sfa B sfb D bias act residual Z M N K
    call = lambda A=OK, sfa=OK, B=OK, sfb=OK, D=OK, bias=OK, act=1, res=OK, Z=OK, M=4, N=8, K=128: f(A, sfa, B, sfb, D, bias, act, res, Z, M, N, K, None)  # noqa: E731
    assert call(act=-1) == 1 and call(act=5) == 1
    assert call(M=-1) == 1 and call(M=0) == 0 and call(N=0) == 0
    assert call(K=0) == 2 and call(K=100) == 2 and call(N=12) == 2
    assert call(D=None) == 1
    assert call(D=ODD8) == 3 and call(bias=ODD2) == 3 and call(res=ODD8) == 3 and call(Z=ODD8) == 3


def test_epilogue_backward_refusals():
    L = dg.load()
    f = L.dg_epilogue_backward                     # dD Z act q sf qt sft dbias ws bytes M N
    call = lambda dD=OK, Z=OK, act=4, q=OK, sf=OK, qt=OK, sft=OK, dbias=OK, ws=OK, size=1 << 30, M=4, N=128: f(dD, Z, act, q, sf, qt, sft, dbias, ws, size, M, N, None)  # noqa: E731
    assert call(M=-1) == 1 and call(act=9) == 1 and call(N=0) == 0
    assert call(q=None, sf=None, qt=None, sft=None, dbias=None) == 0
    assert call(N=120) == 2
    assert call(sf=None) == 1 and call(q=None) == 1 and call(sft=None) == 1 and call(qt=None) == 1
    assert call(dD=None) == 1 and call(Z=None) == 1
    assert call(ws=None) == 1 and call(size=16) == 1
    assert call(dD=ODD8) == 3 and call(Z=ODD8) == 3 and call(q=ODD8) == 3 and call(qt=ODD8) == 3 and call(sf=ODD2) == 3
    assert call(dbias=ODD2) == 3 and call(ws=ODD8) == 3
    assert L.dg_epilogue_backward_workspace(0, 128) == 0
    assert L.dg_epilogue_backward_workspace(129, 256) >= 2 * 256 * 4 + 2 * 4


def test_route_refusals():
    L = dg.load()
    f = L.dg_moe_route                             # logits type bias ids weights T E k scoring renorm scale
    call = lambda l=OK, t=1, b=None, i=OK, w=OK, T=2, E=8, k=2, s=0: f(l, t, b, i, w, T, E, k, s, 1, 1.0, None)  # noqa: E731
    assert call(t=2) == 1 and call(s=2) == 1 and call(T=-1) == 1 and call(k=-1) == 1
    assert call(E=1025) == 2 and call(E=64, k=33) == 2 and call(E=4, k=5) == 2
    assert call(T=0) == 0 and call(k=0) == 0
    assert call(b=OK) == 1                         # a bias moves sigmoid scores only
    assert call(l=None) == 1 and call(i=None) == 1 and call(w=None) == 1
    assert call(l=ODD2) == 3 and call(l=ODD1, t=0) == 3 and call(i=ODD2) == 3 and call(w=ODD2) == 3 and call(b=ODD2, s=1) == 3
    g = L.dg_moe_route_backward                    # logits type ids dweights dlogits T E k scoring renorm scale
    back = lambda l=OK, t=1, i=OK, w=OK, d=OK, T=2, E=8, k=2, s=0: g(l, t, i, w, d, T, E, k, s, 1, 1.0, None)  # noqa: E731
    assert back(t=-1) == 1 and back(E=1025) == 2 and back(k=9) == 2 and back(T=0) == 0
    assert back(l=None) == 1 and back(d=None) == 1 and back(i=None) == 1 and back(w=None) == 1
    assert back(d=ODD2) == 3 and back(w=ODD2) == 3


def test_moe_layer_refusals():
    L = dg.load()
    f = L.dg_moe_layer                             # x ids w W13 s13 W2 s2 res out ws bytes T k E H I act
    size = L.dg_moe_layer_workspace(4, 2, 4, 256, 128)
    assert size > 0
    base = dict(x=OK, ids=OK, w=OK, W13=OK, s13=OK, W2=OK, s2=OK, res=None, out=OK, ws=OK, size=size, T=4, k=2, E=4, H=256, I=128, act=4)
    call = lambda **kw: f(*{**base, **kw}.values(), None)  # noqa: E731
    assert call(T=0) == 0
    assert call(T=-1) == 1 and call(act=5) == 1
    assert call(T=65) == 2 and call(k=0) == 2 and call(T=64, k=17) == 2 and call(E=1025) == 2 and call(E=0) == 2
    assert call(H=200) == 2 and call(I=64) == 2 and call(H=0) == 2
    for name in ("x", "ids", "w", "W13", "s13", "W2", "s2", "out", "ws"):
        assert call(**{name: None}) == 1, name
    assert call(size=size - 1) == 1
    for name in ("x", "W13", "W2", "out", "res"):
        assert call(**{name: ODD8}) == 3, name
    for name in ("ids", "w", "s13", "s2"):
        assert call(**{name: ODD2}) == 3, name
    assert call(ws=_p(0x10010)) == 3
    assert L.dg_moe_layer_workspace(65, 2, 4, 256, 128) == -1 and L.dg_moe_layer_workspace(4, 2, 4, 200, 128) == -1
    assert L.dg_moe_layer_workspace(0, 2, 4, 256, 128) == 0


def test_binding_refuses_host_tensors_types_and_shapes():
    b, f, i, u = torch.bfloat16, torch.float32, torch.int32, torch.uint8
    e = lambda *s, dtype=f: torch.empty(*s, dtype=dtype)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA tensor"):
        dg.dg_moe_route(e(2, 8), e(2, 2, dtype=i), e(2, 2))
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        dg.dg_moe_route(e(2, 8, dtype=torch.float16), e(2, 2, dtype=i), e(2, 2))
    with pytest.raises(ValueError, match="CUDA tensor"):
        dg.dg_moe_route_backward(e(2, 8), e(2, 2, dtype=i), e(2, 2), e(2, 8))
    with pytest.raises(TypeError, match="x must be"):
        dg.dg_moe_layer(e(2, 128), e(2, 1, dtype=i), e(2, 1), e(1, 256, 128, dtype=u).cuda() if torch.cuda.is_available() else _Cuda(e(1, 256, 128, dtype=u)),
                        e(1, 2, 1), _Cuda(e(1, 128, 128, dtype=u)), e(1, 1, 1), e(2, 128, dtype=b), None)
    with pytest.raises(TypeError, match="dD must be"):
        dg.dg_epilogue_backward(e(2, 128), None, None, None, None, None, None)
    with pytest.raises(ValueError, match="shape"):
        dg.dg_epilogue_backward(_Cuda(e(2, 128, dtype=b)), e(3, 128, dtype=b), None, None, None, None, None)
    with pytest.raises(TypeError, match="e4m3 codes"):
        dg.dg_gemm_fp8_nt_epilogue(e(2, 128), e(2, 1), e(8, 128, dtype=u), e(1, 1), e(2, 8, dtype=b))
    with pytest.raises(dg.DGError):
        dg.moe_layer_workspace(65, 1, 1, 128, 128)
    with pytest.raises(ValueError, match="act must be one of"):
        dg._choice(dg.ACTIVATIONS, "swish", "act")


class _Cuda:
    """A host tensor that says it is on the GPU: it gets past the device check to the one under test."""

    def __init__(self, t):
        self._t, self.is_cuda = t, True

    def __getattr__(self, name):
        return getattr(self._t, name)


@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu", "none"])
def test_reference_slopes_are_the_activations_differences(name):
    z, h = np.linspace(-7, 7, 281), 1e-5
    np.testing.assert_allclose(R.act_slope(z, name), (R.act(z + h, name) - R.act(z - h, name)) / (2 * h), atol=1e-9)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_reference_route_gradient_is_its_differences(scoring, renorm):
    rng = np.random.default_rng(1)
    l, dw, h = rng.normal(size=(3, 9)), rng.normal(size=(3, 4)), 1e-5
    l[0, 2] = -np.inf
    ids, w = R.route(l, 4, scoring, renorm, 1.3)
    np.testing.assert_allclose(w, R.route_weights(l, ids, scoring, renorm, 1.3), atol=1e-14)
    got = R.route_backward(l, ids, dw, scoring, renorm, 1.3)
    for e in range(9):
        up, down = l.copy(), l.copy()
        up[:, e] += h
        down[:, e] -= h
        diff = (R.route_weights(up, ids, scoring, renorm, 1.3) - R.route_weights(down, ids, scoring, renorm, 1.3)) / (2 * h)
        np.testing.assert_allclose(got[:, e], (diff * dw).sum(1), atol=1e-9)


def test_reference_quantisation_is_the_input_recipe():
    from moe_grouped_gemm_tma_gb300 import inputs as I
    x = torch.randn(16, 384, generator=torch.Generator().manual_seed(3))
    x[4] *= 1e-7
    q, s = R.quantise(x.double().numpy())
    want_q, want_s = I.quantize_1x128(x)
    np.testing.assert_array_equal(s, want_s.double().numpy())
    np.testing.assert_array_equal(q, want_q.view(torch.float8_e4m3fn).double().numpy())
