"""The gated activation's codes, bit for bit, where the values before the quantisation are known exactly: without an activation, and
with ReLU, every value is one product, rounded to FP32 (of BF16 numbers not even that). A code is e4m3 of the rounded quotient
by the scale then; two million values have some fifty whose product with the scale's rounded reciprocal has another one."""
import pytest
import torch

import moe_grouped_gemm_tma_gb300 as dg
from tests import between_ref as B
from tests.test_gpu_glu import DEV, E4M3, alloc, gen, make_z, run_backward

pytestmark = pytest.mark.gpu


def same(q, s, want, pow2=False):
    codes, scales = B.quantise(want, pow2)
    return torch.equal(s.double(), scales) and torch.equal(q.view(E4M3).double(), codes)


def rounded(a, b):
    """The product of float64 numbers of up to 24 bits, rounded to FP32."""
    return (a * b).float().double()


@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M,I", [(1024, 2048), (37, 384)])
def test_forward_codes_are_of_the_rounded_quotient(M, I, pow2, act):
    Z = make_z(M, I, seed=21)
    g, u = Z.double().split(I, 1)
    for keep in (False, True):
        q, sf, kept, ksf = alloc(M, I, keep)
        dg.dg_glu(Z, q, sf, kept, ksf, act=act, pow2=pow2)
        assert same(q, sf, B.act(g, act) * u, pow2)
        assert kept is None or same(kept, ksf, Z.double())


@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("M,I", [(1024, 2048), (301, 384)])
def test_backward_codes_are_of_the_rounded_quotient(M, I, kept, act):
    Z = make_z(M, I, seed=22)
    dH = (torch.randn(M, I, device=DEV, generator=gen(M)) * 0.05).bfloat16()
    if kept:
        q, sf, codes, ksf = alloc(M, I, True)
        dg.dg_glu(Z, q, sf, codes, ksf, act=act)
        out = run_backward(dH, kept=codes, ksf=ksf, act=act)
        g, u = B.values(codes, ksf).float().double().split(I, 1)
    else:
        out = run_backward(dH, Z=Z, act=act)
        g, u = Z.double().split(I, 1)
    a, d = B.act(g, act), dH.double()
    dz = torch.cat((rounded(d, u) * B.slope(g, act), rounded(d, a)), 1)
    assert same(*out["q"], dz)
    assert same(*out["qt"], B.columns(dz))
    assert same(*out["ht"], B.columns(rounded(a, u)))
