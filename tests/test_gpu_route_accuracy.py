"""The router's softmax where its scores span 35 orders of magnitude, against 64 bits, in every kernel of it.

Logits are multiples of 1/8, so their distance from the largest is exact. Tolerances, in units of 2^-24: an exponential
of FP32 has 2 ulp (4), a sum over up to 32 values a lane and five exchanges 36 additions, the reciprocal 1, the products
by it and by the scale 2, none of them as large as that for most elements: 43. A gradient of an expert that was not
selected is minus its score times the weighted sum of the weights' gradients, here of one sign: one more exponential and
as many products and additions, 5 each: 57.
"""
import pytest
import torch

import moe_grouped_gemm_tma_gb300 as dg

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -24


def inputs(T, E, k):
    g = torch.Generator(device="cuda").manual_seed(E)
    l = -torch.randint(0, 640, (T, E), device="cuda", generator=g).float() / 8
    l[:, 0] = 0.0
    return l, torch.rand(T, k, device="cuda", generator=g) + 0.5


@pytest.mark.parametrize("T,E", [(6150, 7), (6150, 13), (300, 7), (300, 24), (300, 32), (300, 64), (300, 100), (300, 200), (300, 256), (300, 301), (300, 1024)])
@pytest.mark.parametrize("renorm", [False, True])
def test_small_scores(T, E, renorm):
    k = min(E - 1, 6)
    l, dw = inputs(T, E, k)
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    dg.dg_moe_route(l, ids, w, renormalize=renorm, scale=1.5)
    p = torch.softmax(l.double(), 1)
    want = p.gather(1, ids.long())
    want = 1.5 * (want / want.sum(1, keepdim=True) if renorm else want)
    assert ((w.double() - want).abs() <= 43 * UNIT * want).all()
    if not renorm:
        out = torch.empty_like(l)
        dg.dg_moe_route_backward(l, ids, dw, out, renormalize=False, scale=1.5)
        got = out.double().scatter(1, ids.long(), 0.0)
        want = (-p * (want * dw.double()).sum(1, keepdim=True)).scatter(1, ids.long(), 0.0)
        assert ((got - want).abs() <= 57 * UNIT * want.abs()).all()
