"""The router with up to 32 experts over so many rows that its warps take more than one each (16 warps' worth a CTA and
SM, two rounds of CTAs), with a ragged last turn, against the 64-bit definition over whole tensors.

Tolerances: those of test_gpu_route.py.
"""
import math

import pytest
import torch

import moe_grouped_gemm_tma_gb300 as dg

pytestmark = pytest.mark.gpu

F32_TOP = torch.finfo(torch.float32).max


def scores_of(logits, scoring):
    """float64 scores, 0 where an expert cannot be selected, and the logits with those at -inf."""
    l = torch.where(torch.isnan(logits), -math.inf, logits.double().clamp_max(F32_TOP))
    if scoring == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True).clamp_min(-F32_TOP))
        return e / e.sum(1, keepdim=True).clamp_min(1e-300), l
    return torch.where(l > -math.inf, torch.sigmoid(l), 0.0), l


def forward(logits, k, scoring, renorm, scale, bias):
    score, l = scores_of(logits, scoring)
    pick = l
    if bias is not None:
        pick = torch.where(l > -math.inf, (score.float() + bias).double(), -math.inf)
    top, at = torch.sort(pick, dim=1, descending=True, stable=True)
    open_ = top[:, :k] > -math.inf
    w = torch.where(open_, score.gather(1, at[:, :k]), 0.0)
    if renorm:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return torch.where(open_, at[:, :k], -1), w * scale


def backward(logits, ids, dw, scoring, renorm, scale):
    score, _ = scores_of(logits, scoring)
    open_ = ids >= 0
    at = ids.clamp_min(0)
    p = torch.where(open_, score.gather(1, at), 0.0)
    dw = torch.where(open_, dw.double() * scale, 0.0)
    total = p.sum(1, keepdim=True)
    if renorm:
        dp = torch.where(total > 0, dw / total - (dw * p).sum(1, keepdim=True) / total ** 2, 0.0)
    else:
        dp = dw
    d = torch.zeros_like(score).scatter_add_(1, at, torch.where(open_, dp, 0.0))
    return score * (d - (d * score).sum(1, keepdim=True)) if scoring == "softmax" else d * score * (1 - score)


@pytest.mark.parametrize("T", [20011, 40003])
@pytest.mark.parametrize("E,k", [(17, 4), (24, 3), (32, 8)])
@pytest.mark.parametrize("half", [False, True])
def test_warps_that_take_several_rows(T, E, k, half):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert T > 16 * sms * 8                                  # the rows of one turn of all warps
    g = torch.Generator(device="cuda").manual_seed(T + E)
    logits = torch.randn(T, E, device="cuda", generator=g) * 2
    logits[::7, : E // 2] = -math.inf
    logits[T - 40:T - 20] = torch.round(logits[T - 40:T - 20])   # ties in the last turn
    logits[T - 3], logits[T - 2, 1:], logits[5], logits[T - 50, 0] = -math.inf, -math.inf, math.nan, math.inf
    logits = logits.to(torch.bfloat16) if half else logits
    dw = torch.randn(T, k, device="cuda", generator=g)
    # on a grid far coarser than a sigmoid's rounding, and logits for it on one where no two sums are that close but equal
    bias = torch.round(torch.randn(E, device="cuda", generator=g) * 64) / 64
    coarse = torch.round(logits.float())
    for scoring in ("softmax", "sigmoid"):
        for renorm in (False, True):
            for l, b in ((logits, None),) + (((coarse, bias),) if scoring == "sigmoid" else ()):
                ids = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
                w = torch.full((T, k), math.nan, device="cuda")
                dg.dg_moe_route(l, ids, w, bias=b, scoring=scoring, renormalize=renorm, scale=1.5)
                want_ids, want = forward(l.float(), k, scoring, renorm, 1.5, b)
                assert torch.equal(ids.long(), want_ids)
                assert ((w.double() - want).abs() <= 1e-5 * want.abs() + 1e-30).all()
            out = torch.full_like(logits, math.nan)
            ids = forward(logits.float(), k, scoring, renorm, 1.5, None)[0]
            dg.dg_moe_route_backward(logits, ids.int(), dw, out, scoring=scoring, renormalize=renorm, scale=1.5)
            want = backward(logits.float(), ids, dw, scoring, renorm, 1.5)
            bound = 1e-5 * 1.5 * dw.abs().amax(1, keepdim=True) + (want.abs() * 2.0 ** -8 if half else 0)
            assert ((out.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("E", [5, 20, 64, 200, 301, 1024])
@pytest.mark.parametrize("T", [9, 6150])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_of_experts_named_more_than_once(E, T, scoring, renorm):
    # every kernel's way of gathering the slots of an expert; the weights are functions of the slots, each of which
    # names an expert, so an expert named n times has n weights and counts n times in their sum
    k = 5
    g = torch.Generator(device="cuda").manual_seed(E + T)
    logits = torch.randn(T, E, device="cuda", generator=g) * 2
    ids = torch.randint(0, E, (T, k), device="cuda", generator=g)
    ids[:, 3] = ids[:, 0]
    ids[::2, 4] = ids[::2, 0]
    ids[::3, 1] = -1
    dw = torch.randn(T, k, device="cuda", generator=g)
    out = torch.full_like(logits, math.nan)
    dg.dg_moe_route_backward(logits, ids.int(), dw, out, scoring=scoring, renormalize=renorm, scale=1.5)
    want = backward(logits, ids, dw, scoring, renorm, 1.5)
    assert ((out.double() - want).abs() <= 1e-5 * 1.5 * dw.abs().amax(1, keepdim=True) * k).all()
