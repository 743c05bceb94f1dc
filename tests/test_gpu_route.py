"""The router and its gradient on the GPU against the 64-bit definition.

Tolerances. A score is one exponential of an argument of at most 100 or so and one quotient: the fast exponential is
within 2 + 1.2 |x| ulp, so a weight's relative error stays under 150 ulp = 1e-5 of it. Ids are compared exactly.
Gradients are differences of such numbers: 1e-5 of the largest |dw| in the row; BF16 adds half an ulp, 2^-9.
"""
import math

import numpy as np
import pytest
import torch

import moe_grouped_gemm_tma_gb300 as dg
from tests import operators_ref as R

pytestmark = pytest.mark.gpu


def make(T, E, seed, half, masked=0.0):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g) * 2
    if masked:
        l[:, torch.rand(E, generator=g) < masked] = -math.inf
    return l.to(torch.bfloat16) if half else l


def run(logits, k, bias=None, **kw):
    T = logits.shape[0]
    ids = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), math.nan, device="cuda")
    dg.dg_moe_route(logits.cuda(), ids, w, bias=None if bias is None else bias.cuda(), **kw)
    return ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)


def check(logits, k, bias=None, scoring="softmax", renormalize=True, scale=1.0):
    ids, w = run(logits, k, bias, scoring=scoring, renormalize=renormalize, scale=scale)
    want_ids, want = R.route(logits.double().numpy(), k, scoring, renormalize, scale, None if bias is None else bias.numpy())
    np.testing.assert_array_equal(ids, want_ids)
    assert (np.abs(w - want) <= 1e-5 * np.abs(want) + 1e-30).all()


@pytest.mark.parametrize("E", [1, 3, 31, 32, 33, 64, 100, 128, 200, 256, 257, 512, 777, 1024])
@pytest.mark.parametrize("half", [False, True])
def test_every_width(E, half):
    for scoring in ("softmax", "sigmoid"):
        for renorm in (False, True):
            check(make(37, E, E, half), min(E, 8), scoring=scoring, renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("T,E,k", [(1, 64, 6), (1, 8, 8), (5, 256, 32), (300, 40, 1), (9, 32, 32)])
def test_rows_and_selections(T, E, k):
    check(make(T, E, T + E, False), k)


@pytest.mark.parametrize("half", [False, True])
def test_bias_moves_the_selection_and_not_the_weights(half):
    logits = make(200, 160, 3, half)
    # on a grid far coarser than an FP32 sigmoid's rounding, so that no two sums are that close
    bias = torch.round(torch.randn(160, generator=torch.Generator().manual_seed(4)) * 64) / 64
    sig = 1 / (1 + np.exp(-logits.double().numpy()))
    total = sig + bias.double().numpy()
    gaps = np.diff(np.sort(total, axis=1), axis=1)
    rows = (gaps.min(1) > 1e-6) | half            # FP32 rows with a closer pair are not a test of anything
    logits = logits[torch.from_numpy(np.flatnonzero(rows))]
    check(logits, 8, bias, scoring="sigmoid", scale=2.5)


def test_equal_values_take_the_lower_expert():
    # whole rows of ties (more candidates than lanes), ties across lanes, and both zeros
    l = torch.zeros(6, 300)
    l[1, ::2] = 1.0
    l[2, 150:] = -0.0
    l[3, [7, 8, 200, 299]] = 5.0
    l[4] = -3.0
    l[5, 290:] = torch.finfo(torch.float32).min
    for k in (1, 8, 32):
        check(l, k, renormalize=False)
        check(l.to(torch.bfloat16), k)


@pytest.mark.parametrize("T", [1001, 8195])
@pytest.mark.parametrize("E,k", [(2, 1), (7, 7), (8, 2), (9, 3), (16, 16), (17, 4)])
def test_few_experts_and_many_rows(T, E, k):
    logits = make(T, E, T + E, False)
    logits[::5, : E // 2] = -math.inf
    logits[3], logits[4] = -math.inf, math.nan
    logits[5, 0] = math.inf
    logits[7:40] = torch.round(logits[7:40])                 # ties
    for scoring in ("softmax", "sigmoid"):
        for renorm in (False, True):
            check(logits, k, scoring=scoring, renormalize=renorm, scale=1.5)
            ids, _ = R.route(logits[:200].double().numpy(), k, scoring, renorm, 1.0)
            # the whole gradient, with the last row of the forward pass's rows among them
            every = np.concatenate([ids] * (T // 200 + 1))[:T]
            src = torch.cat([logits[:200]] * (T // 200 + 1))[:T].contiguous()
            dw = torch.randn(T, k, generator=torch.Generator().manual_seed(k))
            out = torch.full((T, E), math.nan, device="cuda")
            dg.dg_moe_route_backward(src.cuda(), torch.from_numpy(every).int().cuda(), dw.cuda(), out, scoring=scoring,
                                     renormalize=renorm, scale=1.5)
            want = R.route_backward(src.double().numpy(), every, dw.double().numpy(), scoring, renorm, 1.5)
            bound = 1e-5 * 1.5 * np.abs(dw.numpy()).max(1, keepdims=True) * max(1, k)
            assert (np.abs(out.cpu().double().numpy() - want) <= bound).all()
    bias = torch.round(torch.randn(E, generator=torch.Generator().manual_seed(4)) * 64) / 64
    check(torch.round(logits), k, bias, scoring="sigmoid")


@pytest.mark.parametrize("T,E", [(8195, 7), (8195, 14), (9, 14), (9, 32), (9, 48), (9, 256), (9, 301)])
def test_bias_that_is_not_finite(T, E):
    # a NaN or -inf of the bias takes its expert out of the selection, and no other; +inf puts it first
    bias = torch.zeros(E)
    bias[0], bias[3], bias[E - 1], bias[E // 2] = math.nan, -math.inf, math.nan, math.inf
    check(torch.round(make(T, E, E, False) * 4) / 4, min(E, 6), bias, scoring="sigmoid")


@pytest.mark.parametrize("E", [48, 256, 301, 510, 1024])
@pytest.mark.parametrize("levels", [2, 40])
def test_ties_in_every_layout(E, levels):
    # few distinct logits; with a bias the sums of equal pairs are equal too
    g = torch.Generator().manual_seed(E + levels)
    l = torch.randint(0, levels, (40, E), generator=g).float() / 8
    check(l, 8)
    check(l.to(torch.bfloat16), 8, scoring="sigmoid")
    check(l, 8, torch.full((E,), 0.25), scoring="sigmoid")


@pytest.mark.parametrize("half", [False, True])
def test_masked_experts_and_empty_rows(half):
    l = make(8, 70, 5, half)
    l[0] = -math.inf                              # nothing to select
    l[1, 3:] = -math.inf                          # fewer than k
    l[2] = torch.finfo(l.dtype).min               # the type's lowest value is a value
    l[3, :40] = torch.finfo(l.dtype).min
    l[4, 10] = math.inf
    l[5, 10] = l[5, 60] = math.inf
    l[6, ::3] = math.nan
    l[7] = math.nan
    for scoring in ("softmax", "sigmoid"):
        for renorm in (False, True):
            check(l, 6, scoring=scoring, renormalize=renorm)


def test_scores_that_vanish_give_no_weight():
    ids, w = run(torch.full((2, 16), -1e30), 4, scoring="sigmoid")
    assert (ids == np.arange(4)).all() and (w == 0).all()


def test_rows_off_the_vector_alignment():
    base = torch.randn(4 * 64 + 1, generator=torch.Generator().manual_seed(9)).cuda()
    logits = base[1:].view(4, 64)
    ids = torch.empty(4, 5, dtype=torch.int32, device="cuda")
    w = torch.empty(4, 5, device="cuda")
    dg.dg_moe_route(logits, ids, w)
    want_ids, want = R.route(logits.double().cpu().numpy(), 5, "softmax", True, 1.0)
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    np.testing.assert_allclose(w.cpu().numpy(), want, rtol=1e-5)
    out = torch.empty(4 * 64 + 1, device="cuda")[1:].view(4, 64)
    dw = torch.ones(4, 5, device="cuda")
    dg.dg_moe_route_backward(logits, ids, dw, out, renormalize=False)
    want = R.route_backward(logits.double().cpu().numpy(), want_ids, np.ones((4, 5)), "softmax", False, 1.0)
    assert np.abs(out.cpu().numpy() - want).max() <= 1e-5


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("E,k", [(5, 2), (64, 6), (130, 8), (256, 8), (600, 32)])
def test_gradient_against_the_formula(scoring, renorm, half, E, k):
    logits = make(21, E, E + k, half, masked=0.2)
    logits[0] = -math.inf
    ids, _ = R.route(logits.double().numpy(), k, scoring, renorm, 1.0)
    dw = torch.randn(21, k, generator=torch.Generator().manual_seed(1))
    out = torch.full_like(logits, math.nan).cuda()
    dg.dg_moe_route_backward(logits.cuda(), torch.from_numpy(ids).int().cuda(), dw.cuda(), out, scoring=scoring, renormalize=renorm, scale=1.5)
    want = R.route_backward(logits.double().numpy(), ids, dw.double().numpy(), scoring, renorm, 1.5)
    bound = 1e-5 * 1.5 * np.abs(dw.numpy()).max(1, keepdims=True) + (np.abs(want) * 2.0 ** -8 if half else 0)
    assert (np.abs(out.double().cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(scoring, renorm):
    # central differences of the 64-bit weights: their own error is h^2 times a third derivative of at most 1
    logits = make(4, 11, 2, False)
    l = logits.double().numpy()
    ids, _ = R.route(l, 3, scoring, renorm, 1.0)
    dw = torch.randn(4, 3, generator=torch.Generator().manual_seed(1))
    out = torch.empty(4, 11, device="cuda")
    dg.dg_moe_route_backward(logits.cuda(), torch.from_numpy(ids).int().cuda(), dw.cuda(), out, scoring=scoring, renormalize=renorm)
    h = 1e-4
    for e in range(11):
        up, down = l.copy(), l.copy()
        up[:, e] += h
        down[:, e] -= h
        diff = (R.route_weights(up, ids, scoring, renorm, 1.0) - R.route_weights(down, ids, scoring, renorm, 1.0)) / (2 * h)
        want = (diff * dw.double().numpy()).sum(1)
        assert np.abs(out[:, e].double().cpu().numpy() - want).max() <= 1e-5 * 3 * dw.abs().max().item()


def test_gradient_of_an_expert_named_twice_adds_up():
    logits = make(2, 20, 8, False)
    ids = torch.tensor([[3, 3, 5], [7, -1, 7]], dtype=torch.int32)
    dw = torch.tensor([[1.0, 2.0, -1.0], [0.5, 9.0, 0.25]])
    for scoring in ("softmax", "sigmoid"):
        out = torch.empty(2, 20, device="cuda")
        dg.dg_moe_route_backward(logits.cuda(), ids.cuda(), dw.cuda(), out, scoring=scoring, renormalize=False)
        want = R.route_backward(logits.double().numpy(), ids.numpy(), dw.double().numpy(), scoring, False, 1.0)
        assert np.abs(out.double().cpu().numpy() - want).max() <= 3e-5


def test_on_a_stream_of_its_own():
    logits = make(64, 64, 6, False).cuda()
    ids = torch.empty(64, 4, dtype=torch.int32, device="cuda")
    w = torch.empty(64, 4, device="cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    dg.dg_moe_route(logits, ids, w, stream=st)
    st.synchronize()
    want, _ = R.route(logits.double().cpu().numpy(), 4, "softmax", True, 1.0)
    np.testing.assert_array_equal(ids.cpu().numpy(), want)
