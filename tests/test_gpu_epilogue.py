"""The FP8 product with an epilogue, and its backward pass, on the GPU against 64 bits.

Tolerances. Product: the sums' own error is that of dg_gemm_fp8_nt (1e-2 of the rms, as its tests take it), the
activations have slopes up to 1.13, and the two outputs are rounded to BF16 once: |err| <= 1e-2 |want| + 1.2e-2 rms(z).
Backward: dZ is within 1e-5 of its magnitude (a fast exponential and reciprocal, a product); a scale is the largest of
128 such numbers; a code may be the neighbour of the definition's only where the quotient is within that of a midpoint,
which takes in about 2e-5 / (1/16) of all values. Sums of rows: 1e-5 of the sum of the magnitudes.
"""
import math

import numpy as np
import pytest
import torch

import moe_grouped_gemm_tma_gb300 as dg
from moe_grouped_gemm_tma_gb300 import inputs as I
from oracle import oracle as O
from tests import operators_ref as R
from tests.gpu_util import bits_to_f64, bf16_bits, check_bf16, dev, sentinel_bf16

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def product(c):
    return R.row_values(c.A, c.sfa) @ R.block_values(c.B, c.sfb).T


def extras(M, N, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(N, generator=g) * 5, (torch.randn(M, N, generator=g) * 20).to(torch.bfloat16)


def run(c, act, bias, res, keep, inplace=False):
    D = dev(res) if inplace else sentinel_bf16(c.M, c.N)
    Z = sentinel_bf16(c.M, c.N) if keep else None
    r = None if res is None else (D if inplace else dev(res))
    dg.dg_gemm_fp8_nt_epilogue(dev(c.A), dev(c.sfa), dev(c.B), dev(c.sfb), D, bias=None if bias is None else dev(bias), act=act,
                               residual=r, Z=Z)
    assert dg.dg_device_status() == 0
    return D, Z


def check(c, act, bias, res, keep, inplace=False):
    D, Z = run(c, act, bias, res, keep, inplace)
    z = product(c)
    if bias is not None:
        z = z + bias.double().numpy()
    want = R.act(z, act)
    if res is not None:
        want = want + res.double().numpy()
    rms = math.sqrt(np.mean(z * z))
    got = bits_to_f64(bf16_bits(D))
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= 1e-2 * np.abs(want) + 1.2e-2 * rms).all()
    if keep:
        got = bits_to_f64(bf16_bits(Z))
        assert (np.abs(got - z) <= 1e-2 * np.abs(z) + 1e-2 * rms).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(1, 256, 128), (64, 2112, 1024), (200, 1000, 768), (300, 136, 384), (129, 4096, 256)])
def test_shapes_and_activations(M, N, K, act):
    c = I.make_normal(I.seed_for(2, M + N + K), M, N, K)
    bias, res = extras(M, N, M)
    check(c, act, bias, res, True)


@pytest.mark.parametrize("use_bias", [False, True])
@pytest.mark.parametrize("use_res", [False, True])
@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("M", [30, 260])
def test_every_combination(use_bias, use_res, keep, M):
    c = I.make_normal(I.seed_for(2, 5), M, 520, 512)
    bias, res = extras(M, 520, 1)
    check(c, "silu", bias if use_bias else None, res if use_res else None, keep)


@pytest.mark.parametrize("bn,pair", [(64, 1), (128, 1), (192, 1)])
@pytest.mark.parametrize("M", [40, 200, 520])
def test_every_tile_shape(bn, pair, M, tune):
    # ragged rows and columns; 1000 is a multiple of 8 and not of 16 (narrow stores of Z)
    tune(bn=bn, pair=pair, split=1)
    c = I.make_normal(I.seed_for(2, 900 + bn + M), M, 1000, 512)
    bias, res = extras(M, 1000, bn)
    check(c, "gelu_tanh", bias, res, True)


@pytest.mark.parametrize("bn", [64, 128, 192])
def test_many_tiles_a_cta(bn, tune):
    # several tiles a CTA: the residual's copies and the stores take turns in the staging
    tune(bn=bn)
    c = I.make_normal(I.seed_for(2, 40 + bn), 1500, 4128, 256)
    bias, res = extras(1500, 4128, bn)
    check(c, "relu", bias, res, False)
    check(c, "relu", bias, res, True, inplace=True)


@pytest.mark.parametrize("split", [2, 4, 8])
def test_split_k(split, tune):
    tune(split=split, swap=0)
    c = I.make_normal(I.seed_for(2, 700 + split), 100, 1000, 1408)
    bias, res = extras(100, 1000, split)
    check(c, "gelu", bias, res, True)


@pytest.mark.parametrize("split", [1, 4])
@pytest.mark.parametrize("M", [1, 20, 64])
def test_few_row_kernel(split, M, tune):
    tune(split=split, swap=1)
    c = I.make_normal(I.seed_for(2, 600 + split + M), M, 1000, 1408)
    bias, res = extras(M, 1000, split)
    check(c, "silu", bias, res, True)


def test_residual_in_place():
    for M in (16, 300):
        c = I.make_normal(I.seed_for(2, 8), M, 648, 256)
        bias, res = extras(M, 648, 3)
        check(c, "gelu", bias, res, False, inplace=True)


def test_without_an_epilogue_it_is_the_product():
    c = I.make_normal(I.seed_for(2, 9), 260, 520, 512)
    D, _ = run(c, "none", None, None, False)
    check_bf16(bf16_bits(D), O.gemm_fp8_nt(c.A, c.sfa, c.B, c.sfb), "plain")


def test_nothing_past_the_last_row_is_written():
    c = I.make_normal(I.seed_for(2, 10), 100, 264, 256)
    bias, res = extras(100, 264, 3)
    D, Z = sentinel_bf16(164, 264), sentinel_bf16(164, 264)
    dg.dg_gemm_fp8_nt_epilogue(dev(c.A), dev(c.sfa), dev(c.B), dev(c.sfb), D[:100], bias=dev(bias), act="silu", residual=dev(res), Z=Z[:100])
    assert dg.dg_device_status() == 0
    for t in (D, Z):
        assert (bf16_bits(t[100:]) == I.BF16_SENTINEL).all()


def test_special_values_pass_through():
    # (the product is zero: zero codes) bias carries the infinities and NaN to the activation
    M, N = 4, 16
    A = torch.zeros(M, 128, dtype=torch.uint8)
    B = torch.zeros(N, 128, dtype=torch.uint8)
    ones = torch.ones(M, 1), torch.ones(1, 1)
    bias = torch.zeros(N)
    bias[:6] = torch.tensor([math.inf, math.nan, 300.0, -300.0, 88.5, -88.5])
    for act in ACTS:
        D = sentinel_bf16(M, N)
        dg.dg_gemm_fp8_nt_epilogue(dev(A), dev(ones[0]), dev(B), dev(ones[1]), D, bias=dev(bias), act=act)
        got = D.double().cpu().numpy()
        want = R.act(bias.double().numpy(), act)
        assert np.isinf(got[:, 0]).all() and np.isnan(got[:, 1]).all()
        np.testing.assert_allclose(got[:, 2:], np.tile(want[2:], (M, 1)), rtol=2.0 ** -8, atol=1e-6)


# ------------------------------------------------------------------------------------------------ backward
def backward_inputs(M, N, seed, act):
    g = torch.Generator().manual_seed(seed)
    dD = (torch.randn(M, N, generator=g) * 0.02).to(torch.bfloat16)
    Z = None if act == "none" else (torch.randn(M, N, generator=g) * 1.5).to(torch.bfloat16)
    return dD, Z


def run_backward(dD, Z, act, want=("q", "qt", "dbias"), ws=None):
    M, N = dD.shape
    Mp = (M + 127) // 128 * 128
    e4, f = torch.float8_e4m3fn, torch.float32
    out = {"q": torch.full((M, N), 0xEE, dtype=torch.uint8, device="cuda").view(e4), "sf": torch.full((M, N // 128), -1.0, device="cuda"),
           "qt": torch.full((N, Mp), 0xEE, dtype=torch.uint8, device="cuda").view(e4), "sft": torch.full((N, Mp // 128), -1.0, device="cuda"),
           "dbias": torch.full((N,), math.nan, device="cuda")}
    pick = {"q": ("q", "sf"), "qt": ("qt", "sft"), "dbias": ("dbias",)}
    used = {n for w in want for n in pick[w]}
    if ws is None and "dbias" in want:
        ws = dg.epilogue_backward_workspace(M, N)
    dg.dg_epilogue_backward(dev(dD), None if Z is None else dev(Z), *(out[n] if n in used else None for n in ("q", "sf", "qt", "sft", "dbias")),
                            workspace=ws, act=act)
    assert dg.dg_device_status() == 0
    return {n: out[n].cpu() for n in used}


def check_codes(q, s, dz, what):
    """Codes and scales of 1x128 blocks against the definition on the exact dz [rows, n * 128]."""
    want_q, want_s = R.quantise(dz)
    got_q, got_s = q.double().numpy(), s.double().numpy()
    np.testing.assert_allclose(got_s, want_s, rtol=1e-5, err_msg=what)
    back, exact = R.values(got_q, got_s), np.asarray(dz)
    # half a step of e4m3, 2^-4 of the value or half the smallest step 2^-10 of the scale, and the errors above
    step = np.repeat(got_s, 128, axis=1).reshape(exact.shape)
    assert (np.abs(back - exact) <= (2.0 ** -4 + 2e-5) * np.abs(exact) + 2.0 ** -10 * step * 1.001).all(), what
    assert np.mean(got_q != want_q) <= 1e-3, what


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N", [(1, 128), (128, 256), (333, 384), (130, 1024), (700, 128)])
def test_backward(M, N, act):
    dD, Z = backward_inputs(M, N, M + N, act)
    out = run_backward(dD, Z, act)
    dz = dD.double().numpy() * (1.0 if Z is None else R.act_slope(Z.double().numpy(), act))
    check_codes(out["q"], out["sf"], dz, "rows")
    padded = np.concatenate([dz, np.zeros((-M % 128, N))])
    check_codes(out["qt"], out["sft"], padded.T, "columns")
    if M % 128:
        assert (out["qt"][:, M:].float() == 0).all()
    assert (np.abs(out["dbias"].double().numpy() - dz.sum(0)) <= 1e-5 * np.abs(dz).sum(0) + 1e-12).all()


def test_backward_workspace_serves_smaller_sizes():
    # one tile, several of a strip in one round, and more tiles than run at once, in turn on one workspace
    ws = dg.epilogue_backward_workspace(700, 17024)
    for M, N in [(300, 128), (256, 17024), (3, 256), (700, 17024), (2500, 2048), (300, 128), (256, 17024)]:
        dD, Z = backward_inputs(M, N, M + N, "relu")
        out = run_backward(dD, Z, "relu", ("dbias",), ws)
        dz = dD.double().numpy() * R.act_slope(Z.double().numpy(), "relu")
        assert (np.abs(out["dbias"].double().numpy() - dz.sum(0)) <= 1e-5 * np.abs(dz).sum(0) + 1e-12).all(), (M, N)


@pytest.mark.parametrize("want", [("q",), ("qt",), ("dbias",), ("q", "dbias"), ("qt", "dbias"), ("q", "qt")])
def test_backward_parts(want):
    # each output alone is the same, and what is not asked for is not needed
    dD, Z = backward_inputs(300, 256, 4, "silu")
    full, part = run_backward(dD, Z, "silu"), run_backward(dD, Z, "silu", want)
    for n, t in part.items():
        assert torch.equal(t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t, full[n].view(torch.uint8) if t.dtype == torch.float8_e4m3fn else full[n]), n


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_backward_against_differences(act):
    # dbias with dD = 1 at one element of a column is act'(z): differences of the 64-bit activation, whose own
    # error is h^2 / 6 times its third derivative (under 2), against FP32 arithmetic
    N = 256
    z = torch.linspace(-6, 6, N).to(torch.bfloat16)
    z = torch.where(z.abs() < 0.02, torch.tensor(0.5, dtype=torch.bfloat16), z)      # relu has no slope at 0
    dD = torch.zeros(3, N, dtype=torch.bfloat16)
    dD[1] = 1.0
    got = run_backward(dD, z.expand(3, N).contiguous(), act, ("dbias",))["dbias"].double().numpy()
    x, h = z.double().numpy(), 1e-4
    want = (R.act(x + h, act) - R.act(x - h, act)) / (2 * h)
    assert np.abs(got - want).max() <= 1e-5


def test_backward_workspace_serves_again():
    ws = dg.epilogue_backward_workspace(700, 512)
    for M, N in ((700, 512), (130, 256), (700, 512), (1, 128)):
        dD, Z = backward_inputs(M, N, M, "silu")
        got = run_backward(dD, Z, "silu", ("dbias",), ws)["dbias"].double().numpy()
        dz = dD.double().numpy() * R.act_slope(Z.double().numpy(), "silu")
        assert (np.abs(got - dz.sum(0)) <= 1e-5 * np.abs(dz).sum(0)).all()


def test_backward_is_reproducible():
    dD, Z = backward_inputs(3000, 512, 1, "gelu")
    a, b = run_backward(dD, Z, "gelu"), run_backward(dD, Z, "gelu")
    for n in a:
        assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)), n


def test_backward_without_rows_zeroes_the_bias_gradient():
    dbias = torch.full((256,), 3.0, device="cuda")
    e = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    dg.dg_epilogue_backward(e, e, None, None, None, None, dbias, workspace=dg.epilogue_backward_workspace(1, 256), act="silu")
    assert (dbias == 0).all()


def test_backward_special_values():
    # a NaN spoils its own blocks, an infinity turns its block's finite values to zero; other blocks stay
    dD = torch.full((256, 256), 0.5, dtype=torch.bfloat16)
    dD[3, 5] = math.nan
    dD[140, 200] = math.inf
    out = run_backward(dD, None, "none")
    q, sf = out["q"].float(), out["sf"]
    assert torch.isnan(sf[3, 0]) and torch.isnan(q[3, :128]).all() and torch.isfinite(q[3, 128:]).all()
    assert torch.isinf(sf[140, 1]) and torch.isnan(q[140, 200]) and (q[140, 128:200] == 0).all()
    qt, sft = out["qt"].float(), out["sft"]
    assert torch.isnan(sft[5, 0]) and torch.isnan(qt[5, :128]).all() and torch.isfinite(qt[5, 128:]).all()
    assert torch.isinf(sft[200, 1]) and torch.isnan(qt[200, 140])
    assert torch.isnan(out["dbias"][5]) and torch.isinf(out["dbias"][200])
    assert int(torch.isfinite(sf).sum()) == sf.numel() - 2


def test_quantises_as_the_input_recipe():
    # with no activation it is the package's 1x128 recipe, bit for bit, small blocks (scale floor) included
    x = torch.randn(256, 512, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    x[7] *= 1e-6
    x[9] = 0
    out = run_backward(x, None, "none", ("q", "qt"))
    for q, s, m in ((out["q"], out["sf"], x.float()), (out["qt"], out["sft"], x.float().t().contiguous())):
        want_q, want_s = I.quantize_1x128(m)
        assert torch.equal(s, want_s)
        assert torch.equal(q.view(torch.uint8), want_q)


def test_training_step_of_a_layer_closes():
    # D = act(A B^T + bias): both products of the backward pass on the quantised dZ, against 64 bits on the same
    # quantised operands (which the codes' own tests hold to the definition)
    M, N, K = 256, 384, 256
    c = I.make_normal(I.seed_for(2, 12), M, N, K)
    bias, _ = extras(M, N, 1)
    _, Z = run(c, "silu", bias, None, True)
    dD = (torch.randn(M, N, generator=torch.Generator().manual_seed(2)) * 0.02).to(torch.bfloat16)
    out = run_backward(dD, Z.cpu(), "silu")
    dX = sentinel_bf16(M, K)
    dg.dg_gemm_fp8(out["q"].cuda(), out["sf"].cuda(), dev(c.B), dev(c.sfb.t()), dX, b_mn_major=True)
    want = R.row_values(out["q"], out["sf"]) @ R.block_values(c.B, c.sfb)
    got = dX.double().cpu().numpy()
    assert (np.abs(got - want) <= 1e-2 * np.abs(want) + 1e-2 * math.sqrt(np.mean(want ** 2))).all()
    x = torch.from_numpy(R.row_values(c.A, c.sfa)).to(torch.bfloat16)
    xt = run_backward(x, None, "none", ("qt",))
    dW = torch.zeros(N, K, device="cuda")
    dg.dg_wgrad_fp8_nt(out["qt"].cuda(), out["sft"].cuda(), xt["qt"].cuda(), xt["sft"].cuda(), dW, accumulate=False)
    want = R.row_values(out["qt"], out["sft"]) @ R.row_values(xt["qt"], xt["sft"]).T
    assert np.abs(dW.double().cpu().numpy() - want).max() <= 1e-4 * math.sqrt(np.mean(want ** 2))


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_backward_at_large_pre_activations(act):
    # the slope is 0 or 1 to FP32 there, and finite
    z = torch.tensor([50.0, 1e2, 1e4, 1e8, 1e15], dtype=torch.bfloat16)
    Z = torch.cat([z, -z, torch.zeros(118, dtype=torch.bfloat16)]).expand(2, 128).contiguous()
    dD = torch.ones(2, 128, dtype=torch.bfloat16)
    got = run_backward(dD, Z, act, ("dbias",))["dbias"]
    assert (got[:5] == 2).all() and (got[5:10].abs() <= 1e-12).all()


@pytest.mark.parametrize("act", ["gelu_tanh", "silu"])
def test_special_values_do_not_touch_their_neighbours(act):
    # two columns share a reciprocal: every special value beside every other
    special = [math.nan, math.inf, -math.inf, 3e38, -3e38, -90.0, 90.0, 0.0, 1.0]
    pairs = [(a, b) for a in special for b in special]
    N = 2 * len(pairs) + (-2 * len(pairs)) % 8
    bias = torch.zeros(N)
    bias[:2 * len(pairs)] = torch.tensor(pairs).flatten()
    D = sentinel_bf16(300, N)
    z8 = torch.zeros(300, 128, dtype=torch.uint8), torch.zeros(N, 128, dtype=torch.uint8)
    dg.dg_gemm_fp8_nt_epilogue(dev(z8[0]), dev(torch.ones(300, 1)), dev(z8[1]), dev(torch.ones((N + 127) // 128, 1)), D, bias=dev(bias), act=act)
    got = D[0].double().cpu().numpy()
    x = bias.double().numpy()
    finite = np.isfinite(x)
    np.testing.assert_allclose(got[finite], R.act(x[finite], act), rtol=2.0 ** -8, atol=1e-6)
    assert np.isnan(got[np.isnan(x)]).all() and (got[x == np.inf] == np.inf).all()
