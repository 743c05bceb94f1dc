"""Waits of the operators around the products that run out, without a GPU fault.

As in test_gpu_failure.py: dg_testing_arm_fault has one launch leave something out under a short limit of its waits, so
that a wait runs out (nothing arrives; nothing faults). The launch has to report DG_DEVICE_TIMEOUT once, and the next
one in the same process has to be right. A copy that a warp has stopped waiting for has to be waited for before the CTA
gives up its shared memory; that drain is bounded by 50 ms, which a copy that never comes uses up, so the launch takes
at least that long where it drains, and only its waits' few milliseconds where it does not.
"""
import time

import pytest
import torch

import moe_grouped_gemm_tma_gb300 as dg
from moe_grouped_gemm_tma_gb300 import inputs as I
from tests.gpu_util import bf16_bits, dev, sentinel_bf16
from tests.test_gpu_moe_layer import make as make_layer, run as run_layer

pytestmark = pytest.mark.gpu

DG_DEVICE_TIMEOUT = 6
LIMIT_NS = 5_000_000
DRAIN_S = 0.050


def timed_out(call):
    """Seconds of a call that has to report a wait that ran out, once."""
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    call()
    assert dg.dg_device_status() == DG_DEVICE_TIMEOUT
    took = time.perf_counter() - t0
    assert dg.dg_device_status() == 0
    assert took < 5.0
    return took


def epilogue_call(M, N, K):
    c = I.make_normal(I.seed_for(9, M + N + 1), M, N, K)
    A, sfa, B, sfb = dev(c.A), dev(c.sfa), dev(c.B), dev(c.sfb)
    res = torch.randn(M, N, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()

    def call():
        D, Z = sentinel_bf16(M, N), sentinel_bf16(M, N)
        dg.dg_gemm_fp8_nt_epilogue(A, sfa, B, sfb, D, act="silu", residual=res, Z=Z)
        return D, Z
    return call


@pytest.mark.parametrize("bn", [64, 128, 192])
@pytest.mark.parametrize("M", [300, 1500])
def test_a_residual_that_does_not_come(bn, M, tune):
    tune(bn=bn, split=1, swap=0)
    call = epilogue_call(M, 1032, 512)
    want = [bf16_bits(t) for t in call()]
    assert dg.dg_device_status() == 0
    dg.dg_testing_arm_fault("residual", LIMIT_NS)
    assert timed_out(call) >= DRAIN_S
    got = [bf16_bits(t) for t in call()]
    assert dg.dg_device_status() == 0
    assert all((a == b).all() for a, b in zip(got, want))


@pytest.mark.parametrize("M,split", [(300, 1), (100, 4)])
def test_an_epilogue_product_whose_operands_do_not_come(M, split, tune):
    tune(split=split, swap=0)
    call = epilogue_call(M, 520, 1024)
    want = [bf16_bits(t) for t in call()]
    dg.dg_testing_arm_fault("first_fill", LIMIT_NS)
    timed_out(call)
    got = [bf16_bits(t) for t in call()]
    assert dg.dg_device_status() == 0
    assert all((a == b).all() for a, b in zip(got, want))


def test_an_armed_fault_is_spent_by_the_expert_layer():
    # not left for a later launch of another kind
    c = make_layer(3, 2, 4, 256, 128, seed=1)
    call = epilogue_call(300, 520, 1024)
    dg.dg_testing_arm_fault("residual", 1_000_000_000)
    run_layer(c)                                      # (has no residual copy: it runs as usual)
    call()
    assert dg.dg_device_status() == 0


@pytest.mark.parametrize("fault,least", [("first_fill", 0.0), ("token_scales", DRAIN_S), ("grid_barrier", 0.0)])
@pytest.mark.parametrize("T,k,E,H,In", [(5, 2, 8, 1024, 384), (55, 4, 8, 1152, 128), (64, 8, 16, 512, 384)])
def test_an_expert_layer_that_gives_up(fault, least, T, k, E, H, In):
    # (the scales that do not come: a few stages a CTA, so the warp that copies them is done before the wait runs out)
    c = make_layer(T, k, E, H, In, seed=T)
    ws = dg.moe_layer_workspace(T, k, E, H, In)
    want = run_layer(c, ws=ws).clone()
    t = [c[n].cuda() for n in ("x", "ids", "w", "W13", "s13", "W2", "s2")]
    out = sentinel_bf16(T, H)
    dg.dg_testing_arm_fault(fault, LIMIT_NS)
    assert timed_out(lambda: dg.dg_moe_layer(*t, out, ws)) >= least
    ws.zero_()
    for _ in range(3):                                # (run_layer looks at the status after each)
        assert torch.equal(run_layer(c, ws=ws), want)


def test_arming_refuses():
    for fault, limit in (("residual", 0), ("residual", 1 << 60), (0, 1000), (99, 1000)):
        with pytest.raises(dg.DGError):
            dg.dg_testing_arm_fault(fault, limit)
    with pytest.raises(KeyError):
        dg.dg_testing_arm_fault("nothing", 1000)
