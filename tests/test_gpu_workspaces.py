"""Workspaces with anything in them past the bytes that have to be zero, NaN codes and NaN sums among it, give the same
results as zeroed ones."""
import pytest
import torch

import moe_grouped_gemm_tma_gb300 as dg
from tests.test_gpu_epilogue import backward_inputs, run_backward
from tests.test_gpu_moe_layer import make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,E,H,In", [(1, 1, 1, 128, 128), (5, 2, 8, 1024, 384), (33, 6, 16, 512, 256), (64, 8, 16, 512, 384), (48, 2, 128, 256, 128)])
def test_expert_layer(T, k, E, H, In):
    c = make(T, k, E, H, In, seed=T)
    ws = dg.moe_layer_workspace(T, k, E, H, In)
    want = run(c, ws=ws.zero_()).clone()
    for fill in (0x7F, 0xFF):
        ws.fill_(fill)
        ws[:4096] = 0
        assert torch.equal(run(c, ws=ws), want)


@pytest.mark.parametrize("M,N", [(128, 256), (700, 512), (2500, 2048)])
def test_bias_gradient(M, N):
    dD, Z = backward_inputs(M, N, M, "silu")
    ws = dg.epilogue_backward_workspace(M, N)
    want = run_backward(dD, Z, "silu", ("dbias",), ws.zero_())["dbias"]
    ws.fill_(0xFF)
    ws[:1024] = 0
    assert torch.equal(run_backward(dD, Z, "silu", ("dbias",), ws)["dbias"], want)
