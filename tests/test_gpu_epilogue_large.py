"""The backward pass of the product with an epilogue at more tiles than run at once: the tiles that a CTA asks into L2
ahead of its turn, ragged rows at their end, and the bias gradient's second launch. Against 64 bits, on the GPU.

Tolerances: those of test_gpu_epilogue.py.
"""
import math

import pytest
import torch

import moe_grouped_gemm_tma_gb300 as dg

pytestmark = pytest.mark.gpu


def slope(z, act):
    z = z.double().requires_grad_(True)
    f = {"none": lambda v: v, "relu": torch.relu, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu,
         "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[act]
    return torch.autograd.grad(f(z).sum(), z)[0]


def check_rows(q, s, dz):
    """Codes with their 1x128 scales against exact values."""
    b = dz.unflatten(1, (-1, 128))
    amax = b.abs().amax(2)
    want_s = (amax.clamp_min(float(torch.tensor(1e-4))) / 448).float().double()
    assert ((s.double() - want_s).abs() <= 1e-5 * want_s).all()
    step = s.double().unsqueeze(2)
    back = q.double().unflatten(1, (-1, 128)) * step
    # half a step of e4m3, 2^-4 of the value or half the smallest step 2^-10 of the scale, and the errors above
    assert ((back - b).abs() <= (2.0 ** -4 + 2e-5) * b.abs() + 2.0 ** -10 * step * 1.001).all()


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M,N", [(3001, 5248), (200, 65664)])
def test_more_tiles_than_run_at_once(act, M, N):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    Mp = (M + 127) // 128 * 128
    assert (Mp // 128) * (N // 128) >= 6 * sms
    g = torch.Generator(device="cuda").manual_seed(M)
    dD = (torch.randn(M, N, device="cuda", generator=g) * 0.02).to(torch.bfloat16)
    Z = (torch.randn(M, N, device="cuda", generator=g) * 1.5).to(torch.bfloat16)
    e4 = torch.float8_e4m3fn
    ws = dg.epilogue_backward_workspace(M, N)
    runs = []
    for _ in range(2):
        q, qt = torch.full((M, N), math.nan, device="cuda").to(e4), torch.full((N, Mp), math.nan, device="cuda").to(e4)
        sf, sft = torch.full((M, N // 128), -1.0, device="cuda"), torch.full((N, Mp // 128), -1.0, device="cuda")
        dbias = torch.full((N,), math.nan, device="cuda")
        dg.dg_epilogue_backward(dD, Z, q, sf, qt, sft, dbias, ws, act=act)
        runs.append((q.view(torch.uint8), sf, qt.view(torch.uint8), sft, dbias))
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    dz = dD.double() * slope(Z, act)
    check_rows(q.float(), sf, dz)
    check_rows(qt.float(), sft, torch.nn.functional.pad(dz, (0, 0, 0, Mp - M)).t().contiguous())
    assert (qt[:, M:].float() == 0).all()
    assert ((dbias.double() - dz.sum(0)).abs() <= 1e-5 * dz.abs().sum(0) + 1e-12).all()
