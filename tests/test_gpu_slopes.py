"""The slopes of the backward pass at every BF16 pre-activation, against 64 bits.

With one row and dD = 1 the bias gradient is the slope itself. Tolerance: a slope lies between -0.2 and 1.13 and ends with a
rounding of up to 2^-24; before that stand the sigmoid's or the tail's (half of it, as they are under 1), the
exponential's error of 2^-22.5 times p (1 - p) <= 1/4, which is 0.7 of it, and the roundings of a product that is under 0.3:
two and a half times 2^-24.
"""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_tma_gb300 as dg
from tests import operators_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_every_slope_is_right_to_fp32(act):
    z = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    z = z[torch.isfinite(z.float())]
    N = z.numel() // 128 * 128
    Z = z[:N].view(1, N).contiguous()
    out = torch.empty(N, device="cuda")
    dg.dg_epilogue_backward(torch.ones(1, N, dtype=torch.bfloat16, device="cuda"), Z.cuda(), None, None, None, None, out,
                            dg.epilogue_backward_workspace(1, N), act=act)
    x = Z[0].double().numpy()
    # (beyond 30 the 64-bit forms give 0 and 1 too, but for products of an infinity and a zero)
    want = np.where(np.abs(x) > 30, (x > 0).astype(np.float64), R.act_slope(np.clip(x, -30, 30), act))
    assert np.abs(out.cpu().double().numpy() - want).max() <= 2.5 * 2.0 ** -24
