"""Operators back to back, each starting while the one that writes its input ends, in place and many times over: the same
bits as with the device idle between the calls."""
import pytest
import torch

import moe_grouped_gemm_tma_gb300 as dg
from moe_grouped_gemm_tma_gb300 import inputs as I
from tests.gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 20, 60, 300])
def test_a_residual_stream(M):
    # h += act(W Q(h) + b), its quantisation, routing by its first columns and the backward pass of it, 30 layers
    H, E, k = 1152, 128, 6
    c = I.make_normal(I.seed_for(9, M), M, H, H)
    W, s, g = dev(c.B), dev(c.sfb), torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, H, device="cuda", generator=g).to(torch.bfloat16)
    bias = torch.randn(H, device="cuda", generator=g)
    Mp = (M + 127) // 128 * 128
    e4 = torch.float8_e4m3fn
    ws = dg.epilogue_backward_workspace(M, H)

    def layers(between):
        h, q, sf = x.clone(), torch.empty(M, H, dtype=e4, device="cuda"), torch.empty(M, H // 128, device="cuda")
        qt, sft, db = torch.empty(H, Mp, dtype=e4, device="cuda"), torch.empty(H, Mp // 128, device="cuda"), torch.empty(H, device="cuda")
        Z, ids, w = torch.empty_like(h), torch.empty(M, k, dtype=torch.int32, device="cuda"), torch.empty(M, k, device="cuda")
        logits = torch.empty(M, E, dtype=torch.bfloat16, device="cuda")
        dl, seen = torch.empty_like(logits), []
        torch.cuda.synchronize()
        for _ in range(30):
            dg.dg_epilogue_backward(h, None, q, sf, None, None, None)
            between()
            dg.dg_gemm_fp8_nt_epilogue(q, sf, W, s, h, bias=bias, act="silu", residual=h, Z=Z)
            between()
            dg.dg_gemm_fp8_nt_epilogue(q, sf, W[:E], s[:1], logits)
            between()
            dg.dg_moe_route(logits, ids, w, scoring="sigmoid")
            between()
            dg.dg_moe_route_backward(logits, ids, w, dl, scoring="sigmoid")
            between()
            dg.dg_epilogue_backward(h, Z, q, sf, qt, sft, db, ws, act="silu")
            between()
            seen += [t.clone() for t in (h, Z, ids, w, dl, q.view(torch.uint8), sf, qt.view(torch.uint8), sft, db)]
        torch.cuda.synchronize()
        return seen

    want = layers(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(a.nan_to_num() if a.is_floating_point() else a, b.nan_to_num() if b.is_floating_point() else b)
                   for a, b in zip(layers(lambda: None), want))
    assert dg.dg_device_status() == 0
