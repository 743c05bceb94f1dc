"""The few-token expert layer on the GPU against 64 bits.

Tolerance. The products' sums carry the error that dg_gemm_fp8_nt's tests allow theirs, 1e-2 of the rms at most, twice
in a row; a hidden activation whose quotient is within FP32 rounding of a midpoint may take the neighbouring code, one
sixteenth off, which moves an output by a sixteenth of one of I terms; the output is rounded to BF16 once (2^-9):
|err| <= 1e-2 |want| + 2e-2 rms(want), and the whole output within 3e-3 of its norm.
"""
import math

import numpy as np
import pytest
import torch

import moe_grouped_gemm_tma_gb300 as dg
from moe_grouped_gemm_tma_gb300 import inputs as I
from tests import operators_ref as R
from tests.gpu_util import sentinel_bf16

pytestmark = pytest.mark.gpu


def make(T, k, E, H, In, seed=0, distinct=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    if distinct:
        ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    else:
        ids = torch.randint(0, E, (T, k), generator=g).to(torch.int32)
    w = torch.rand(T, k, generator=g) + 0.1
    w13 = [I.quantize_128x128(torch.randn(2 * In, H, generator=g) / math.sqrt(H)) for _ in range(E)]
    w2 = [I.quantize_128x128(torch.randn(H, In, generator=g) / math.sqrt(In)) for _ in range(E)]
    return {"x": x, "ids": ids, "w": w, "W13": torch.stack([a for a, _ in w13]), "s13": torch.stack([b for _, b in w13]),
            "W2": torch.stack([a for a, _ in w2]), "s2": torch.stack([b for _, b in w2])}


def run(c, act="silu", residual=None, ws=None, out=None):
    T, H = c["x"].shape
    E, _, In = c["W2"].shape
    if ws is None:
        ws = dg.moe_layer_workspace(T, c["ids"].shape[1], E, H, In)
    if out is None:
        out = sentinel_bf16(T, H)
    dg.dg_moe_layer(*(c[n].cuda() for n in ("x", "ids", "w", "W13", "s13", "W2", "s2")), out, ws, act=act,
                    residual=None if residual is None else residual.cuda())
    assert dg.dg_device_status() == 0
    return out


def check(c, act="silu", residual=None, ws=None):
    got = run(c, act, residual, ws).double().cpu().numpy()
    want = R.moe(c["x"].double().numpy(), c["ids"].numpy(), c["w"].double().numpy(), c["W13"], c["s13"], c["W2"], c["s2"], act,
                 None if residual is None else residual.double().numpy())
    assert np.isfinite(got).all()
    rms = math.sqrt(np.mean(want ** 2))
    assert (np.abs(got - want) <= 1e-2 * np.abs(want) + 2e-2 * rms).all(), np.abs(got - want).max() / max(rms, 1e-30)
    assert np.linalg.norm(got - want) <= 3e-3 * np.linalg.norm(want)


@pytest.mark.parametrize("T,k,E,H,In", [
    (1, 1, 1, 128, 128), (1, 8, 16, 512, 256), (2, 2, 4, 256, 128), (5, 2, 8, 1024, 384), (16, 4, 8, 384, 256), (17, 4, 8, 640, 128),
    (33, 6, 16, 512, 256), (64, 8, 16, 512, 384), (64, 1, 2, 256, 256), (64, 3, 3, 896, 640), (7, 16, 64, 256, 128), (48, 2, 128, 256, 128),
])
def test_shapes(T, k, E, H, In):
    c = make(T, k, E, H, In, seed=T + E)
    check(c)
    check(c, residual=torch.randn(T, H, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16))


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_activations(act):
    check(make(9, 2, 4, 384, 256, seed=3), act)


@pytest.mark.parametrize("T", [3, 40])
def test_empty_slots(T):
    c = make(T, 4, 6, 256, 256, seed=T)
    g = torch.Generator().manual_seed(8)
    lost = torch.rand(T, 4, generator=g) < 0.6
    lost[0] = True                                   # a token without any expert
    c["ids"] = torch.where(lost, torch.tensor([-1, 6, 1 << 30, -(1 << 31)], dtype=torch.int64), c["ids"].long()).to(torch.int32)
    check(c)
    check(c, residual=torch.randn(T, 256, generator=g).to(torch.bfloat16))


def test_no_expert_at_all():
    c = make(5, 2, 4, 384, 128, seed=1)
    c["ids"].fill_(-1)
    assert (run(c) == 0).all()
    res = torch.randn(5, 384).to(torch.bfloat16)
    assert torch.equal(run(c, residual=res).cpu(), res)


@pytest.mark.parametrize("T,k,E", [(6, 8, 2), (40, 3, 2), (64, 16, 3), (1, 300, 2)])
def test_an_expert_named_more_than_once(T, k, E):
    # more rows of an expert than a chunk holds, and a token with several columns of one chunk
    check(make(T, k, E, 256, 128, seed=T + k, distinct=False))


def test_one_expert_meets_every_token():
    c = make(64, 2, 8, 512, 256, seed=5)
    c["ids"][:, 0] = 3
    c["ids"][:, 1] = torch.where(c["ids"][:, 1] == 3, 4, c["ids"][:, 1])
    check(c)


def test_unmet_experts_are_not_read():
    c = make(4, 2, 6, 256, 128, seed=6)
    c["ids"][c["ids"] == 5] = 0
    c["ids"][:, 1] = torch.where(c["ids"][:, 1] == c["ids"][:, 0], 4, c["ids"][:, 1])
    want = run(c).clone()
    c["W13"][5] = 0x7F                                # NaN codes
    c["s2"][5] = math.nan
    assert torch.equal(run(c), want)


def test_reproducible_and_independent_of_the_workspace_history():
    c = make(33, 4, 8, 640, 384, seed=7)
    ws = dg.moe_layer_workspace(64, 8, 16, 1024, 512)
    first = run(c, ws=ws).clone()
    other = make(64, 8, 16, 1024, 512, seed=9)
    for _ in range(3):
        run(other, ws=ws)
        assert torch.equal(run(c, ws=ws), first)
    assert torch.equal(run(c), first)


def test_residual_and_output_in_place():
    c = make(20, 3, 6, 512, 256, seed=11)
    res = torch.randn(20, 512).to(torch.bfloat16)
    want = run(c, residual=res)
    buf = res.cuda()
    dg.dg_moe_layer(*(c[n].cuda() for n in ("x", "ids", "w", "W13", "s13", "W2", "s2")), buf, dg.moe_layer_workspace(20, 3, 6, 512, 256), residual=buf)
    assert torch.equal(buf, want)
    x = c["x"].cuda()
    dg.dg_moe_layer(x, *(c[n].cuda() for n in ("ids", "w", "W13", "s13", "W2", "s2")), x, dg.moe_layer_workspace(20, 3, 6, 512, 256), residual=x)
    assert torch.equal(x, run(c, residual=c["x"]))


def test_zero_blocks_and_special_values():
    c = make(4, 2, 4, 384, 256, seed=12)
    c["x"][0, :128] = 0                               # an all-zero block takes the scale floor
    check(c)
    c["x"][1, 5] = math.nan                           # spoils its token only
    out = run(c)
    assert torch.isnan(out[1]).all() and torch.isfinite(out[[0, 2, 3]]).all()


def test_integer_exact():
    # every step exact: x[0] = 448 is code 448 with scale 1, one gate row and one up row pick it up (448 each), the
    # only hidden value 448 * 448 is code 448 with scale 448, and the output is that times a power of two
    H, In = 256, 128
    one = 0x38                                        # 1.0
    c = make(3, 1, 2, H, In, seed=13)
    c["x"] = torch.zeros(3, H, dtype=torch.bfloat16)
    c["x"][:, 0] = 448.0                              # code 448, scale 1
    c["ids"] = torch.tensor([[0], [1], [0]], dtype=torch.int32)
    c["w"] = torch.tensor([[1.0], [0.5], [2.0]])
    c["W13"].zero_()
    c["s13"].fill_(1.0)
    c["W13"][:, 3, 0] = one                           # gate row 3: 448
    c["W13"][:, In + 3, 0] = one                      # up row 3: 448
    c["W2"].zero_()
    c["W2"][0, :, 3] = one
    c["W2"][1, ::2, 3] = one
    c["s2"].fill_(2.0 ** -10)
    out = run(c, "none").double().cpu().numpy()
    v = 448.0 * 448.0 * 2.0 ** -10                    # 196
    assert (out[0] == v).all() and (out[2] == 2 * v).all()
    assert (out[1, ::2] == v / 2).all() and (out[1, 1::2] == 0).all()


def test_replayed_from_a_cuda_graph():
    c = make(8, 2, 4, 512, 256, seed=14)
    t = {n: c[n].cuda() for n in ("x", "ids", "w", "W13", "s13", "W2", "s2")}
    ws = dg.moe_layer_workspace(8, 2, 4, 512, 256)
    out = sentinel_bf16(8, 512)
    call = lambda: dg.dg_moe_layer(*(t[n] for n in ("x", "ids", "w", "W13", "s13", "W2", "s2")), out, ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed in (1, 2):
        other = make(8, 2, 4, 512, 256, seed=seed)
        t["x"].copy_(other["x"])
        t["ids"].copy_(other["ids"])
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, run({**c, "x": other["x"], "ids": other["ids"]}))


def test_on_a_stream_of_its_own():
    c = make(3, 2, 4, 512, 256, seed=15)
    want = run(c)
    t = [c[n].cuda() for n in ("x", "ids", "w", "W13", "s13", "W2", "s2")]
    ws, out = dg.moe_layer_workspace(3, 2, 4, 512, 256), sentinel_bf16(3, 512)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    dg.dg_moe_layer(*t, out, ws, stream=st)
    st.synchronize()
    assert torch.equal(out, want)


def test_router_feeds_the_layer():
    c = make(11, 2, 6, 256, 128, seed=16)
    logits = torch.randn(11, 6, generator=torch.Generator().manual_seed(2))
    logits[4] = -math.inf
    ids = torch.empty(11, 2, dtype=torch.int32, device="cuda")
    w = torch.empty(11, 2, device="cuda")
    dg.dg_moe_route(logits.cuda(), ids, w)
    c["ids"], c["w"] = ids.cpu(), w.cpu()
    check(c)
    assert (run(c)[4] == 0).all()


def test_divided_units_repeat_bit_for_bit():
    # units in many parts finished by one CTA or by all of them together, in turn on one workspace
    ws = dg.moe_layer_workspace(64, 8, 16, 1152, 768)
    cases = [make(55, 4, 8, 1152, 128, seed=1), make(3, 2, 4, 1024, 256, seed=2), make(40, 2, 2, 1152, 640, seed=3), make(20, 3, 16, 384, 128, seed=4)]
    first = [run(c, ws=ws).clone() for c in cases]
    for c in cases:
        check(c, ws=ws)
    for _ in range(10):
        for c, f in zip(cases, first):
            assert torch.equal(run(c, ws=ws), f)
