"""The few-token expert layer at sizes where its weight stream is cut every way that it can be: two halves of the
chunks with a third barrier, more units than CTAs, shares that begin inside a unit, CTAs with more segments than there
are slots between the promoting and the finishing warps, a half that ends inside an expert. What a case is there for is
asserted from the sharing rule, restated here, so that a change of that rule cannot leave a path untested.

Tolerances: those of test_gpu_moe_layer.py.
"""
import math

import numpy as np
import pytest
import torch

import moe_grouped_gemm_tma_gb300 as dg
from tests.test_gpu_moe_layer import check, run

pytestmark = pytest.mark.gpu

PART_SLOTS = 4


def make(T, k, E, H, In, seed, distinct=True):
    """Weights as random codes of 0.25 to 8 in magnitude (quantising this many takes longer than all else here)."""
    g = torch.Generator().manual_seed(seed)
    codes = lambda *s: (torch.randint(0x28, 0x48, s, generator=g) | (torch.randint(0, 2, s, generator=g) << 7)).to(torch.uint8)  # noqa: E731
    scales = lambda K, *s: (torch.rand(*s, generator=g) + 0.5) / (3 * math.sqrt(K))  # noqa: E731
    if distinct:
        ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    else:
        ids = torch.randint(0, E, (T, k), generator=g).to(torch.int32)
    return {"x": torch.randn(T, H, generator=g).to(torch.bfloat16), "ids": ids, "w": torch.rand(T, k, generator=g) + 0.1,
            "W13": codes(E, 2 * In, H), "s13": scales(H, E, 2 * In // 128, H // 128), "W2": codes(E, H, In), "s2": scales(In, E, H // 128, In // 128)}


def plan(c):
    """What the sharing rule makes of a case on this GPU: the set of paths that it takes."""
    T, H = c["x"].shape
    In, A = c["W2"].shape[2], c["ids"].numel()
    G = min(torch.cuda.get_device_properties(0).multi_processor_count, 160)
    nt = 16 if T <= 16 else 32 if T <= 32 else 64
    per = np.bincount(c["ids"].flatten().numpy())
    owner = [e for e, n in enumerate(per) for _ in range((n + nt - 1) // nt)]
    chunks = len(owner)
    halves = chunks * (In // 128) * (H // 128) >= 22 * G
    first = (chunks * 5 + 7) // 8 if halves else chunks
    paths = set()
    if halves:
        paths.add("halves")
        if owner[first - 1] == owner[first]:
            paths.add("half inside an expert")
    for line in range(4):
        nc = first if line % 2 == 0 else chunks - first
        kbs = (H if line < 2 else In) // 128
        blocks = In // 128 if line < 2 else (H + 255) // 256
        units, total = nc * blocks, nc * blocks * kbs
        if total == 0:
            continue
        sharers = min(total, G)
        if units <= G:
            m = min(kbs, G // units)
            if line >= 2 and A >= 64:
                m = min(m, 2)
            if ((kbs + m - 1) // m - 6) * G <= total:
                sharers = units * m
                paths.add("whole CTAs a unit, phase %d" % (line // 2 + 1))
        else:
            paths.add("more units than CTAs, phase %d" % (line // 2 + 1))
        cut = [total * i // sharers for i in range(sharers + 1)]
        segments = [(b - 1) // kbs - a // kbs + 1 for a, b in zip(cut, cut[1:])]
        if any(a % kbs and s > 1 for a, s in zip(cut, segments)):
            paths.add("cuts inside units, phase %d" % (line // 2 + 1))
        if line < 2 and max(segments) > PART_SLOTS:
            paths.add("part slots in turn")
    return paths


CASES = {
    # name: sizes, distinct experts of a token, the paths that it is there for
    "64 columns, two halves": ((40, 4, 16, 2560, 1408), True, {"halves", "whole CTAs a unit, phase 1", "whole CTAs a unit, phase 2"}),
    "64 columns, two halves, more units than CTAs": ((40, 4, 32, 1024, 1792), True, {"halves", "more units than CTAs, phase 1", "cuts inside units, phase 1"}),
    "16 columns, two halves, half a pair of blocks": ((12, 8, 24, 2944, 1408), True, {
        "halves", "more units than CTAs, phase 1", "cuts inside units, phase 1", "more units than CTAs, phase 2", "cuts inside units, phase 2"}),
    "32 columns, two halves, more units than CTAs": ((24, 6, 24, 2560, 1408), True, {"halves", "more units than CTAs, phase 1", "cuts inside units, phase 1"}),
    "many experts of few rows": ((48, 8, 128, 256, 2048), True, {"halves", "more units than CTAs, phase 1", "part slots in turn", "cuts inside units, phase 2"}),
    "one half, several units a CTA": ((40, 4, 96, 1024, 512), True, {
        "more units than CTAs, phase 1", "more units than CTAs, phase 2", "cuts inside units, phase 1", "cuts inside units, phase 2"}),
    "16 columns, a half inside an expert": ((16, 16, 4, 2560, 1408), False, {"halves", "half inside an expert"}),
    "64 columns, a half inside an expert": ((64, 16, 4, 2560, 1536), False, {"halves", "half inside an expert"}),
}


@pytest.mark.parametrize("name", CASES)
def test_cuts_of_the_lines(name):
    sizes, distinct, want = CASES[name]
    c = make(*sizes, seed=sum(sizes), distinct=distinct)
    if name.startswith("64 columns, a half"):
        # 4 experts of 256 rows: 16 chunks of 64, of which 10 are the first half
        c["ids"] = torch.arange(4, dtype=torch.int32).repeat(64, 4)
    paths = plan(c)
    assert want <= paths, paths
    if name.startswith("one half"):
        assert "halves" not in paths
    T, k, E, H, In = sizes
    ws = dg.moe_layer_workspace(64, 16, E, H, In)
    check(c, ws=ws)
    first = run(c, ws=ws).clone()
    # on a workspace that another case has used, and with a residual and empty slots
    other = make(33, 6, E, H, In, seed=1, distinct=False)
    other["ids"][::5] = -1
    check(other, "gelu_tanh", torch.randn(33, H, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16), ws)
    for _ in range(5):
        assert torch.equal(run(c, ws=ws), first)
    assert torch.equal(run(c), first)


def values64(v):
    """The 1x128 quantisation's values of float64 [rows, n * 128] on the GPU."""
    b = v.unflatten(1, (-1, 128))
    s = (b.abs().amax(2, keepdim=True).clamp_min(float(torch.tensor(1e-4))) / 448).float().double()
    return ((b / s).float().to(torch.float8_e4m3fn).double() * s).flatten(1)


@pytest.mark.parametrize("T,k,E", [(1, 8, 128), (16, 8, 128), (64, 4, 40)])
def test_serving_sizes(T, k, E):
    # many experts of a large layer, most of them met by a token or two
    H, In = 7168, 2048
    g = torch.Generator(device="cuda").manual_seed(T + E)
    codes = lambda *s: torch.randint(0x28, 0x48, s, device="cuda", generator=g, dtype=torch.uint8) | (torch.randint(0, 2, s, device="cuda", generator=g, dtype=torch.uint8) << 7)  # noqa: E731
    scales = lambda K, *s: (torch.rand(*s, device="cuda", generator=g) + 0.5) / (3 * math.sqrt(K))  # noqa: E731
    W13, s13, W2, s2 = codes(E, 2 * In, H), scales(H, E, 2 * In // 128, H // 128), codes(E, H, In), scales(In, E, H // 128, In // 128)
    x = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
    ids = torch.rand(T, E, device="cuda", generator=g).topk(k, 1)[1].int()
    w = torch.rand(T, k, device="cuda", generator=g) + 0.1
    out = torch.full_like(x, math.nan)
    ws = dg.moe_layer_workspace(T, k, E, H, In)
    dg.dg_moe_layer(x, ids, w, W13, s13, W2, s2, out, ws, act="silu", residual=x)
    assert dg.dg_device_status() == 0
    want, xv = x.double(), values64(x.double())
    block = lambda q, s: q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)  # noqa: E731
    for e in ids.unique().tolist():
        t, j = (ids == e).nonzero(as_tuple=True)
        gate, up = (xv[t] @ block(W13[e], s13[e]).t()).chunk(2, 1)
        h = values64(gate * torch.sigmoid(gate) * up)
        want.index_add_(0, t, w[t, j].double().unsqueeze(1) * (h @ block(W2[e], s2[e]).t()))
    got = out.double()
    rms = want.square().mean().sqrt()
    assert ((got - want).abs() <= 1e-2 * want.abs() + 2e-2 * rms).all()
    assert (got - want).norm() <= 3e-3 * want.norm()
    again = torch.full_like(x, math.nan)
    dg.dg_moe_layer(x, ids, w, W13, s13, W2, s2, again, ws, act="silu", residual=x)
    assert torch.equal(again, out)
