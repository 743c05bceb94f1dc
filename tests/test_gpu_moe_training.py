"""The operators between the grouped products in a run, as the example's block uses them: each step of its forward and backward
pass against the 64-bit form of that step's own inputs, captured passes, several streams."""
import pytest
import torch

import moe_grouped_gemm_tma_gb300 as dg
from tests import between_ref as B
from tests.test_gpu_glu import check_backward

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def blocks(codes, s):
    """float64 weights [E, N, K] of 128x128-scaled codes."""
    q = codes.view(torch.float8_e4m3fn).double()
    return q * s.double().repeat_interleave(128, 1).repeat_interleave(128, 2)


def product_bound(a, b, want):
    """FP32 sums of K exact products, scaled once per 128 of them (2^-24 each of the absolute sum), one rounding to BF16."""
    K = a.shape[1]
    return 2.0 ** -8 * want.abs() + (K + 2 * K // 128 + 2) * 2.0 ** -24 * (a.abs() @ b.abs().t()) + 2.0 ** -133


def check_product(A, sa, W, sw, m_indices, got):
    a, w = B.values(A, sa), blocks(W, sw)
    for e in range(w.shape[0]):
        r = (m_indices == e).nonzero()[:, 0]
        want = a[r] @ w[e].t()
        assert ((got[r].double() - want).abs() <= product_bound(a[r], w[e], want)).all(), e


@pytest.mark.parametrize("T,H,I,E,k,act", [(300, 512, 256, 8, 2, "silu"), (77, 256, 384, 5, 5, "gelu_tanh"), (1, 256, 128, 4, 1, "silu"), (900, 384, 128, 40, 3, "gelu")])
def test_every_step_of_a_training_step(T, H, I, E, k, act):
    from examples.moe_block import Experts
    block = Experts(H, I, E, k, act=act, seed=T)
    block.norm.normal_(generator=gen(4)).mul_(0.2).add_(1)
    x = torch.randn(T, H, device=DEV, generator=gen(1)).bfloat16()
    dout = (torch.randn(T, H, device=DEV, generator=gen(2)) * 0.1).bfloat16()
    out = block.train_forward(x)
    dx = block.backward(dout)
    assert dg.dg_device_status() == 0
    s, b, mi = block.saved, block.steps, block.saved["m_indices"]
    # forward
    n = B.rmsnorm(x, block.norm, float(torch.tensor(1e-6)))
    assert ((s["y"].double() - n).abs() <= (2.0 ** -8 + 2.0 ** -18) * n.abs() + 2.0 ** -133).all()
    want = B.sort(s["ids"].tolist(), E, dg.moe_sort_rows(T, k, E))
    assert s["rows"].tolist() == want[0] and s["counts"].tolist() == want[1] and mi.tolist() == want[2][: len(mi)]
    row = s["rows"][s["rows"] >= 0].long()
    token = (s["rows"] >= 0).nonzero()[:, 0]
    B.check_codes(s["A"][row], s["sfa"][row], n[token], 2.0 ** -19 * n[token].abs())
    assert (s["A"][B.pads(mi)].view(torch.uint8) == 0).all() and (s["kept"][B.pads(mi)].view(torch.uint8) == 0).all()
    # out is x plus the weighted rows
    y, mag = B.combine(s["Y"], s["rows"], s["weights"], x)
    assert ((out.double() - y).abs() <= 2.0 ** -8 * y.abs() + (k + 2) * 2.0 ** -23 * mag + 2.0 ** -133).all()
    # backward
    dY = torch.zeros_like(b["dY"], dtype=torch.float64)
    dY[row] = (s["weights"].double().unsqueeze(2) * dout.double().unsqueeze(1))[s["rows"] >= 0]
    assert ((b["dY"].double() - dY).abs() <= (2.0 ** -8 + 2.0 ** -22) * dY.abs() + 2.0 ** -133).all()
    check_product(*b["q"], block.W2t, block.s2t, mi, b["dH"])
    tagged = mi >= 0
    used = mi.view(-1, 128)[:, :1].expand(-1, 128).reshape(-1) >= 0
    assert (b["dH"][used & ~tagged] == 0).all()                       # zeros go through the products
    g, u = B.values(s["kept"], s["kept_sf"]).split(I, 1)
    check_backward(b["dH"], g, u, act, {"q": b["z"], "qt": b["zt"], "ht": b["ht"]}, 2.0 ** -24)
    check_product(*b["z"], block.W13t, block.s13t, mi, b["dA"])
    got, scale = B.quantise(B.columns(B.values(s["A"], s["sfa"]).float()))
    assert torch.equal(b["At"][0].double(), got) and torch.equal(b["At"][1].double(), scale)
    # weight gradients, each over its own rows: FP32 sums of as many products
    at = 0
    for e, kk in enumerate(block.ks):
        for left, right, d in ((b["qt"], b["ht"], block.dmaster2[e]), (b["zt"], b["At"], block.dmaster13[e])):
            l, r = B.values(*left)[:, at:at + kk], B.values(*right)[:, at:at + kk]
            want = l @ r.t()
            assert ((d.double() - want).abs() <= (kk + 2) * 2.0 ** -23 * (l.abs() @ r.abs().t()) + 1e-30).all(), e
        at += kk
    want, want_dw = B.rmsnorm_backward(b["dy"], x, block.norm, float(torch.tensor(1e-6)), dout)
    mag = (b["dy"].double().abs() * block.norm.double() + dout.double().abs() + 1e-3) * 4
    assert ((dx.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * mag).all()
    assert ((block.dnorm.double() - want_dw).abs() <= 2.0 ** -16 * (b["dy"].double() * n).abs().sum(0) + 1e-9).all()


def test_prefill_and_its_graph():
    from examples.moe_block import Experts
    block = Experts(512, 256, 16, 4, seed=3)
    x, out, g = block.graph(200)
    for seed in (1, 2):                           # (another routing each time: the counts stay on the device)
        x.copy_(torch.randn(200, 512, device=DEV, generator=gen(seed)))
        g.replay()
        eager = block.train_forward(x.clone())
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_two_streams_at_once():
    """Two sets of calls on two streams, a workspace each, give what each gives alone."""
    T, k, E, H, I = 3000, 8, 64, 1024, 512
    def work(seed, ws):
        ids = torch.randint(-1, E, (T, k), generator=gen(seed), device=DEV, dtype=torch.int32)
        x = torch.randn(T, H, device=DEV, generator=gen(seed + 1)).bfloat16()
        Mt = dg.moe_sort_rows(T, k, E)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
        rows, counts, mi = i32(T, k), i32(E), i32(Mt)
        A = torch.zeros(Mt, H, dtype=torch.bfloat16, device=DEV)
        q, sf = torch.zeros(Mt, I, dtype=torch.uint8, device=DEV), torch.zeros(Mt, I // 128, device=DEV)
        out, dx, dw, dwt = torch.empty_like(x), torch.empty_like(x), torch.empty(H, device=DEV), torch.empty(T, k, device=DEV)
        dy = torch.zeros_like(A)

        def run():
            dg.dg_moe_sort_contiguous(ids, rows, counts, mi, ws[0])
            dg.dg_moe_gather(x, None, rows, A, m_indices=mi)
            dg.dg_glu(A, q, sf, m_indices=mi)
            dg.dg_moe_combine(A, rows, out)
            dg.dg_moe_combine_backward(out, rows, dy, y=A, dweights=dwt, m_indices=mi)
            dg.dg_rmsnorm_backward(out, x, torch.ones(H, device=DEV), dx, dw, ws[1])
            return [t.clone() for t in (rows, counts, mi, A, q, sf, out, dy, dwt, dx, dw)]
        return run

    spaces = [(dg.moe_sort_workspace(T, k, E), dg.rmsnorm_backward_workspace(T, H)) for _ in range(2)]
    runs = [work(10 * i, spaces[i]) for i in range(2)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for r, st in zip(runs, streams):
            with torch.cuda.stream(st):
                got.append(r())
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for u, v in zip(a, b):
                assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))


def test_a_given_stream_is_the_one_used():
    side = torch.cuda.Stream()
    x = torch.randn(64, 512, device=DEV, generator=gen(1)).bfloat16()
    w = torch.ones(512, device=DEV)
    y = torch.zeros_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)             # (tens of milliseconds)
    dg.dg_rmsnorm(x, w, y=y, stream=side)
    assert not side.query()
    side.synchronize()
    want = torch.empty_like(y)
    dg.dg_rmsnorm(x, w, y=want)
    assert torch.equal(y, want)


def test_the_workspaces_hold_anything():
    T, k, E, H = 4000, 8, 100, 640
    ids = torch.randint(0, E, (T, k), generator=gen(3), device=DEV, dtype=torch.int32)
    dy, x = (torch.randn(T, H, device=DEV, generator=gen(i)).bfloat16() for i in (4, 5))
    big = dg.moe_sort_workspace(2 * T, k, E), dg.rmsnorm_backward_workspace(2 * T, 2 * H)
    seen = []
    for fill in (0, 0x7F, 0xFF):
        for w in big:
            w.fill_(fill)
        rows, counts = torch.empty_like(ids), torch.empty(E, dtype=torch.int32, device=DEV)
        mi = torch.empty(dg.moe_sort_rows(T, k, E), dtype=torch.int32, device=DEV)
        dg.dg_moe_sort_contiguous(ids, rows, counts, mi, big[0])
        dx, dw = torch.empty_like(x), torch.empty(H, device=DEV)
        dg.dg_rmsnorm_backward(dy, x, torch.ones(H, device=DEV), dx, dw, big[1])
        seen.append((rows, counts, mi, dx, dw))
    for other in seen[1:]:
        assert all(torch.equal(a, b) for a, b in zip(seen[0], other))


def test_the_example_trains():
    from examples.moe_block import train_experts
    losses = train_experts(H=256, I=128, E=8, k=2, tokens=300, steps=3)
    assert len(losses) == 3 and all(l == l and l < float("inf") for l in losses)
