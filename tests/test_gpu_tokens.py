"""Tokens sorted by expert and back, against their plain forms: lists of slots for the sort, copies for the gather, 64-bit sums
for the weighted sum and its gradient."""
import pytest
import torch

import moe_grouped_gemm_tma_gb300 as dg
from tests import between_ref as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def make_ids(T, k, E, kind, seed=0):
    g = gen(seed + 17 * T + k)
    if kind == "spread":
        return torch.randint(0, E, (T, k), generator=g, device=DEV, dtype=torch.int32)       # (an expert may be named twice)
    if kind == "one":
        return torch.full((T, k), E - 1, dtype=torch.int32, device=DEV)
    if kind == "none":
        return torch.full((T, k), -1, dtype=torch.int32, device=DEV)
    ids = torch.randint(-3, E + 3, (T, k), generator=g, device=DEV, dtype=torch.int32)       # some outside [0, E)
    ids[::5] = 2 ** 31 - 1
    ids[1::7] = -2 ** 31
    return ids


def sort_contiguous(ids, E, extra=0, ws=None):
    T, k = ids.shape
    Mt = dg.moe_sort_rows(T, k, E) + extra
    rows = torch.full((T, k), 777, dtype=torch.int32, device=DEV)
    counts = torch.full((E,), 777, dtype=torch.int32, device=DEV)
    m_indices = torch.full((Mt,), 777, dtype=torch.int32, device=DEV)
    ws = dg.moe_sort_workspace(T, k, E).fill_(0xFF) if ws is None else ws
    dg.dg_moe_sort_contiguous(ids, rows, counts, m_indices, ws)
    return rows, counts, m_indices


SIZES = [(1, 1, 1), (1, 8, 64), (5, 2, 8), (33, 6, 3), (127, 1, 2), (128, 4, 256), (511, 8, 256), (512, 8, 1024), (513, 8, 7), (1000, 32, 40), (512, 32, 256), (2049, 8, 64), (8189, 8, 256),
         (2500, 3, 1000), (20000, 4, 600)]


@pytest.mark.parametrize("kind", ["spread", "one", "none", "outside"])
@pytest.mark.parametrize("T,k,E", SIZES)
def test_sort(T, k, E, kind):
    ids = make_ids(T, k, E, kind)
    want = B.sort(ids.tolist(), E, dg.moe_sort_rows(T, k, E) + 256)
    rows, counts, m_indices = sort_contiguous(ids, E, extra=256)
    assert rows.tolist() == want[0] and counts.tolist() == want[1] and m_indices.tolist() == want[2]
    for max_m in (1, max(1, T * k // E), T * k + 1):
        if E * max_m >= 2 ** 31:
            continue
        want = B.sort(ids.tolist(), E, max_m=max_m)
        masked_m = torch.full((E,), 777, dtype=torch.int32, device=DEV)
        rows.fill_(777)
        dg.dg_moe_sort_masked(ids, rows, masked_m, max_m, dg.moe_sort_workspace(T, k, E))
        assert rows.tolist() == want[0] and masked_m.tolist() == want[1], max_m


def test_sort_of_many_slots():
    T, k, E = 40000, 8, 128                       # (several groups of 32 slots a warp)
    ids = make_ids(T, k, E, "outside")
    rows, counts, m_indices = sort_contiguous(ids, E)
    flat = ids.view(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    n = torch.bincount(key, minlength=E + 1)
    assert torch.equal(counts.long(), n[:E])
    room = (n[:E] + 127) // 128 * 128
    base = room.cumsum(0) - room
    order = torch.sort(key, stable=True).indices[: int(n[:E].sum())]
    place = torch.arange(len(order), device=DEV) - (n.cumsum(0) - n)[key[order]]
    want = torch.full_like(flat, -1)
    want[order] = base[key[order]] + place
    assert torch.equal(rows.view(-1).long(), want)
    at = torch.full((len(m_indices),), -1, device=DEV)
    at[want[order]] = key[order]
    assert torch.equal(m_indices.long(), at)


def test_sort_of_nothing():
    E = 6
    rows, counts, m_indices = sort_contiguous(torch.empty(0, 4, dtype=torch.int32, device=DEV), E, extra=256)
    assert counts.tolist() == [0] * E and m_indices.tolist() == [-1] * 256
    rows, counts, m_indices = sort_contiguous(torch.empty(9, 0, dtype=torch.int32, device=DEV), E, extra=128)
    assert counts.tolist() == [0] * E and m_indices.tolist() == [-1] * 128
    counts.fill_(5)
    dg.dg_moe_sort_masked(torch.empty(0, 4, dtype=torch.int32, device=DEV), torch.empty(0, 4, dtype=torch.int32, device=DEV), counts, 3)
    assert counts.tolist() == [0] * E


def test_sort_refuses_too_few_rows_and_no_workspace():
    ids = make_ids(2100, 8, 16, "spread")
    out = lambda n: torch.empty(n, dtype=torch.int32, device=DEV)  # noqa: E731
    with pytest.raises(dg.DGError, match="UNSUPPORTED"):
        dg.dg_moe_sort_contiguous(ids, torch.empty_like(ids), out(16), out(dg.moe_sort_rows(2100, 8, 16) - 128), dg.moe_sort_workspace(2100, 8, 16))
    with pytest.raises(dg.DGError, match="INVALID"):
        dg.dg_moe_sort_contiguous(ids, torch.empty_like(ids), out(16), out(dg.moe_sort_rows(2100, 8, 16)))


# ---------------------------------------------------------------- rows
def gathered(x, sf, rows, m_indices, Mt, fill):
    """The expected rows: `fill` everywhere that nothing is written."""
    out = torch.full((Mt, x.shape[1]), fill, dtype=torch.uint8, device=DEV) if sf is not None else torch.full((Mt, x.shape[1]), fill, dtype=torch.bfloat16, device=DEV)
    osf = None if sf is None else torch.full((Mt, sf.shape[1]), -7.0, device=DEV)
    if m_indices is not None:
        pad = B.pads(m_indices)
        out[pad] = 0
        if osf is not None:
            osf[pad] = torch.tensor(1e-4) / torch.tensor(448.0)
    for j in range(rows.shape[1]):
        t = ((rows[:, j] >= 0) & (rows[:, j] < Mt)).nonzero()[:, 0]
        out[rows[t, j].long()] = x[t]
        if osf is not None:
            osf[rows[t, j].long()] = sf[t]
    return out, osf


@pytest.mark.parametrize("layout", ["contiguous", "masked"])
@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 128), (1, 8, 64, 7168), (5, 2, 8, 1024), (33, 6, 3, 2176), (130, 4, 16, 384), (700, 8, 32, 2048), (50, 32, 32, 128)])
def test_gather_codes(T, k, E, H, layout):
    ids = make_ids(T, k, E, "outside" if T > 20 else "spread")
    if layout == "contiguous":
        rows, counts, m_indices = sort_contiguous(ids, E, extra=128)
        Mt, shape = m_indices.numel(), (m_indices.numel(),)
    else:
        m_indices, max_m = None, max(1, T * k // E)
        rows, masked_m = torch.empty_like(ids), torch.empty(E, dtype=torch.int32, device=DEV)
        dg.dg_moe_sort_masked(ids, rows, masked_m, max_m, dg.moe_sort_workspace(T, k, E))
        Mt, shape = E * max_m, (E, max_m)
    x = torch.randint(0, 256, (T, H), dtype=torch.uint8, device=DEV, generator=gen(T))
    sf = torch.rand(T, H // 128, device=DEV, generator=gen(T + 1))
    out = torch.full((*shape, H), 0xA5, dtype=torch.uint8, device=DEV)
    osf = torch.full((*shape, H // 128), -7.0, device=DEV)
    dg.dg_moe_gather(x, sf, rows, out, osf, m_indices=m_indices)
    want, wsf = gathered(x, sf, rows, m_indices, Mt, 0xA5)
    assert torch.equal(out.view(Mt, H), want) and torch.equal(osf.view(Mt, -1), wsf)


@pytest.mark.parametrize("H", [8, 24, 1000, 1032, 4104])
@pytest.mark.parametrize("padded", [False, True])
def test_gather_bf16(H, padded):
    T, k, E = 77, 3, 5
    ids = make_ids(T, k, E, "outside")
    rows, counts, m_indices = sort_contiguous(ids, E, extra=128)
    x = torch.randn(T, H, device=DEV, generator=gen(H)).bfloat16()
    out = torch.full((m_indices.numel(), H), 3.0, dtype=torch.bfloat16, device=DEV)
    dg.dg_moe_gather(x, None, rows, out, m_indices=m_indices if padded else None)
    assert torch.equal(out, gathered(x, None, rows, m_indices if padded else None, m_indices.numel(), 3.0)[0])


def test_rows_outside_are_left_out():
    T, k, H, Mt = 6, 2, 256, 10
    rows = torch.tensor([[0, -1], [10, 3], [-2 ** 31, 2 ** 31 - 1], [9, 5], [11, -5], [1, 2]], dtype=torch.int32, device=DEV)
    x = torch.randn(T, H, device=DEV, generator=gen(1)).bfloat16()
    out = torch.full((Mt, H), 3.0, dtype=torch.bfloat16, device=DEV)
    dg.dg_moe_gather(x, None, rows, out)
    assert torch.equal(out, gathered(x, None, rows, None, Mt, 3.0)[0])
    y = torch.randn(Mt, H, device=DEV, generator=gen(2)).bfloat16()
    got = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    dg.dg_moe_combine(y, rows, got)
    want, mag = B.combine(y, rows, None, None)
    check_sum(got, want, mag, 2)
    assert (got[2] == 0).all()
    dy, dw = torch.full_like(y, 3.0), torch.full((T, k), 9.0, device=DEV)
    dg.dg_moe_combine_backward(x, rows, dy, y=y, dweights=dw)
    assert torch.equal(dy, gathered(x, None, rows, None, Mt, 3.0)[0])
    assert (dw[(rows < 0) | (rows >= Mt)] == 0).all()


# ---------------------------------------------------------------- weighted sum
def check_sum(got, want, mag, k):
    """FP32 sums of k + 1 terms, each rounded (2^-24 of the terms' magnitudes), then one rounding to BF16 (2^-8)."""
    bound = 2.0 ** -8 * want.abs() + (k + 2) * 2.0 ** -24 * (1 + 2.0 ** -8) * mag + 2.0 ** -133
    assert ((got.double() - want).abs() <= bound).all(), float(((got.double() - want).abs() / bound.clamp_min(1e-30)).max())


SUMS = [(1, 1, 1, 8), (1, 8, 64, 7168), (5, 2, 8, 1024), (64, 5, 16, 1032), (333, 9, 16, 264), (1000, 8, 32, 2048), (50, 32, 32, 128), (3, 4, 4, 16640)]


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,k,E,H", SUMS)
def test_combine(T, k, E, H, weighted, residual):
    ids = make_ids(T, k, E, "outside" if T > 20 else "spread")
    rows, counts, m_indices = sort_contiguous(ids, E)
    y = torch.randn(m_indices.numel(), H, device=DEV, generator=gen(1)).bfloat16()
    y[m_indices < 0] = float("nan")               # what no slot has is not read
    w = torch.randn(T, k, device=DEV, generator=gen(2)) if weighted else None
    if weighted:
        w[rows < 0] = float("nan")
    res = torch.randn(T, H, device=DEV, generator=gen(3)).bfloat16() if residual else None
    want, mag = B.combine(y, rows, w, res)
    out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    dg.dg_moe_combine(y, rows, out, weights=w, residual=res)
    check_sum(out, want, mag, k)
    again = res.clone() if residual else torch.empty_like(out)
    dg.dg_moe_combine(y, rows, again, weights=w, residual=again if residual else None)       # in place, and the same bits
    assert torch.equal(again, out)


def test_combine_without_slots_or_rows():
    res = torch.randn(7, 264, device=DEV, generator=gen(3)).bfloat16()
    y = torch.empty(0, 264, dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(res)
    dg.dg_moe_combine(y, torch.empty(7, 0, dtype=torch.int32, device=DEV), out, residual=res)
    assert torch.equal(out, res)
    dg.dg_moe_combine(y, torch.zeros(7, 3, dtype=torch.int32, device=DEV), out)
    assert (out == 0).all()


def test_infinities_and_nan_stay_in_their_tokens():
    rows = torch.arange(12, dtype=torch.int32, device=DEV).view(4, 3)
    y = torch.randn(12, 512, device=DEV, generator=gen(4)).bfloat16()
    y[4, 100], y[8, 7], y[9, 7] = float("nan"), float("inf"), float("-inf")
    w = torch.rand(4, 3, device=DEV, generator=gen(5)) + 0.5
    out = torch.empty(4, 512, dtype=torch.bfloat16, device=DEV)
    dg.dg_moe_combine(y, rows, out, weights=w)
    bad = ~torch.isfinite(out)
    assert bad.nonzero().tolist() == [[1, 100], [2, 7], [3, 7]] and out[2, 7] == float("inf") and out[3, 7] == float("-inf") and out[1, 100].isnan()


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("T,k,E,H", SUMS + [(40, 3, 4, 1024), (40, 3, 4, 4096), (9, 8, 8, 9000), (1100, 3, 4, 2600), (2100, 3, 4, 5000)])
def test_combine_backward(T, k, E, H, weighted):
    ids = make_ids(T, k, E, "outside" if T > 20 else "spread")
    rows, counts, m_indices = sort_contiguous(ids, E, extra=128)
    Mt = m_indices.numel()
    y = torch.randn(Mt, H, device=DEV, generator=gen(1)).bfloat16()
    y[m_indices < 0] = float("nan")
    w = torch.randn(T, k, device=DEV, generator=gen(2)) if weighted else None
    dout = torch.randn(T, H, device=DEV, generator=gen(3)).bfloat16()
    dy = torch.full((Mt, H), 3.0, dtype=torch.bfloat16, device=DEV)
    dw = torch.full((T, k), float("nan"), device=DEV)
    dg.dg_moe_combine_backward(dout, rows, dy, weights=w, y=y, dweights=dw, m_indices=m_indices)
    want_dw = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(want_dw)
    want = torch.full((Mt, H), 3.0, dtype=torch.float64, device=DEV)
    want[B.pads(m_indices)] = 0.0
    for j in range(k):
        t = (rows[:, j] >= 0).nonzero()[:, 0]
        r = rows[t, j].long()
        terms = y[r].double() * dout[t].double()
        want_dw[t, j], mag[t, j] = terms.sum(1), terms.abs().sum(1)
        want[r] = dout[t].double() * (1.0 if w is None else w[t, j, None].double())
    # a product in FP32, rounded to BF16
    assert ((dy.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -22) * want.abs() + 2.0 ** -133).all()
    # 16 products, 2 halves, 5 exchanges and the running sum for each piece of 1024 values a warp, 8 warps: a rounding each
    chain = (16 + 1 + 5 + 1) * (H // 1024 + 1) + 8
    assert ((dw.double() - want_dw).abs() <= chain * 2.0 ** -24 * mag).all()
    # one without the other, and the same bits
    only, alone = torch.full_like(dy, 3.0), torch.empty_like(dw)
    dg.dg_moe_combine_backward(dout, rows, only, weights=w, m_indices=m_indices)
    dg.dg_moe_combine_backward(dout, rows, None, weights=w, y=y, dweights=alone)
    assert torch.equal(only, dy) and torch.equal(alone, dw)


def test_the_gather_and_the_unweighted_sum_are_each_others_gradients():
    # <gather(x), y> = <x, sum(y)> for whole numbers, exactly
    T, k, E, H = 60, 4, 8, 256
    rows, counts, m_indices = sort_contiguous(make_ids(T, k, E, "outside"), E)
    x = torch.randint(-8, 9, (T, H), device=DEV, generator=gen(1)).bfloat16()
    y = torch.randint(-8, 9, (m_indices.numel(), H), device=DEV, generator=gen(2)).bfloat16()
    gx = torch.zeros_like(y)
    dg.dg_moe_gather(x, None, rows, gx)
    back = torch.empty_like(x)
    dg.dg_moe_combine(y, rows, back)
    assert (gx.double() * y.double()).sum() == (x.double() * back.double()).sum()


def test_gradient_against_differences():
    # the loss sum(out * dout) is linear in y and in the weights: one difference of a whole step is the derivative
    T, k, E, H = 12, 3, 4, 64
    rows, counts, m_indices = sort_contiguous(make_ids(T, k, E, "spread"), E)
    y = torch.randint(-4, 5, (m_indices.numel(), H), device=DEV, generator=gen(1)).bfloat16()
    w = torch.randint(1, 4, (T, k), device=DEV, generator=gen(2)).float()
    dout = torch.randint(-2, 3, (T, H), device=DEV, generator=gen(3)).bfloat16()

    def loss(y, w):
        out = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)      # (sums of up to 36: exact)
        dg.dg_moe_combine(y, rows, out, weights=w)
        return float((out.double() * dout.double()).sum())

    dy, dw = torch.zeros_like(y), torch.empty_like(w)
    dg.dg_moe_combine_backward(dout, rows, dy, weights=w, y=y, dweights=dw)
    for t, j in ((0, 0), (5, 2), (11, 1)):
        up = w.clone()
        up[t, j] += 1
        assert loss(y, up) - loss(y, w) == float(dw[t, j])
        r = int(rows[t, j])
        more = y.clone()
        more[r, 7] += 1
        assert loss(more, w) - loss(y, w) == float(dy[r, 7])


def test_offsets_past_32_bits():
    H, Mt = 16384, 2 ** 18 + 128                  # 4.3 GB of codes, 8.6 GB of BF16
    rows = torch.tensor([[0, Mt - 1], [Mt - 128, 131072]], dtype=torch.int32, device=DEV)
    x = torch.randint(0, 256, (2, H), dtype=torch.uint8, device=DEV, generator=gen(1))
    sf = torch.rand(2, H // 128, device=DEV, generator=gen(2))
    out, osf = torch.zeros(Mt, H, dtype=torch.uint8, device=DEV), torch.zeros(Mt, H // 128, device=DEV)
    m_indices = torch.full((Mt,), -1, dtype=torch.int32, device=DEV)
    m_indices[-128:] = 0
    m_indices[-100:-1] = -1
    out[-128:] = 9
    dg.dg_moe_gather(x, sf, rows, out, osf, m_indices=m_indices)
    for t in range(2):
        for j in range(2):
            assert torch.equal(out[rows[t, j]], x[t]) and torch.equal(osf[rows[t, j]], sf[t])
    assert (out[-100:-1] == 0).all() and (out[-127:-100] == 9).all() and (out[1:131072] == 0).all()
    del out, osf
    y = torch.zeros(Mt, H, dtype=torch.bfloat16, device=DEV)
    y[rows.view(-1).long()] = torch.randn(4, H, device=DEV, generator=gen(3)).bfloat16()
    got, w = torch.empty(2, H, dtype=torch.bfloat16, device=DEV), torch.rand(2, 2, device=DEV, generator=gen(4))
    dg.dg_moe_combine(y, rows, got, weights=w)
    check_sum(got, *B.combine(y, rows, w, None), 2)
    dw = torch.empty(2, 2, device=DEV)
    dy = torch.zeros_like(y)
    dg.dg_moe_combine_backward(got, rows, dy, weights=w, y=y, dweights=dw)
    for t in range(2):
        for j in range(2):
            want = got[t].double() * w[t, j].double()
            assert ((dy[rows[t, j]].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -22) * want.abs()).all()
    assert int((dy != 0).any(1).sum()) == 4
