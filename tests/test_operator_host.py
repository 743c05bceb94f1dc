"""The host's side of the operators around the products (no GPU needed)."""
import ctypes
import random
import time

import moe_grouped_gemm_tma_gb300 as dg


def layer_workspace(T, k, E, H, I):
    """The expert layer's workspace from its definition: the sums of phase 2 for every number of chunks of up to nt tokens,
    in halves or in one, each half's rows (at most nt a chunk, every expert's a multiple of 4) times its parts."""
    nt, a, ctas = 16 if T <= 16 else 32 if T <= 32 else 64, T * k, 160
    cap = (a + 3 * min(a, E) + 3) // 4 * 4

    def parts(nc):
        kbs = I // 128
        total = nc * ((H + 255) // 256) * kbs
        if total == 0:
            return 1
        least = total // min(total, ctas)
        return (kbs - 1 + least - 1) // least + 1

    most = 0
    for chunks in range(1, a + 1):
        for ca in ((chunks * 5 + 7) // 8, chunks):
            cb = chunks - ca
            pa, pb = parts(ca), parts(cb) if cb else 1
            ra, rb = min(cap, ca * nt), min(cap, cb * nt)
            most = max(most, rb * pb + min(ra, cap - rb) * pa if pb >= pa else ra * pa + min(rb, cap - ra) * pb)
    up = lambda v: (v + 1023) // 1024 * 1024  # noqa: E731
    y = 4096 + up(cap * H) + up(cap * (H // 128) * 4) + up(cap * I) + up(cap * (I // 128) * 4) + ctas * 8 * nt * 256 * 4
    return y + most * ((H + 255) // 256) * 256 * 4


def test_layer_workspace_is_the_largest_that_any_routing_needs():
    rng = random.Random(1)
    for _ in range(400):
        T = rng.choice((1, 2, 7, 16, 17, 32, 33, 64, rng.randint(1, 64)))
        k = rng.randint(1, 1024 // T if rng.random() < 0.2 else 16)
        E, H, I = rng.choice((1, 2, 8, 16, 100, 256, 1024)), 128 * rng.randint(1, 56), 128 * rng.randint(1, 56)
        assert dg.load().dg_moe_layer_workspace(T, k, E, H, I) == layer_workspace(T, k, E, H, I), (T, k, E, H, I)


def test_the_sizes_of_a_large_step_take_no_longer_than_those_of_a_small_one():
    # a decode step makes this call every time: against one token and expert, 64 x 16 may cost a few times the call itself
    f, p = dg.load().dg_moe_layer, ctypes.c_void_p(0x10000)

    def shortest(T, k):
        best = 1.0
        for _ in range(500):
            t0 = time.perf_counter()
            st = f(p, p, p, p, p, p, p, None, p, p, 16, T, k, 256, 7168, 2048, 4, None)   # (refused: the workspace is too small)
            best = min(best, time.perf_counter() - t0)
            assert st == 1
        return best

    assert shortest(64, 16) < 5 * shortest(1, 1)


def test_workspaces_are_zeroed_only_where_a_first_call_reads(monkeypatch):
    import os
    import re

    import torch
    header = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "dg.h")).read()
    zeroed = {n: int(v) for n, v in re.findall(r"enum \{ (DG_\w+_ZEROED) = (\d+) \};", header)}
    monkeypatch.setattr(torch, "empty", lambda size, **kw: torch.full((size,), 0xFF, **kw))
    for ws, n in ((dg.moe_layer_workspace(64, 8, 16, 1024, 512, device="cpu"), zeroed["DG_MOE_LAYER_ZEROED"]),
                  (dg.epilogue_backward_workspace(700, 512, device="cpu"), zeroed["DG_EPILOGUE_BACKWARD_ZEROED"])):
        assert ws.numel() > 2 * n and not ws[:n].any() and (ws[n:] == 0xFF).all()


def test_kernels_that_start_early_do_not_read_through_the_read_only_path():
    # a kernel launched to overlap the previous grid's end may not take data that this grid still writes for constant
    import os
    import re
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_grouped_gemm_tma_gb300", "csrc")
    early = []
    for f in sorted(os.listdir(csrc)):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(csrc, f)).read())
        if re.search(r"\bgrid_dependency_wait\(\);", text):
            early.append(f)
            assert not re.search(r"__ldg\(|__restrict__|ld\.global\.nc|__ldcs\(", text), f
    assert {"dg_kernel.cuh", "dg_kernel_decode.cuh", "dg_kernel_bs.cuh", "dg_route.cu", "dg_epilogue_backward.cu"} <= set(early)
