"""What the binding of the operators between the grouped products takes and refuses (no GPU needed, but for the calls it takes)."""
import pytest
import torch

import moe_grouped_gemm_tma_gb300 as dg
from tests.test_between_refusals import _Cuda, c

b, i, u = torch.bfloat16, torch.int32, torch.uint8


@pytest.mark.parametrize("shape", [(4, 2, 3), (4,), (8,), (4, 2, 1), (1, 4, 2), (5, 2), (3, 2)])
def test_gather_wants_rows_of_two_axes_and_as_many_as_tokens(shape):
    # (the numbers of a [4, 2, 3] would be taken as those of a [4, 2])
    with pytest.raises(ValueError):
        dg.dg_moe_gather(c(4, 128, dtype=b), None, c(*shape, dtype=i), c(16, 128, dtype=b))
    with pytest.raises(ValueError):
        dg.dg_moe_gather(c(4, 128, dtype=u), c(4, 1), c(*shape, dtype=i), c(16, 128, dtype=u), c(16, 1))


def test_glu_backward_without_dh_refuses_what_needs_it():
    for out in ({"q": c(2, 256, dtype=u), "sf": c(2, 2)}, {"qt": c(256, 128, dtype=u), "sft": c(256, 1)}):
        args = [out.get(n) for n in ("q", "sf", "qt", "sft", "ht", "hsft")]
        with pytest.raises(ValueError, match="need dH"):
            dg.dg_glu_backward(None, *args, Z=c(2, 256, dtype=b))
    with pytest.raises(ValueError, match="one of Z and kept"):
        dg.dg_glu_backward(None, *[None] * 4, c(128, 128, dtype=u), c(128, 1))
    with pytest.raises(ValueError, match="ht must have shape"):
        dg.dg_glu_backward(None, *[None] * 4, c(64, 128, dtype=u), c(128, 1), Z=c(2, 256, dtype=b))
    with pytest.raises(ValueError, match="Z must have shape"):
        dg.dg_glu_backward(None, *[None] * 4, c(128, 128, dtype=u), c(128, 1), Z=c(2, 257, dtype=b))
    with pytest.raises(ValueError, match="CUDA tensor"):
        dg.dg_glu_backward(None, *[None] * 4, c(128, 128, dtype=u), c(128, 1), Z=torch.empty(2, 256, dtype=b))


@pytest.mark.gpu
@pytest.mark.parametrize("kept", [False, True])
def test_glu_backward_without_dh_gives_the_transposed_activation(kept):
    from tests.test_gpu_glu import alloc, make_z, run_backward
    M, I = 200, 256
    Z = make_z(M, I)
    q, sf, codes, ksf = alloc(M, I, True)
    dg.dg_glu(Z, q, sf, codes, ksf)
    given = {"kept": codes, "kept_sf": ksf} if kept else {"Z": Z}
    want = run_backward(torch.ones(M, I, dtype=b, device="cuda"), **({"kept": codes, "ksf": ksf} if kept else {"Z": Z}))["ht"]
    ht, hsft = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    dg.dg_glu_backward(None, None, None, None, None, ht, hsft, **given)
    assert torch.equal(ht, want[0]) and torch.equal(hsft, want[1])


BIG = 2 ** 32 + 4                                 # 4, cut to 32 bits


def m(*shape, dtype=torch.float32):
    return _Cuda(torch.empty(*shape, dtype=dtype, device="meta"))


@pytest.mark.parametrize("big", [BIG, 2 ** 31, 2 ** 33 + 1])
def test_sizes_beyond_32_bits_are_refused(big):
    with pytest.raises(dg.DGError):
        dg.moe_sort_rows(big, 1, 8)
    with pytest.raises(dg.DGError):
        dg.moe_sort_rows(4, 1, big)
    with pytest.raises(dg.DGError):
        dg.moe_sort_workspace(4, big, 8)
    with pytest.raises(dg.DGError):
        dg.rmsnorm_backward_workspace(big, 8)
    calls = [
        lambda: dg.dg_moe_sort_contiguous(m(big, 1, dtype=i), m(big, 1, dtype=i), m(8, dtype=i), m(1024, dtype=i)),
        lambda: dg.dg_moe_sort_contiguous(m(4, 1, dtype=i), m(4, 1, dtype=i), m(big, dtype=i), m(1024, dtype=i)),
        lambda: dg.dg_moe_sort_masked(m(4, 1, dtype=i), m(4, 1, dtype=i), m(big, dtype=i), 8),
        lambda: dg.dg_moe_sort_masked(m(4, 1, dtype=i), m(4, 1, dtype=i), m(8, dtype=i), big),
        lambda: dg.dg_moe_sort_masked(m(4, 1, dtype=i), m(4, 1, dtype=i), m(8, dtype=i), 8 - 2 ** 32),
        lambda: dg.dg_moe_gather(m(big, 8, dtype=b), None, m(big, 0, dtype=i), m(16, 8, dtype=b)),
        lambda: dg.dg_moe_gather(m(4, 8, dtype=b), None, m(4, 2, dtype=i), m(big, 8, dtype=b)),
        lambda: dg.dg_moe_combine(m(big, 8, dtype=b), m(4, 1, dtype=i), m(4, 8, dtype=b)),
        lambda: dg.dg_moe_combine(m(16, 8, dtype=b), m(big, 1, dtype=i), m(big, 8, dtype=b)),
        lambda: dg.dg_moe_combine_backward(m(big, 8, dtype=b), m(big, 1, dtype=i), m(16, 8, dtype=b)),
        lambda: dg.dg_moe_combine_backward(m(4, 8, dtype=b), m(4, 1, dtype=i), m(big, 8, dtype=b)),
        lambda: dg.dg_rmsnorm(m(big, 8, dtype=b), m(8), y=m(big, 8, dtype=b)),
        lambda: dg.dg_rmsnorm_backward(m(big, 8, dtype=b), m(big, 8, dtype=b), m(8), m(big, 8, dtype=b)),
        lambda: dg.dg_glu(m(big, 256, dtype=b), m(big, 128, dtype=u), m(big, 1)),
        lambda: dg.dg_glu(m(8, 256, dtype=b), m(8, 128, dtype=u), m(8, 1), masked_m=m(big, dtype=i)),
        lambda: dg.dg_glu_backward(m(big, 128, dtype=b), *[None] * 6, Z=m(big, 256, dtype=b)),
        lambda: dg.dg_transpose_fp8(m(big, 128, dtype=u), m(big, 1), m(128, big, dtype=u), m(128, big // 128)),
    ]
    for n, call in enumerate(calls):
        with pytest.raises(dg.DGError):
            call()
            pytest.fail(f"call {n}")
