"""What the binding of the operators between the grouped products takes and refuses (no GPU needed, but for the calls it takes)."""
import pytest
import torch

import moe_grouped_gemm_tma_gb300 as dg
from tests.test_between_refusals import c

b, i, u = torch.bfloat16, torch.int32, torch.uint8


@pytest.mark.parametrize("shape", [(4, 2, 3), (4,), (8,), (4, 2, 1), (1, 4, 2), (5, 2), (3, 2)])
def test_gather_wants_rows_of_two_axes_and_as_many_as_tokens(shape):
    # (the numbers of a [4, 2, 3] would be taken as those of a [4, 2])
    with pytest.raises(ValueError):
        dg.dg_moe_gather(c(4, 128, dtype=b), None, c(*shape, dtype=i), c(16, 128, dtype=b))
    with pytest.raises(ValueError):
        dg.dg_moe_gather(c(4, 128, dtype=u), c(4, 1), c(*shape, dtype=i), c(16, 128, dtype=u), c(16, 1))
