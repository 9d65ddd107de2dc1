"""The few-row kernels over rows of 2 GiB and more, whose lengths in bytes pass
31 bits: rows of zeros with a few small whole numbers at their starts, in the
middle and at their ends, so every sum is exact."""
import pytest
import torch

import tiled_layout_algebra_amd as tla

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [1 << 30, (1 << 30) + 41], ids=["dwords", "odd"])
def test_rows_past_two_gib(K):
    rows, N = 2, 2
    A = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    B = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 5, K // 2 + 1, K - 70, K - 9, K - 1], device="cuda")
    a = torch.tensor([[1, 2, 3, 4, 5, 6], [6, -5, 4, -3, 2, -1.]])
    b = torch.tensor([[1, 1, 2, 1, 3, 1], [-1, 2, 1, 2, 1, 7.]])
    A[:, at], B[:, at] = a.cuda().bfloat16(), b.cuda().bfloat16()
    D = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    args = (1, rows, N, K, None, A, tla.BF16, K, B, tla.COL_MAJOR, K, 0, D, tla.BF16, N)
    assert tla.grouped_gemm_variant(*args).startswith("grouped_few_rows")
    for variant in (None, 4, 5, 6):
        D.fill_(99)
        tla.grouped_gemm(*args, variant=variant)
        assert torch.equal(D.float().cpu(), a @ b.t()), variant
