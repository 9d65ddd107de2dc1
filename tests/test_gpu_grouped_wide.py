"""Products over more columns than the workgroups of a one-dimensional launch of
every kernel reach: each call is right or refused, and the library's own choice
is right; and 8-bit [K, N] weights over many tiles."""
import pytest
import torch

import tiled_layout_algebra_amd as tla
from tests.grouped_util import Product

pytestmark = pytest.mark.gpu


def test_a_token_times_half_a_billion_columns():
    N, K = (1 << 29) + 5, 16
    a = torch.ones(1, K, dtype=torch.int8, device="cuda")
    b = torch.ones(N, K, dtype=torch.int8, device="cuda")
    d = torch.empty(1, N, dtype=torch.bfloat16, device="cuda")
    for variant in [None] + list(range(tla.GROUPED_VARIANTS)):
        d.fill_(7)
        args = (1, 1, N, K, None, a, tla.I8, K, b, tla.COL_MAJOR, K, 0, d, tla.BF16, N)
        if variant in (4, 5, 6):
            with pytest.raises(tla.TlaError) as err:
                tla.grouped_gemm(*args, variant=variant)
            assert err.value.status == tla.ERR_UNSUPPORTED
            assert (d == 7).all()
        else:
            tla.grouped_gemm(*args, variant=variant)
            assert (d == K).all(), variant


@pytest.mark.parametrize("kind", [tla.E4M3, tla.I8], ids=["e4m3", "i8"])
def test_8_bit_weights_stored_k_by_n_over_many_tiles(kind):
    for z in (tla.Z_STORE, tla.Z_GRAD):
        Product([1500, 0, 2100, 777], 2312, 320, kind, order=tla.ROW_MAJOR, bias=z == tla.Z_STORE,
                act=tla.ACT_GELU, z=z, seed=7).call().verify()
