"""What the block-scaled products keep of small terms beside two large ones that
cancel: 448 x 448 and -448 x 448 in a block of ones.

The sum is K - 2.  In fp32 it is off by at most (K + 8) 2^-24 S with S = 2 448^2 + K
(gated_util's bound for sums without the 8-bit matrix instruction): 3.3 for K = 128,
12.5 for 510, so that nearly every one counts.  The matrix instruction drops what lies
2^-14.3 to 2^-16 below a block's largest term, 3 to 10: all ones of that block."""
import pytest
import torch

import tiled_layout_algebra_amd as tla
from tests.gated_util import VARIANTS, Blocks, Gated

pytestmark = pytest.mark.gpu


def ones_and_two_large(A, mats, at):
    A.fill_(1.0)
    A[:, list(at)] = 448.0
    for W in mats:
        W.fill_(1.0)
        W[:, at[0]], W[:, at[1]] = 448.0, -448.0


def plain(counts, N, K, at):
    b = Blocks(counts, N, K)
    ones_and_two_large(b.A, [b.B], at)
    b.sa.fill_(1.0), b.sb.fill_(1.0)
    return b


def gated(counts, N, K, at):
    c = Gated(counts, N, K, tla.E4M3, act=tla.ACT_NONE)
    ones_and_two_large(c.X, c.W, at)
    c.sx.fill_(1.0), [s.fill_(1.0) for s in c.sw]
    return c


def verify_fp32(c):
    c.exact_sums = True  # (gated_util: no allowance for the matrix instruction)
    c.verify()


@pytest.mark.parametrize("make", [plain, gated])
@pytest.mark.parametrize("K,at", [(128, (3, 100)), (256, (130, 255)), (384, (0, 127)), (500, (400, 420))])
@pytest.mark.parametrize("counts", [[1], [40], [300], [1100], [200, 0, 333]])
def test_short_sums_are_fp32(make, K, at, counts):
    """Below 512 terms, whatever the number of rows: the library's choice."""
    verify_fp32(make(counts, 520, K, at).call())


@pytest.mark.parametrize("make", [plain, gated])
@pytest.mark.parametrize("variant", ["direct128", "direct64", "few64", "few32", "few16"])
def test_short_sums_by_kernel(make, variant):
    for K, at in ((128, (127, 0)), (396, (256, 390))):
        verify_fp32(make([70, 150], 200, K, at).call(variant=VARIANTS[variant]))


@pytest.mark.parametrize("make", [plain, gated])
@pytest.mark.parametrize("variant", ["few64", "few32", "few16"])
def test_few_rows_are_fp32_at_any_length(make, variant):
    for K, at in ((512, (129, 200)), (1000, (999, 900)), (777, (0, 64))):
        verify_fp32(make([5, 20], 40, K, at).call(variant=VARIANTS[variant]))
