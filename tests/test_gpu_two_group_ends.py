"""How the two-group kernel ends: whole 256-row tiles, their last k-tile in each of
the three B slots, where a wave begins its epilogue while others still multiply.
More than 128 tiles, so that they are not cut into halves.  Bounds:
tests/gated_util.py; a second call gives the same bits."""
import pytest
import torch

import tiled_layout_algebra_amd as tla
from tests.gated_util import VARIANTS, Blocks, Gated

pytestmark = pytest.mark.gpu
# 12 blocks of rows and 11 of columns; K / 128 leaves 1, 2 and 0 over three, and a block cut short
ROWS, COLUMNS, LENGTHS = 3016, 2816, (896, 640, 768, 520)


def same_again(c, out):
    first = out.clone()
    for _ in range(3):
        out.fill_(7.0)
        c.again(variant=VARIANTS["two_group"])
        torch.cuda.synchronize()
        assert torch.equal(first.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("K", LENGTHS)
def test_block_scales(K):
    c = Blocks([ROWS], COLUMNS, K, no_offsets=True).call(variant=VARIANTS["two_group"])
    c.verify()
    same_again(c, c.D)


@pytest.mark.parametrize("K", LENGTHS)
def test_block_scales_gated(K):
    c = Gated([ROWS], COLUMNS // 2, K, tla.E4M3, no_offsets=True).call(variant=VARIANTS["two_group"])
    c.verify()
    same_again(c, c.H)
