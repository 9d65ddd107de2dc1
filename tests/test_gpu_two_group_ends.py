"""How the two-group kernel ends: whole 256-row tiles, their last k-tile in each of
the three B slots, where a wave begins its epilogue while others still multiply.
More than 128 tiles, so that they are not cut into halves.  Bounds:
tests/gated_util.py; a second call gives the same bits."""
import pytest
import torch

import tiled_layout_algebra_amd as tla
from tests.gated_util import VARIANTS, Blocks, Gated, Grad
from tests.grouped_util import Product

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


# in 16 bits a k-tile is 64 of K
SHORTER = (192, 256, 320, 200)
NK, KN = tla.COL_MAJOR, tla.ROW_MAJOR


@pytest.mark.parametrize("order", [NK, KN])
@pytest.mark.parametrize("K", SHORTER)
def test_gated(K, order):
    c = Gated([ROWS], COLUMNS // 2, K, tla.BF16, order=order, no_offsets=True, keep=True)
    c.call(variant=VARIANTS["two_group"]).verify()
    same_again(c, c.H)


@pytest.mark.parametrize("order", [NK, KN])
@pytest.mark.parametrize("K", SHORTER)
def test_gradient(K, order):
    c = Grad([ROWS], COLUMNS, K, tla.BF16, order=order, no_offsets=True)
    c.call(variant=VARIANTS["two_group"]).verify()
    same_again(c, c.D)


@pytest.mark.parametrize("kind,order,variant,lengths", [
    (tla.BF16, NK, 1, SHORTER), (tla.F16, KN, 1, SHORTER), (tla.I8, NK, 1, LENGTHS), (tla.E4M3, NK, 1, LENGTHS),
    (tla.BF16, NK, 7, (144, 192, 240, 200)), (tla.E4M3, NK, 7, (576, 672, 768, 520))])
def test_grouped(kind, order, variant, lengths):
    for K in lengths:
        c = Product([ROWS], COLUMNS, K, kind, order=order, no_offsets=True).call(variant=variant)
        c.verify()
        first = c.D.clone()
        for _ in range(3):
            c.D.fill_(7.0)
            tla.grouped_gemm(*c.keep[0], **c.keep[1], variant=variant)
            torch.cuda.synchronize()
            assert torch.equal(first.view(torch.int16), c.D.view(torch.int16))
