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


@pytest.mark.parametrize("kind,orders,lengths", [
    (tla.BF16, (tla.ROW_MAJOR, tla.COL_MAJOR), SHORTER), (tla.F16, (tla.ROW_MAJOR, tla.ROW_MAJOR), SHORTER),
    (tla.BF16, (tla.COL_MAJOR, tla.ROW_MAJOR), SHORTER), (tla.E4M3, (tla.ROW_MAJOR, tla.COL_MAJOR), (384, 512, 640))])
def test_ungrouped(kind, orders, lengths):
    """The same program without groups (variant 0), 264 tiles."""
    M, N = 5904, 2816
    t = {tla.BF16: torch.bfloat16, tla.F16: torch.float16, tla.E4M3: torch.float8_e4m3fn}[kind]
    gen = torch.Generator(device="cuda").manual_seed(6)
    for K in lengths:
        A, B = (torch.randn(*s, generator=gen, device="cuda").to(t) for s in ((M, K), (N, K)))
        want, size = A.double() @ B.double().t(), A.double().abs() @ B.double().abs().t()
        bound = size * ((K + 4) * 2.0 ** -24 + (2.0 ** -14 if kind == tla.E4M3 else 0.0)) + want.abs() * 2.0 ** -8
        a, b = (x if o == major else x.view(torch.int16).t().contiguous().view(t)
                for x, o, major in ((A, orders[0], tla.ROW_MAJOR), (B, orders[1], tla.COL_MAJOR)))
        first = None
        for _ in range(4):
            D = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
            tla.gemm_epilogue(M, N, K, a, kind, orders[0], a.shape[1], b, kind, orders[1], b.shape[1], D, tla.BF16,
                              tla.ROW_MAJOR, N, act=tla.ACT_NONE, variant=0)
            torch.cuda.synchronize()
            assert ((D.double() - want).abs() <= bound).all()
            assert first is None or torch.equal(first.view(torch.int16), D.view(torch.int16))
            first = D
