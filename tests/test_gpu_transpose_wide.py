"""Transposes and copies of more elements than one launch's threads, which end
at 2^32, reach: every element is in its place."""
import pytest
import torch

import tiled_layout_algebra_amd as tla

pytestmark = pytest.mark.gpu


def _bytes(M, N):
    """Rows of bytes that differ from their neighbours, made in pieces."""
    x = torch.empty(M, N, dtype=torch.uint8, device="cuda")
    for i in range(0, N, 1 << 27):
        piece = x[:, i:i + (1 << 27)]
        at = torch.arange(i, i + piece.shape[1], device="cuda") * 40503 >> 8
        for r in range(M):
            piece[r] = (at + 31 * r).to(torch.uint8)
    return x


@pytest.mark.parametrize("M,N", [(1, (1 << 29) + 7), (33, (1 << 28) + 9)])
def test_transpose(M, N):
    src = _bytes(M, N)
    dst = torch.full((N, M), 7, dtype=torch.uint8, device="cuda")
    tla.tiled_transpose(src, N, dst, M, M, N, 1)
    back = torch.full((M, N), 7, dtype=torch.uint8, device="cuda")
    tla.tiled_transpose(dst, M, back, N, N, M, 1)
    for r in range(M):
        assert torch.equal(src[r], dst[:, r]), r
    assert torch.equal(src, back)


def test_copy():
    N = (1 << 32) + 3
    src, dst = _bytes(1, N), torch.full((N + 1,), 7, dtype=torch.uint8, device="cuda")
    tla.tiled_copy(src, N, dst[1:], N, 1, N, 1)
    assert torch.equal(dst[1:], src[0]) and dst[0] == 7
