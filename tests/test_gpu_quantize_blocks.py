"""The e4m3 block quantizer on the GPU: codes bit for bit against the exactly
rounded quotient in 64 bits."""
import pytest
import torch

import tiled_layout_algebra_amd as tla
from oracle import gated as oga
from tests.grouped_util import TORCH, shifted

pytestmark = pytest.mark.gpu


def run(x, kind, block_rows, order=tla.COL_MAJOR, padx=0, padq=0, shift=0, pads=0):
    M, K = x.shape
    kb, mb = -(-K // 128), -(-M // block_rows)
    X = torch.full((M, K + padx), float("nan"), dtype=TORCH[kind])
    X[:, :K] = x
    Xd = shifted(X.reshape(-1), shift)
    Q = torch.full((M * (K + padq) + shift,), 0x55, dtype=torch.uint8, device="cuda")[shift:]
    r, c = (mb, kb) if order == tla.ROW_MAJOR else (kb, mb)
    S = torch.full((r, c + pads), -1.0, device="cuda")
    tla.quantize_blocks(M, K, Xd, kind, K + padx, block_rows, Q, K + padq, S, order, c + pads)
    torch.cuda.synchronize()
    Q, S = Q.cpu().view(M, K + padq), S.cpu()
    assert (Q[:, K:] == 0x55).all() and (S[:, c:] == -1).all()
    S = S[:, :c] if order == tla.ROW_MAJOR else S[:, :c].t()
    return Q[:, :K], S


def verify(x, kind, block_rows, **kw):
    x = x.to(TORCH[kind])
    q, s = run(x, kind, block_rows, **kw)
    want, scale = oga.quantize_blocks(x, block_rows)
    assert torch.equal(s.nan_to_num(7.5), scale.nan_to_num(7.5))
    got = q.contiguous().view(torch.float8_e4m3fn).double()
    assert torch.equal(got, want), (got - want).abs().max()


@pytest.mark.parametrize("kind", [tla.F16, tla.BF16, tla.F32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 64), (64, 128), (129, 200), (17, 1000), (260, 2056), (5, 4111)])
def test_codes(kind, block_rows, M, K):
    gen = torch.Generator().manual_seed(M * 7 + K)
    x = torch.randn(M, K, generator=gen) * torch.exp(torch.randn(M, 1, generator=gen))
    verify(x, kind, block_rows)
    verify(x, kind, block_rows, order=tla.ROW_MAJOR, padx=3, padq=5, shift=1, pads=2)


@pytest.mark.parametrize("kind", [tla.F16, tla.BF16, tla.F32])
def test_ties_and_neighbours(kind):
    """Quotients at midpoints of two codes and one unit of x to either side, with
    scales that are and are not powers of two."""
    codes = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mids = torch.cat([(codes[:-1] + codes[1:]) / 2, codes])
    rows = []
    for top in (448.0, 1.0, 3.7, 0.0123, 611.0):
        t = torch.tensor(top).to(TORCH[kind]).float()
        s = t / 448
        v = (mids * s).to(TORCH[kind])
        raw = torch.int32 if kind == tla.F32 else torch.int16
        bits = v.view(raw)
        for d in (-1, 0, 1):
            n = (bits + d).clamp(min=0).view(TORCH[kind]).float().clamp(max=t.item())
            row = torch.zeros(3 * 128)
            # each block holds its maximum, so that its scale is s
            for b in range(3):
                part = n[127 * b:127 * (b + 1)]
                row[128 * b:128 * b + part.numel()] = part
                row[128 * b + 127] = t
            rows += [row, -row]
    verify(torch.stack(rows), kind, 1)


def test_every_e4m3_value_comes_back():
    """A power-of-two scale hands codes through, subnormal ones among them."""
    codes = torch.arange(0, 256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    codes = codes[~codes.isnan()]
    x = torch.zeros(2, 128)
    x[0, :127], x[1, :127] = codes[:127], codes[127:]
    x[:, 127] = 448
    for f in (1.0, 2.0 ** -8, 2.0 ** 6):
        q, s = run((x * f).to(torch.float32), tla.F32, 1)
        assert torch.equal(q.contiguous().view(torch.float8_e4m3fn).float(), x) and (s == f).all()


@pytest.mark.parametrize("block_rows", [1, 128])
def test_zeros_infinities_and_small_scales(block_rows):
    gen = torch.Generator().manual_seed(5)
    x = torch.randn(300, 400, generator=gen)
    x[0:130, 0:128] = 0
    x[140, 130], x[141, 300], x[270, 5] = float("inf"), float("nan"), -float("inf")
    q, s = run(x, tla.F32, block_rows)
    want, scale = oga.quantize_blocks(x, block_rows)
    assert torch.equal(s.nan_to_num(7.5, 8.5), scale.nan_to_num(7.5, 8.5))
    assert torch.equal(q.contiguous().view(torch.float8_e4m3fn).double(), want)
    for e in (-95, -118, -126, -135, -140, -146, -149):
        t = torch.randn(140, 256, generator=gen) * 2.0 ** e
        verify(t, tla.F32, block_rows)
    verify(torch.randn(140, 256, generator=gen) * 2e38 / 8, tla.F32, block_rows)


def test_shared_buffers_and_graph():
    """A captured call over changing inputs."""
    M, K = 33, 640
    X = torch.randn(M, K, device="cuda", dtype=torch.bfloat16)
    Q = torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda")
    S = torch.empty(5, M, device="cuda")
    call = lambda: tla.quantize_blocks(M, K, X, tla.BF16, K, 1, Q, K, S, tla.COL_MAJOR, M)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(4):
        X.copy_(torch.randn(M, K, device="cuda") * (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        want, scale = oga.quantize_blocks(X.cpu(), 1)
        assert torch.equal(Q.cpu().double(), want) and torch.equal(S.cpu().t(), scale)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_offsets_past_32_bits(block_rows):
    """Rows 128 MiB apart, codes 64 MiB apart, scales far apart."""
    M, K, ldx, ldq, lds = 70, 300, 1 << 25, 1 << 26, 1 << 24
    gen = torch.Generator().manual_seed(8)
    x = torch.randn(M, K, generator=gen)
    X = torch.empty(M * ldx, device="cuda")
    X.view(M, ldx)[:, :K] = x.cuda()
    Q = torch.empty(M * ldq, dtype=torch.uint8, device="cuda")
    S = torch.empty(M * lds, device="cuda")
    tla.quantize_blocks(M, K, X, tla.F32, ldx, block_rows, Q, ldq, S, tla.ROW_MAJOR, lds)
    torch.cuda.synchronize()
    want, scale = oga.quantize_blocks(x, block_rows)
    got = Q.view(M, ldq)[:, :K].cpu().contiguous().view(torch.float8_e4m3fn).double()
    assert torch.equal(got, want)
    assert torch.equal(S.view(M, lds)[:scale.shape[0], :3].cpu(), scale)


@pytest.mark.parametrize("kind", [tla.F16, tla.BF16, tla.F32])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_many_blocks(kind, block_rows):
    """Enough blocks for several a lane, a row's last block short."""
    gen = torch.Generator().manual_seed(2)
    verify(torch.randn(2100, 8200, generator=gen), kind, block_rows)
