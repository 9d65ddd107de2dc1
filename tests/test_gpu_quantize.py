"""The token quantizer on the GPU: codes and scales equal to the exact
rounding of the definition, at every register form of the kernel, odd
pitches and alignments, ties, zeros, infinities, NaN and subnormals."""
import pytest
import torch

import tiled_layout_algebra_amd as tla
from oracle import grouped as og
from tests.grouped_util import TORCH, pitched, shifted

pytestmark = pytest.mark.gpu
TYPES = [tla.BF16, tla.F16, tla.F32]


def run(x, kind, pad=0, shift=0, qpad=None, qshift=0):
    M, K = x.shape
    qpad = pad if qpad is None else qpad
    buf = torch.full((M, K + pad), float("nan")).to(TORCH[kind])
    buf[:, :K] = x
    Q = shifted(torch.full((M * (K + qpad),), 99, dtype=torch.int8), qshift)
    s = torch.full((M,), 7.0, device="cuda")
    tla.quantize_rows(M, K, shifted(buf.reshape(-1), shift), kind, K + pad, Q, K + qpad, s)
    q = Q.cpu().view(M, K + qpad)
    assert (q[:, K:] == 99).all()
    return q[:, :K], s.cpu()


def same(x, kind, **kw):
    q, s = run(x, kind, **kw)
    wq, ws = og.quantize_rows(x)
    assert torch.equal(s.view(torch.int32)[~ws.isnan()], ws.view(torch.int32)[~ws.isnan()])
    assert torch.equal(s.isnan(), ws.isnan())
    assert torch.equal(q, wq), (q != wq).nonzero()[:4].tolist()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (5, 8), (2, 15), (9, 64), (7, 511), (6, 513), (5, 1024),
                                 (3, 2047), (2, 2049), (4, 4096), (3, 8191), (2, 8200), (1, 16385),
                                 (2, 40003), (300, 96)])
def test_sizes(kind, M, K):
    gen = torch.Generator().manual_seed(M * K)
    x = (torch.randn(M, K, generator=gen) * torch.exp(torch.randn(M, 1, generator=gen))).to(TORCH[kind])
    same(x, kind)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("pad,shift,qpad,qshift", [(1, 0, 1, 0), (0, 1, 0, 3), (5, 3, 0, 1), (8, 8, 24, 8)])
def test_pitch_and_alignment(kind, pad, shift, qpad, qshift):
    gen = torch.Generator().manual_seed(pad)
    for K in (100, 3000):
        same(torch.randn(11, K, generator=gen).to(TORCH[kind]), kind, pad=pad, shift=shift, qpad=qpad,
             qshift=qshift)


@pytest.mark.parametrize("kind", TYPES)
def test_ties_go_to_even(kind):
    """amax 127 gives scale 1 up to its last place, so halves are ties or
    next to ties; also halves of other scales, one step to either side."""
    half = torch.arange(-126.5, 127.0, 1.0)
    x = torch.cat([half, torch.tensor([127.0])]).repeat(6, 1)
    x = x * torch.tensor([1.0, 0.5, 2.0, 2.0 ** -10, 4.0, 1.5])[:, None]
    same(x.to(TORCH[kind]), kind)
    if kind == tla.F32:
        up = torch.nextafter(x, torch.full_like(x, 9e9))
        down = torch.nextafter(x, torch.full_like(x, -9e9))
        same(up, kind)
        same(down, kind)


@pytest.mark.parametrize("kind", TYPES)
def test_special_rows(kind):
    x = torch.randn(7, 300, generator=torch.Generator().manual_seed(2))
    x[0] = 0
    x[1, 17] = float("inf")
    x[2, 299] = float("nan")
    x[3, 0] = float("-inf")
    x[4] = -0.0
    x[5, 1:] = 0
    same(x.to(TORCH[kind]), kind)


def test_subnormal_scales():
    """fp32 rows down to the smallest subnormal, where the scale itself rounds
    to a few bits or to zero and codes reach the clamp."""
    rows = [torch.arange(-200, 200).float() * 2.0 ** -149]
    for e in (-149, -148, -140, -130, -127, -120, -101, -100, -99):
        rows.append(torch.linspace(-1, 1, 400) * 127 * 2.0 ** e)
        rows.append(torch.linspace(-1, 1, 400) * 63 * 2.0 ** e)
    same(torch.stack(rows), tla.F32)


def test_codes_and_scales_feed_the_product():
    """x -> codes, scales -> int8 product: off from the product of x itself by
    at most half a code a term and the output's rounding."""
    M, N, K = 37, 96, 512
    gen = torch.Generator().manual_seed(4)
    x, w = torch.randn(M, K, generator=gen).bfloat16(), torch.randn(N, K, generator=gen).bfloat16()
    qs = []
    for t in (x, w):
        q = torch.empty(t.shape, dtype=torch.int8, device="cuda")
        s = torch.empty(t.shape[0], device="cuda")
        tla.quantize_rows(t.shape[0], K, t.cuda(), tla.BF16, K, q, K, s)
        qs.append((q, s))
    D = torch.empty(M, N, dtype=torch.float16, device="cuda")
    tla.gemm_i8(M, N, K, qs[0][0], K, qs[1][0], tla.COL_MAJOR, K, D, tla.F16, N, scale_a=qs[0][1],
                scale_b=qs[1][1])
    ref = x.double() @ w.double().t()
    sx, sw = qs[0][1].cpu().double()[:, None], qs[1][1].cpu().double()[:, None]
    bound = (sx / 2) * w.double().abs().sum(1) + (x.double().abs().sum(1)[:, None] + K * sx / 2) * sw.t() / 2
    assert ((D.cpu().double() - ref).abs() <= bound * (1 + 1e-5) + ref.abs() * 2.0 ** -10).all()


@pytest.mark.parametrize("M,K", [((1 << 26) + 5, 8), ((1 << 24) + 3, 2056)])
def test_more_rows_than_one_launch_holds(M, K):
    """A launch's threads end at 2^32, 2^26 short rows or 2^24 long ones: rows on
    both sides of that, and that every row's scale was written."""
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    x.view(torch.int16).fill_(0x3F80)  # ones
    probe = torch.tensor(sorted({0, 1, (1 << 24) - 1, 1 << 24, (1 << 24) + 1, M - 2, M - 1}), device="cuda")
    some = torch.randn(len(probe), K, generator=torch.Generator().manual_seed(K)).bfloat16()
    x[probe] = some.cuda()
    Q = torch.empty(M, K, dtype=torch.int8, device="cuda")
    s = torch.full((M,), 7.0, device="cuda")
    tla.quantize_rows(M, K, x, tla.BF16, K, Q, K, s)
    wq, ws = og.quantize_rows(some)
    assert torch.equal(Q[probe].cpu(), wq) and torch.equal(s[probe].cpu(), ws)
    assert not (s == 7.0).any()
    s[probe] = s[2].clone()
    assert (s == s[2]).all()
