"""Calls whose natural grid holds 2^32 threads or more: one launch cannot, the extents
allow them.  Outputs of 0.3 to 17 GB."""
import pytest
import torch

import tiled_layout_algebra_amd as tla
from oracle import gated as oga

pytestmark = pytest.mark.gpu
NK = tla.COL_MAJOR


def test_an_expert_a_row():
    """65536 experts with one row each and 2048 columns: 2^23 workgroups of the few-row
    kernel's eight waves.  The experts share one matrix."""
    rows, N, K = 1 << 16, 2048, 16
    gen = torch.Generator(device="cuda").manual_seed(1)
    X, W = (torch.randn(*s, generator=gen, device="cuda").bfloat16() for s in ((rows, K), (2 * N, K)))
    off = torch.arange(rows + 1, dtype=torch.int32, device="cuda")
    H = torch.full((rows, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    tla.gated_gemm(rows, rows, N, K, off, X, tla.BF16, K, W, W[N:], NK, K, 0, H, tla.BF16, N)
    torch.cuda.synchronize()
    for lo in range(0, rows, 8192):
        x = X[lo:lo + 8192].double()
        g, u = x @ W[:N].double().t(), x @ W[N:].double().t()
        e = (K + 4) * 2.0 ** -24 * (x.abs().sum(1, keepdim=True) * W.double().abs().max())
        want = oga.act(g, tla.ACT_SILU) * u
        bound = 1.2 * e * (g.abs() + u.abs() + e) + want.abs() * (2.0 ** -8 + 2.0 ** -16) + 1e-30
        assert ((H[lo:lo + 8192].double() - want).abs() <= bound).all()


@pytest.mark.parametrize("gated", [True, False])
def test_no_k_and_many_elements(gated):
    """Block scales, K = 0: the biases in every row."""
    rows, N = (131075, 16384) if gated else (131100, 65536)
    gen = torch.Generator(device="cuda").manual_seed(2)
    b, up = (torch.randn(N, generator=gen, device="cuda").bfloat16() for _ in range(2))
    out = torch.full((rows, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    if gated:
        tla.gated_gemm(1, rows, N, 0, None, None, tla.E4M3, 0, None, None, NK, 0, 0, out, tla.BF16, N, b_gate=b,
                       b_up=up, act=tla.ACT_NONE)
        want = (b.double() * up.double()).bfloat16()
    else:
        tla.gemm_blocks(1, rows, N, 0, None, None, 0, None, NK, 0, None, 0, 0, None, tla.ROW_MAJOR, 0, 0, out,
                        tla.BF16, N, bias=b)
        want = b
    torch.cuda.synchronize()
    for lo in range(0, rows, 16384):
        assert (out[lo:lo + 16384] == want).all()


@pytest.mark.parametrize("K", [0, 3])
def test_short_sums_and_many_elements(K):
    """16 bits, lines shorter than a chunk: 2^32 elements and more."""
    rows, N = 131075, 32776
    gen = torch.Generator(device="cuda").manual_seed(3)
    X, W = (torch.randn(*s, generator=gen, device="cuda").bfloat16() for s in ((rows, K), (2 * N, K)))
    b, up = (torch.randn(N, generator=gen, device="cuda").bfloat16() for _ in range(2))
    H = torch.full((rows, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    tla.gated_gemm(1, rows, N, K, None, X, tla.BF16, K, W, W[N:], NK, K, 0, H, tla.BF16, N, b_gate=b, b_up=up,
                   act=tla.ACT_RELU)
    torch.cuda.synchronize()
    for lo in range(0, rows, 8192):
        assert not H[lo:lo + 8192].isnan().any()
    for r in (0, 1, 65535, 131039, 131040, rows - 1):  # (row 131040 and column 0: element 2^32 and a little)
        x = X[r].double()
        g, u = W[:N].double() @ x + b.double(), W[N:].double() @ x + up.double()
        e = (K + 4) * 2.0 ** -24 * (W.double().abs() @ x.abs()).view(2, N).amax(0) + 2.0 ** -24 * (b.abs() + up.abs())
        want = g.clamp(min=0) * u
        assert ((H[r].double() - want).abs() <= e * (g.abs() + u.abs() + e) + want.abs() * 2.0 ** -8 * 1.01 + 1e-30).all()
