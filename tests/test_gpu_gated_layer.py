"""The gated layer end to end.

Training against float64: a bf16 value is off by at most 2^-9 of itself.  y sums
hidden values rounded once; dx, dW and dW2 sum products of which one factor comes
from gate and up rounded once (silu' and silu'' stay below 1.1 and 0.5, so that
passes on less than twice their roundings) and one was rounded itself: at most four
roundings a term.  The largest value of a sum exceeds the root mean square of its
error's bound by far less than 4, so 16 2^-9 of the largest value covers them.

Serving, step by step: the codes are the oracle's bit for bit, the hidden layer is
within gated_util's bounds of the formula on the codes' values, and so is y on the
codes of the hidden layer that the call returned."""
import pytest
import torch

import tiled_layout_algebra_amd as tla
from oracle import gated as oga
from oracle import grouped as og
from tests.gated_util import check, half_step, hidden_bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,experts", [(3, 8), (1000, 8), (257, 1)])
def test_training_against_float64(rows, experts):
    from tiled_layout_algebra_amd.gated_layer import example
    for name, err in example(rows, experts=experts).items():
        if "e4m3" not in name:
            assert err <= 16 * 2.0 ** -9, (name, err)


def _sum(A, B, off):
    z, S = og.pre_activation(A, B, off)
    return z, S * (2.0 ** -14 + (A.shape[1] + 8) * 2.0 ** -24)


@pytest.mark.parametrize("counts,width,hidden", [([1], 256, 384), ([5, 0, 90], 200, 136), ([300, 31], 128, 1000)])
def test_serving_step_by_step(counts, width, hidden):
    from tiled_layout_algebra_amd.gated_layer import GatedLayer
    gen = torch.Generator().manual_seed(1)
    g, rows = len(counts), sum(counts)
    off = [sum(counts[:i]) for i in range(g + 1)]
    W = (torch.randn(g, 2 * hidden, width, generator=gen) * width ** -0.5).bfloat16()
    W2 = (torch.randn(g, width, hidden, generator=gen) * hidden ** -0.5).bfloat16()
    x = torch.randn(rows, width, generator=gen).bfloat16()
    layer = GatedLayer(W.cuda(), W2.cuda()).quantize()
    y, act = layer.serve(x.cuda(), torch.tensor(off, dtype=torch.int32).cuda())
    y, act = y.cpu(), act.cpu()

    def values(t, block_rows):
        q, s = oga.quantize_blocks(t, block_rows)
        return q * oga.expand(s, block_rows, *t.shape)

    def weights(t):
        return torch.stack([values(m, 128).t() for m in t])

    xv = values(x, 1)
    (gate, eg), (up, eu) = (_sum(xv, weights(t), off) for t in (W[:, :hidden], W[:, hidden:]))
    h = oga.act(gate, tla.ACT_SILU) * up
    eh = hidden_bound(gate, up, eg, eu, tla.ACT_SILU)
    check(act, h, eh + half_step(h.abs() + eh, tla.BF16), "hidden")
    z, e = _sum(values(act, 1), weights(W2), off)
    check(y, z, e + half_step(z.abs() + e, tla.BF16), "y")


def test_rows_of_no_expert():
    """No rows at all, and experts that end before the last row: what is there equals
    the same layer's results on those rows alone, and gradients without a row are zero."""
    from tiled_layout_algebra_amd.gated_layer import GatedLayer
    gen = torch.Generator().manual_seed(2)
    W = torch.randn(2, 2 * 72, 136, generator=gen).bfloat16().cuda()
    W2 = torch.randn(2, 136, 72, generator=gen).bfloat16().cuda()
    layer = GatedLayer(W, W2).quantize()
    x, dy = (torch.randn(9, 136, generator=gen).bfloat16().cuda() for _ in range(2))

    def run(x, dy, off):
        off = torch.tensor(off, dtype=torch.int32).cuda()
        y, saved = layer.forward(x, off)
        return y, layer.backward(dy, saved), layer.serve(x, off)[0]

    y, grads, few = run(x[:0], dy[:0], [0, 0, 0])
    assert y.shape == few.shape == grads[0].shape == (0, 136)
    assert not grads[1].any() and not grads[2].any()
    some, all_ = run(x[:5], dy[:5], [0, 0, 5]), run(x, dy, [0, 0, 5])
    assert torch.equal(some[0], all_[0][:5]) and torch.equal(some[2], all_[2][:5])
    assert torch.equal(some[1][0], all_[1][0][:5])
    for a, b in zip(some[1][1:], all_[1][1:]):
        assert torch.equal(a, b) and not b[0].any()


def test_command():
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-m", "tiled_layout_algebra_amd.gated_layer", "64"], capture_output=True,
                       text=True, timeout=100)
    assert r.returncode == 0 and "y in e4m3" in r.stdout, r.stderr


def test_refusals():
    from tiled_layout_algebra_amd.gated_layer import GatedLayer
    W = torch.zeros(1, 64, 32, dtype=torch.bfloat16, device="cuda")
    W2 = torch.zeros(1, 32, 32, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        GatedLayer(W.float(), W2)
    with pytest.raises(ValueError):
        GatedLayer(W[:, :63], W2)
    with pytest.raises(ValueError):
        GatedLayer(W, W2.transpose(1, 2)[:, :16])
    with pytest.raises(ValueError):
        GatedLayer(W, W2).forward(torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")[:, ::2])
