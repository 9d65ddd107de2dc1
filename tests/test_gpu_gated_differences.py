"""The gradient call against differences of the forward call itself, element by
element.  Every row is an expert of its own, so that a bias moves one element.

H(g, u) = act(g) u; the gradient call's dZ_gate = dh u act'(g) and dZ_up = dh act(g) are
held against dh (H(g + d) - H(g - d)) / 2 d and the same in u.  What the two may differ by,
f16 outputs (half a step: h = 2^-11 of a value), fp32 biases:
  roundings of the two H         |dh| h (|H+| + |H-|) / 2 d, and as much of the sums' own errors
  the difference's own error     in g: |dh u| d^2 / 6 max|act'''|, 0.31 (SiLU), 0.78 (GELU); in u none
  gate and up as they are kept   each rounded once: h |g| through act'' (0.5, 0.8) and act' (1.13),
                                 h |u| through act' (1.13)
  the gradient                   its sums and its store: gated_util's bounds"""
import pytest
import torch

import tiled_layout_algebra_amd as tla
from tests.gated_util import Gated, Grad, act_error, check, half_step, raw

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -11


@pytest.mark.parametrize("act,second,third", [(tla.ACT_SILU, 0.5, 0.31), (tla.ACT_GELU, 0.8, 0.78),
                                              (tla.ACT_NONE, 0.0, 0.0)])
@pytest.mark.parametrize("order", [tla.COL_MAJOR, tla.ROW_MAJOR])
def test_gradient_against_the_forward_call(act, second, third, order):
    rows, N, K = 40, 48, 64
    f = Gated([1] * rows, N, K, tla.F16, order=order, act=act, keep=True, bias=(True, True),
              bias_type=tla.F32).call()
    torch.cuda.synchronize()
    (g, eg), (u, eu) = f.sums()
    b = Grad([1] * rows, N, 72, tla.F16, order=order, act=act, seed=3)
    b.Z = f.Z.cpu()[:rows * 2 * N].view(rows, 2 * N).clone()
    b.call().verify()
    got, _ = raw(b.D, rows, 2 * N, 2 * N)
    dh = torch.stack([b.dY[r].double() @ b.W[r].double() for r in range(rows)])

    def forward(name, by):
        f.kw[name].add_(by)
        f.again()
        torch.cuda.synchronize()
        f.kw[name].sub_(by)  # (multiples of 2^-4: exact to an fp32 rounding, far below)
        return raw(f.H, rows, N, N)[0].double()

    for name, part, d in (("b_gate", 0, 2.0 ** -4), ("b_up", 1, 1.0)):
        hi, lo = forward(name, d), forward(name, -d)
        diff = dh * (hi - lo) / (2 * d)
        size = (g.abs() + d) * (u.abs() + d)  # |H+| and |H-| are less
        own = 1.13 * eg * (u.abs() + d) + eu * (g.abs() + d) + act_error(g.abs() + d, act) * (u.abs() + d)
        bound = dh.abs() * (2 * HALF * size + 2 * own) / (2 * d)
        if part == 0:
            bound += dh.abs() * u.abs() * (d * d / 6 * third + HALF * (second * g.abs() + 1.13))
        else:
            bound += dh.abs() * HALF * 1.13 * g.abs()
        _, want, e = b.expect()[part]
        bound += e + half_step(want.abs() + e, tla.F16)
        check(got[:, part * N:(part + 1) * N], diff, bound, name)
        # (the bound is not vacuous: it is a small part of the gradients themselves)
        assert bound.mean() < 0.03 * want.abs().mean()
