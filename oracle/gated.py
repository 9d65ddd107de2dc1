"""64-bit forms of the gated feed-forward products, the block-scaled product and
its quantizer, in torch on the CPU, straight from the definitions in
include/tla.h.  Every product returns the sum of its terms' magnitudes too, which
rounding errors are measured against."""
import torch

from . import grouped

ACT_SILU = 3


def act(y, kind):
    return y * torch.sigmoid(y) if kind == ACT_SILU else grouped.act(y, kind)


def act_slope(z, kind):
    if kind == ACT_SILU:
        p = torch.sigmoid(z)
        return p + z * p * torch.sigmoid(-z)
    return grouped.act_slope(z, kind)


def expand(scale, block_rows, rows, cols):
    """A matrix of block scales, a value for each element of rows x cols."""
    s = scale.double().repeat_interleave(block_rows, dim=-2)[..., :rows, :]
    return s.repeat_interleave(128, dim=-1)[..., :cols]


def round_e4m3(x):
    """float64 to the nearest e4m3 value (as float64), ties to even, at most +-448."""
    x = x.clamp(-448, 448)
    _, e = torch.frexp(x)
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64), (e.clamp(min=-5) - 4).double())
    return torch.round(x / step) * step


def quantize_blocks(x, block_rows):
    """(values of the codes, scales): float64 quotients of fp32 values round as the
    true quotient does: they cannot come closer to a midpoint of 5 bits than 2^-29
    of it without meeting it."""
    x = x.float()
    M, K = x.shape
    mb, kb = -(-M // block_rows), -(-K // 128)
    full = torch.nn.functional.pad(x, (0, kb * 128 - K, 0, mb * block_rows - M))
    a = full.view(mb, block_rows, kb, 128).abs().amax(dim=(1, 3))
    # (amax does not hand a NaN on everywhere: asked for by itself)
    bad = full.view(mb, block_rows, kb, 128).isnan().any(dim=3).any(dim=1)
    a = torch.where(bad, torch.full_like(a, float("nan")), a)
    scale = a / 448
    ok = torch.isfinite(scale) & (scale > 0)
    by = expand(torch.where(ok, scale, torch.ones_like(scale)), block_rows, M, K)
    live = expand(ok.float(), block_rows, M, K) > 0
    q = round_e4m3(torch.where(live, x.double() / by, torch.zeros(M, K, dtype=torch.float64)))
    return q, scale
