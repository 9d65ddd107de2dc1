"""64-bit forms of the expert-grouped products, the int8 product and the
token quantizer, in torch on the CPU: one expert after another, straight from
the definitions in include/tla.h."""
import math

import torch

ACT_NONE, ACT_RELU, ACT_GELU = 0, 1, 2


def act(y, kind):
    if kind == ACT_RELU:
        return torch.where(y < 0, torch.zeros_like(y), y)
    if kind == ACT_GELU:
        return y * 0.5 * torch.special.erfc(-y / math.sqrt(2.0))
    return y


def act_slope(z, kind):
    if kind == ACT_RELU:
        return (z > 0).double()
    if kind == ACT_GELU:
        return (0.5 * torch.special.erfc(-z / math.sqrt(2.0))
                + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    return torch.ones_like(z)


def spans(offsets):
    return list(zip(offsets[:-1], offsets[1:]))


def pre_activation(A, B, offsets, scale_a=None, scale_b=None, bias=None):
    """(z, S) in float64 from A (rows x K) and B (groups x K x N): the value
    and the sum of the products' magnitudes (with the bias), which rounding
    errors are measured against.  Rows of no expert are NaN."""
    rows, N = A.shape[0], B.shape[2]
    z = torch.full((rows, N), float("nan"), dtype=torch.float64)
    S = torch.zeros((rows, N), dtype=torch.float64)
    for e, (lo, hi) in enumerate(spans(offsets)):
        a, b = A[lo:hi].double(), B[e].double()
        y, s = a @ b, a.abs() @ b.abs()
        for f in ((scale_a[lo:hi, None] if scale_a is not None else None),
                  (scale_b[e] if scale_b is not None else None)):
            if f is not None:
                y, s = y * f.double(), s * f.double().abs()
        if bias is not None:
            y, s = y + bias[e].double(), s + bias[e].double().abs()
        z[lo:hi], S[lo:hi] = y, s
    return z, S


def wgrad(A, Y, offsets):
    """(D, S, dbias, Sb): groups x K x N and groups x N, with the sums of
    magnitudes."""
    D, S, db, Sb = [], [], [], []
    for lo, hi in spans(offsets):
        a, y = A[lo:hi].double(), Y[lo:hi].double()
        D.append(a.t() @ y)
        S.append(a.abs().t() @ y.abs())
        db.append(y.sum(0))
        Sb.append(y.abs().sum(0))
    return torch.stack(D), torch.stack(S), torch.stack(db), torch.stack(Sb)


def quantize_rows(x):
    """(codes, scale): float64 quotients of fp32 values round as the true
    quotient does, because two such values cannot come closer to a half
    integer than 2^-33 of it without meeting it."""
    x = x.float()
    r = torch.tensor(1.0, dtype=torch.float32) / 127
    scale = x.abs().amax(dim=1) * r if x.shape[1] else torch.zeros(x.shape[0])
    ok = torch.isfinite(scale) & (scale > 0)
    q = torch.round(x.double() / torch.where(ok, scale, torch.ones_like(scale)).double()[:, None])
    q = torch.where(ok[:, None], q.clamp(-127, 127), torch.zeros_like(q))
    return q.to(torch.int8), scale
