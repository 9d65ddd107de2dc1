"""A feed-forward layer of experts on the grouped products: training in 16
bits and decoding in 8 bits.

    python -m tiled_layout_algebra_amd.expert_layer [rows]

Tokens are sorted by expert; expert e computes y = gelu(x W1_e + b1_e) W2_e.

Training keeps the pre-activation z (grouped_gemm, TLA_Z_STORE) and goes back
through dz = (dy W2_e^T) gelu'(z) (the same weights read in the other order,
TLA_Z_GRAD), dW = A^T dY with the bias gradient beside it (grouped_gemm_wgrad)
and dx = dz W1_e^T.  Decoding quantizes each token (quantize_rows) and takes
both products in int8 with a scale for each token and each output channel.

The module's command runs one training step and one decoding step and prints
each output's distance from the same layer in float64.
"""
import sys

import tiled_layout_algebra_amd as tla


def _check(t, what, shape):
    """Refuses what the calls below, which take dense bf16, would misread."""
    import torch
    if t.dtype is not torch.bfloat16 or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous bfloat16 tensor of shape %s" % (what, list(shape)))


class ExpertLayer:
    """Weights W1 [experts, width, hidden], b1 [experts, hidden] and W2
    [experts, hidden, width], contiguous bf16 CUDA tensors, stored [K, N] for
    their own forward product."""

    def __init__(self, W1, b1, W2):
        self.W1, self.b1, self.W2 = W1, b1, W2
        self.experts, self.width, self.hidden = g, w, h = tuple(W1.shape)
        _check(W1, "W1", (g, w, h))
        _check(b1, "b1", (g, h))
        _check(W2, "W2", (g, h, w))

    def forward(self, x, offsets):
        """y and what the backward pass needs.  x [rows, width] sorted by
        expert, offsets int32 [experts + 1]."""
        import torch
        _check(x, "x", (x.shape[0], self.width))
        g, w, h, rows = self.experts, self.width, self.hidden, x.shape[0]
        act, z = (torch.empty(rows, h, dtype=x.dtype, device=x.device) for _ in range(2))
        y = torch.empty(rows, w, dtype=x.dtype, device=x.device)
        tla.grouped_gemm(g, rows, h, w, offsets, x, tla.BF16, w, self.W1, tla.ROW_MAJOR, h, w * h,
                         act, tla.BF16, h, bias=self.b1, Z=z, ldz=h, z_mode=tla.Z_STORE,
                         act=tla.ACT_GELU)
        tla.grouped_gemm(g, rows, w, h, offsets, act, tla.BF16, h, self.W2, tla.ROW_MAJOR, w, w * h,
                         y, tla.BF16, w)
        return y, (x, act, z, offsets)

    def backward(self, dy, saved):
        """dx and the gradients (fp32) dW1, db1, dW2."""
        import torch
        x, act, z, offsets = saved
        _check(dy, "dy", tuple(x.shape))
        g, w, h, rows = self.experts, self.width, self.hidden, x.shape[0]
        dz = torch.empty(rows, h, dtype=x.dtype, device=x.device)
        dx = torch.empty_like(x)
        dW1 = torch.empty(g, w, h, device=x.device)
        db1 = torch.empty(g, h, device=x.device)
        dW2 = torch.empty(g, h, w, device=x.device)
        # W [K, N] is its transpose's column-major form: the same buffer
        tla.grouped_gemm(g, rows, h, w, offsets, dy, tla.BF16, w, self.W2, tla.COL_MAJOR, w, w * h,
                         dz, tla.BF16, h, Z=z, ldz=h, z_mode=tla.Z_GRAD, act=tla.ACT_GELU)
        tla.grouped_gemm(g, rows, w, h, offsets, dz, tla.BF16, h, self.W1, tla.COL_MAJOR, h, w * h,
                         dx, tla.BF16, w)
        tla.grouped_gemm_wgrad(g, rows, w, h, offsets, act, h, dy, w, tla.BF16, dW2, tla.F32,
                               tla.ROW_MAJOR, w, w * h)
        tla.grouped_gemm_wgrad(g, rows, h, w, offsets, x, w, dz, h, tla.BF16, dW1, tla.F32,
                               tla.ROW_MAJOR, h, w * h, dbias=db1)
        return dx, dW1, db1, dW2

    def quantize(self):
        """The weights in int8, [N, K] as the few-row kernel reads them, with a
        scale for each expert's output channel; laid out once."""
        import torch
        out = []
        for W in (self.W1, self.W2):
            nk = W.transpose(1, 2).contiguous()
            g, n, k = nk.shape
            q = torch.empty(g, n, k, dtype=torch.int8, device=W.device)
            s = torch.empty(g, n, device=W.device)
            tla.quantize_rows(g * n, k, nk, tla.BF16, k, q, k, s)
            out.append((q, s))
        self.q1, self.q2 = out
        return self

    def decode(self, x, offsets):
        """y in int8: tokens quantized, both products with their scales."""
        import torch
        _check(x, "x", (x.shape[0], self.width))
        g, w, h, rows = self.experts, self.width, self.hidden, x.shape[0]
        for k, n, (W, s), bias, act in ((w, h, self.q1, self.b1, tla.ACT_GELU),
                                        (h, w, self.q2, None, tla.ACT_NONE)):
            q = torch.empty(rows, k, dtype=torch.int8, device=x.device)
            sx = torch.empty(rows, device=x.device)
            y = torch.empty(rows, n, dtype=torch.bfloat16, device=x.device)
            tla.quantize_rows(rows, k, x, tla.BF16, k, q, k, sx)
            tla.grouped_gemm(g, rows, n, k, offsets, q, tla.I8, k, W, tla.COL_MAJOR, k, n * k, y,
                             tla.BF16, n, scale_a=sx, scale_b=s, bias=bias, act=act)
            x = y
        return x


def example(rows=1024, experts=8, width=512, hidden=1024, seed=0):
    """One training step and one decoding step; returns the largest distance
    of each output from float64, relative to that output's largest value."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).bfloat16()

    layer = ExpertLayer(normal(experts, width, hidden, std=width ** -0.5),
                        normal(experts, hidden, std=0.1),
                        normal(experts, hidden, width, std=hidden ** -0.5))
    x, dy = normal(rows, width), normal(rows, width)
    expert = torch.randint(experts, (rows,), generator=gen, device="cuda").sort().values
    offsets = torch.searchsorted(expert, torch.arange(experts + 1, device="cuda")).int()
    y, saved = layer.forward(x, offsets)
    grads = layer.backward(dy, saved)
    few = layer.quantize().decode(x, offsets)
    torch.cuda.synchronize()

    leaves = [t.double().cpu().requires_grad_() for t in (x, layer.W1, layer.b1, layer.W2)]
    xd, W1, b1, W2 = leaves
    off, parts = offsets.tolist(), []
    for e in range(experts):
        z = xd[off[e]:off[e + 1]] @ W1[e] + b1[e]
        parts.append((z * 0.5 * torch.special.erfc(-z / 2 ** 0.5)) @ W2[e])
    ref = torch.cat(parts)
    want = torch.autograd.grad((ref * dy.double().cpu()).sum(), leaves)
    out = {}
    for name, got, r in (("y", y, ref), ("dx", grads[0], want[0]), ("dW1", grads[1], want[1]),
                         ("db1", grads[2], want[2]), ("dW2", grads[3], want[3]),
                         ("y in int8", few, ref)):
        out[name] = ((got.double().cpu() - r).abs().max() / r.abs().max()).item()
    return out


if __name__ == "__main__":
    for name, err in example(int(sys.argv[1]) if len(sys.argv) > 1 else 1024).items():
        print("%-10s largest error / largest value %.2e" % (name, err))
