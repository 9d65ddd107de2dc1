"""A gated feed-forward layer, dense or of experts: training in 16 bits and
serving in e4m3 with block scales.

    python -m tiled_layout_algebra_amd.gated_layer [rows]

Tokens are sorted by expert; expert e computes
y = (silu(x Wg_e^T) * (x Wu_e^T)) W2_e^T, weights stored [N, K].

Training keeps gate and up (gated_gemm) but not the hidden layer, which the
backward pass computes again beside dz (gated_gemm_grad, W2 read in the other
order); dx = dz W (grouped_gemm), the weight gradients are grouped_gemm_wgrad.
Serving quantizes each token in blocks of 128 (quantize_blocks), takes both
projections and the activation in e4m3 (gated_gemm), quantizes the hidden layer
and takes the down projection in e4m3 (gemm_blocks).

The module's command runs one training step and one serving step and prints
each output's distance from the same layer in float64.
"""
import sys

import tiled_layout_algebra_amd as tla


def _check(t, what, shape):
    """Refuses what the calls below, which take dense bf16, would misread."""
    import torch
    if t.dtype is not torch.bfloat16 or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous bfloat16 tensor of shape %s" % (what, list(shape)))


def _check_offsets(offsets, experts):
    """The kernels read experts + 1 values (None, for one expert: none)."""
    if offsets is not None and offsets.numel() < experts + 1:
        raise ValueError("offsets must hold %d values" % (experts + 1))


def _up(n, to):
    return -(-n // to) * to


def quantize_tokens(x):
    """e4m3 codes [rows, width rounded up to 16] of a contiguous bf16 tensor and
    their scales [blocks of 128, rows], as gated_gemm and gemm_blocks read them."""
    import torch
    _check(x, "x", tuple(x.shape))
    rows, width = x.shape
    pitch = _up(width, 16)
    q = torch.empty(rows, pitch, dtype=torch.float8_e4m3fn, device=x.device)
    s = torch.empty(_up(width, 128) // 128, rows, device=x.device)
    tla.quantize_blocks(rows, width, x, tla.BF16, width, 1, q, pitch, s, tla.COL_MAJOR, max(rows, 1))
    return q, s


class GatedLayer:
    """Weights W [experts, 2 hidden, width] (a matrix' first half the gate's rows,
    the other the up projection's) and W2 [experts, width, hidden], contiguous
    bf16 CUDA tensors; one expert: a dense layer, offsets None."""

    def __init__(self, W, W2):
        self.experts, twice, self.width = g, t, w = tuple(W.shape)
        self.hidden = twice // 2
        _check(W, "W", (g, 2 * self.hidden, w))
        _check(W2, "W2", (g, w, self.hidden))
        self.W, self.W2 = W, W2

    def forward(self, x, offsets=None):
        """y and what the backward pass needs.  x [rows, width] sorted by
        expert, offsets int32 [experts + 1]."""
        import torch
        _check(x, "x", (x.shape[0], self.width))
        _check_offsets(offsets, self.experts)
        g, w, h, rows = self.experts, self.width, self.hidden, x.shape[0]
        act = torch.empty(rows, h, dtype=x.dtype, device=x.device)
        z = torch.empty(rows, 2 * h, dtype=x.dtype, device=x.device)
        y = torch.empty_like(x)
        tla.gated_gemm(g, rows, h, w, offsets, x, tla.BF16, w, self.W, self.W[:, h:], tla.COL_MAJOR, w,
                       2 * h * w, act, tla.BF16, h, Z_gate=z, Z_up=z[:, h:], ldz=2 * h)
        tla.grouped_gemm(g, rows, w, h, offsets, act, tla.BF16, h, self.W2, tla.COL_MAJOR, h, w * h, y,
                         tla.BF16, w)
        return y, (x, z, offsets)

    def backward(self, dy, saved):
        """dx and the gradients (fp32) dW, dW2."""
        import torch
        x, z, offsets = saved
        _check(dy, "dy", tuple(x.shape))
        g, w, h, rows = self.experts, self.width, self.hidden, x.shape[0]
        dz, act = torch.empty_like(z), torch.empty(rows, h, dtype=x.dtype, device=x.device)
        dx = torch.empty_like(x)
        dW = torch.empty(g, 2 * h, w, device=x.device)
        dW2 = torch.empty(g, w, h, device=x.device)
        # a matrix stored [N, K] is its transpose's row-major form: the same buffer
        tla.gated_gemm_grad(g, rows, h, w, offsets, dy, tla.BF16, w, self.W2, tla.ROW_MAJOR, h, w * h, z,
                            z[:, h:], 2 * h, dz, dz[:, h:], tla.BF16, 2 * h, H=act, ldh=h)
        tla.grouped_gemm(g, rows, w, 2 * h, offsets, dz, tla.BF16, 2 * h, self.W, tla.ROW_MAJOR, w,
                         2 * h * w, dx, tla.BF16, w)
        tla.grouped_gemm_wgrad(g, rows, w, 2 * h, offsets, dz, 2 * h, x, w, tla.BF16, dW, tla.F32,
                               tla.ROW_MAJOR, w, 2 * h * w)
        tla.grouped_gemm_wgrad(g, rows, h, w, offsets, dy, w, act, h, tla.BF16, dW2, tla.F32,
                               tla.ROW_MAJOR, h, w * h)
        return dx, dW, dW2

    def quantize(self):
        """The weights in e4m3 with a scale for each 128 x 128 block; laid out once."""
        import torch

        def codes(W):
            g, n, k = W.shape
            pitch, nb, kb = _up(k, 16), _up(n, 128) // 128, _up(k, 128) // 128
            q = torch.empty(g, n, pitch, dtype=torch.float8_e4m3fn, device=W.device)
            s = torch.empty(g, nb, kb, device=W.device)
            for e in range(g):
                tla.quantize_blocks(n, k, W[e], tla.BF16, k, 128, q[e], pitch, s[e], tla.ROW_MAJOR, kb)
            return q, s

        self.gate, self.up, self.down = (codes(t) for t in (self.W[:, :self.hidden],
                                                            self.W[:, self.hidden:], self.W2))
        return self

    def serve(self, x, offsets=None):
        """y and the hidden layer, both products in e4m3."""
        import torch
        _check(x, "x", (x.shape[0], self.width))
        _check_offsets(offsets, self.experts)
        g, w, h, rows = self.experts, self.width, self.hidden, x.shape[0]
        act = torch.empty(rows, h, dtype=x.dtype, device=x.device)
        y = torch.empty_like(x)
        (Wg, sg), (Wu, su), (Wd, sd) = self.gate, self.up, self.down
        q, s = quantize_tokens(x)
        tla.gated_gemm(g, rows, h, w, offsets, q, tla.E4M3, q.shape[1], Wg, Wu, tla.COL_MAJOR,
                       Wg.shape[2], h * Wg.shape[2], act, tla.BF16, h, scale_x=s,
                       sx_order=tla.COL_MAJOR, ldsx=rows, scale_gate=sg, scale_up=su,
                       sw_order=tla.ROW_MAJOR, ldsw=sg.shape[2], stride_sw=sg.shape[1] * sg.shape[2])
        q, s = quantize_tokens(act)
        tla.gemm_blocks(g, rows, w, h, offsets, q, q.shape[1], s, tla.COL_MAJOR, rows, Wd, Wd.shape[2],
                        w * Wd.shape[2], sd, tla.ROW_MAJOR, sd.shape[2], sd.shape[1] * sd.shape[2], y,
                        tla.BF16, w)
        return y, act


def reference(x, dy, W, W2, offsets):
    """The layer and its gradients in float64 on the CPU: y, dx, dW, dW2."""
    import torch
    leaves = [t.double().cpu().requires_grad_() for t in (x, W, W2)]
    xd, Wd, W2d = leaves
    off = [0, x.shape[0]] if offsets is None else offsets.tolist()
    parts, h = [], W.shape[1] // 2
    for e in range(W.shape[0]):
        z = xd[off[e]:off[e + 1]] @ Wd[e].t()
        parts.append((torch.nn.functional.silu(z[:, :h]) * z[:, h:]) @ W2d[e].t())
    y = torch.cat(parts)
    return (y, *torch.autograd.grad((y * dy.double().cpu()).sum(), leaves))


def example(rows=1024, experts=8, width=512, hidden=640, seed=0):
    """One training step and one serving step; returns the largest distance of
    each output from float64, relative to that output's largest value."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).bfloat16()

    layer = GatedLayer(normal(experts, 2 * hidden, width, std=width ** -0.5),
                       normal(experts, width, hidden, std=hidden ** -0.5))
    x, dy = normal(rows, width), normal(rows, width)
    offsets = None
    if experts > 1:
        expert = torch.randint(experts, (rows,), generator=gen, device="cuda").sort().values
        offsets = torch.searchsorted(expert, torch.arange(experts + 1, device="cuda")).int()
    y, saved = layer.forward(x, offsets)
    grads = layer.backward(dy, saved)
    few, _ = layer.quantize().serve(x, offsets)
    torch.cuda.synchronize()
    want = reference(x, dy, layer.W, layer.W2, offsets)
    out = {}
    for name, got, r in (("y", y, want[0]), ("dx", grads[0], want[1]), ("dW", grads[1], want[2]),
                         ("dW2", grads[2], want[3]), ("y in e4m3", few, want[0])):
        out[name] = ((got.double().cpu() - r).abs().max() / r.abs().max()).item()
    return out


if __name__ == "__main__":
    for name, err in example(int(sys.argv[1]) if len(sys.argv) > 1 else 1024).items():
        print("%-10s largest error / largest value %.2e" % (name, err))
