"""Inputs, calls and error bounds shared by the tests of the expert-grouped
products: pitched storage with poisoned padding, one call through the
binding, and the bound an output may be off by.

The bound counts roundings.  A sum of K products in fp32 is off by at most
(K + 4) 2^-24 S, S the sum of the terms' magnitudes (each product exact or
rounded once, K additions, the scales, the bias); int8 sums are exact and only
the conversion and the epilogue's three operations round (5 2^-24 S).  The
activation passes that on with a slope of at most 1.13 and adds its own
error: 3e-7 |z| for GELU, 1e-6 (1 + |z|) for its derivative.  The store adds
half a unit of the output's last place, finfo.eps / 2 relative, or half its
smallest subnormal."""
import torch

import tiled_layout_algebra_amd as tla
from oracle import grouped as og

TORCH = {tla.F16: torch.float16, tla.BF16: torch.bfloat16, tla.F32: torch.float32,
         tla.E4M3: torch.float8_e4m3fn, tla.I8: torch.int8}
POISON = {tla.F16: float("nan"), tla.BF16: float("nan"), tla.E4M3: float("nan"), tla.I8: 101}


def values(gen, shape, kind, std=1.0):
    if kind == tla.I8:
        return torch.randint(-127, 128, shape, generator=gen, dtype=torch.int32).to(torch.int8)
    return (torch.randn(shape, generator=gen) * std).to(TORCH[kind])


def pitched(mats, ld, kind, gap=0):
    """[groups, r, c] matrices as one flat buffer: pitch ld, gap elements
    between matrices, everything else poison.  Returns (buffer, stride)."""
    g, r, c = mats.shape
    stride = r * ld + gap
    buf = torch.full((g * stride,), 0.0).fill_(POISON[kind]).to(TORCH[kind])
    raw = torch.int8 if buf.element_size() == 1 else torch.int16
    b, m = buf.view(raw), mats.contiguous().view(raw)
    for e in range(g):
        b[e * stride:e * stride + r * ld].view(r, ld)[:, :c] = m[e]
    return buf, stride


def shifted(buf, by):
    """buf on the GPU, its first element `by` elements past an allocation's start."""
    t = torch.empty(buf.numel() + by, dtype=buf.dtype, device="cuda")
    raw = {1: torch.int8, 2: torch.int16, 4: torch.int32}[buf.element_size()]
    t.view(raw)[by:].copy_(buf.view(raw))
    return t[by:]


def offsets_of(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return out


def half_step(ref, kind):
    f = torch.finfo(TORCH[kind])
    return torch.maximum(ref.abs() * f.eps / 2, torch.tensor(f.smallest_normal * f.eps / 2,
                                                             dtype=torch.float64))


def sum_error(S, K, kind):
    return S * ((5 if kind == tla.I8 else K + 4) * 2.0 ** -24)


def check(got, ref, bound, what):
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), "%s: %d of %d off, worst %g of the bound at %s" % (
        what, int(bad.sum()), bad.numel(),
        ((got.double() - ref).abs() / bound).nan_to_num(9e9).max().item(),
        bad.nonzero()[0].tolist())


class Product:
    """One grouped product: inputs on the host, its call, its check."""

    def __init__(self, counts, N, K, kind, d_type=None, order=tla.COL_MAJOR, bias=False,
                 bias_type=None, act=tla.ACT_NONE, z=tla.Z_NONE, scales=None, pad=0, shift=0,
                 lost=0, seed=0, no_offsets=False):
        self.counts, self.N, self.K, self.kind, self.order = counts, N, K, kind, order
        self.act, self.z, self.pad, self.shift, self.no_offsets = act, z, pad, shift, no_offsets
        self.g, self.off = len(counts), offsets_of(counts)
        self.rows = self.off[-1] + lost
        self.d_type = d_type if d_type is not None else (tla.F16 if kind == tla.F16 else tla.BF16)
        gen = torch.Generator().manual_seed(seed)
        self.A = values(gen, (self.rows, K), kind)
        std = 1.0 if kind in (tla.I8, tla.E4M3) else max(K, 1) ** -0.5
        self.B = values(gen, (self.g, K, N), kind, std)
        scales = kind in (tla.I8, tla.E4M3) if scales is None else scales
        mid = (0.03 if kind == tla.I8 else 1.0)
        self.sa = mid * torch.exp(0.5 * torch.randn(self.rows, generator=gen)) if scales else None
        self.sb = (mid * max(K, 1) ** -0.5 * torch.exp(0.5 * torch.randn(self.g, N, generator=gen))
                   if scales else None)
        self.bias_type = self.d_type if bias_type is None else bias_type
        self.bias = (torch.randn(self.g, N, generator=gen).to(TORCH[self.bias_type])
                     if bias else None)
        self.Z = torch.randn(self.rows, N, generator=gen).to(TORCH[self.d_type])

    def call(self, stream=None, variant=None):
        pad, sh = self.pad, self.shift
        A, _ = pitched(self.A[None], self.K + pad, self.kind)
        kn = self.B if self.order == tla.ROW_MAJOR else self.B.view(
            torch.int8 if self.B.element_size() == 1 else torch.int16).transpose(1, 2).contiguous(
            ).view(self.B.dtype)
        ldb = kn.shape[2] + pad
        B, stride_b = pitched(kn, ldb, self.kind, gap=pad)
        ldd = self.N + pad
        self.D = shifted(torch.full((self.rows * ldd,), 7.0).to(TORCH[self.d_type]), sh)
        Z, _ = pitched(self.Z[None], ldd, self.d_type)
        if self.z == tla.Z_STORE:
            Z.fill_(7.0)
        self.Zd = shifted(Z, sh) if self.z != tla.Z_NONE else None
        off = None if self.no_offsets else torch.tensor(self.off, dtype=torch.int32).cuda()
        up = lambda t, by=0: None if t is None else shifted(t.reshape(-1), by)  # noqa: E731
        args = (self.g, self.rows, self.N, self.K, off, shifted(A, sh), self.kind, self.K + pad,
                shifted(B, sh), self.order, ldb, stride_b, self.D, self.d_type, ldd)
        kw = dict(scale_a=up(self.sa), scale_b=up(self.sb, sh), bias=up(self.bias, sh),
                  bias_type=self.bias_type, Z=self.Zd, ldz=ldd, z_mode=self.z, act=self.act)
        tla.grouped_gemm(*args, stream=stream, variant=variant, **kw)
        self.keep = (args, kw)
        return self

    def logical(self, buf):
        m = buf.cpu().view(self.rows, self.N + self.pad)
        return m[:, :self.N], m[:, self.N:]

    def expect(self):
        """[(name, reference, bound)] of the covered rows, D first."""
        z, S = og.pre_activation(self.A.float(), self.B.float(), self.off, self.sa, self.sb,
                                 self.bias)
        z, S = z[:self.off[-1]], S[:self.off[-1]]
        ez = sum_error(S, self.K, self.kind)
        if self.z == tla.Z_GRAD:
            zin = self.Z[:self.off[-1]].double()
            slope = og.act_slope(zin, self.act)
            d = z * slope
            es = 0.0 if self.act != tla.ACT_GELU else 1e-6 * (1 + zin.abs()) * z.abs()
            ed = ez * slope.abs() + es + d.abs() * 2.0 ** -23
        else:
            d = og.act(z, self.act)
            ed = 1.13 * ez + (3e-7 * z.abs() if self.act == tla.ACT_GELU else 0.0)
        out = [("D", d, ed + half_step(d.abs() + ed, self.d_type))]
        if self.z == tla.Z_STORE:
            out.append(("Z", z, ez + half_step(z.abs() + ez, self.d_type)))
        return out

    def verify(self):
        torch.cuda.synchronize()
        for (name, ref, bound), buf in zip(self.expect(), (self.D, self.Zd)):
            got, pad = self.logical(buf)
            check(got[:self.off[-1]], ref, bound, name)
            assert (pad == 7.0).all() if name == "D" or self.z == tla.Z_STORE else True
            assert (got[self.off[-1]:] == 7.0).all(), "rows of no expert were written"
