"""Inputs, calls and error bounds shared by the tests of the gated feed-forward
products and of the block-scaled product.

Bounds.  A sum of K products in fp32 is off by at most e = (K + 4) 2^-24 S, S the
sum of the terms' magnitudes.  SiLU, GELU and ReLU have slopes of at most 1.13 and
errors of their own: the sigmoid (|z| + 4) 2^-24 and two roundings, so SiLU is off
by (|z| + 6) 2^-24 of its value; where 1 + e^-z passes 2^126 the hardware's reciprocal,
which has no subnormal results, is 0, so the sigmoid is off by at most 2^-126 there and
SiLU by |z| 2^-126 (in bf16 and fp32 a number; z < -87); GELU by 3e-7 |z|.  Derivatives: SiLU's p + z p (1
- p) by 2^-24 ((|z| + 6) (1 + |z|) p + 2), GELU's by 1e-6 (1 + |z|).  Products
pass each factor's error on times the other factor and round once (2^-24); a
store adds half a unit of the output's last place.

Block-scaled sums on the 8-bit matrix instruction: within a block of 128 it drops
from each term what lies below 2^-16 of the block's largest (measured: 2^-15.8 of
the terms' magnitudes for many terms, 2^-14.3 for two), so a block is off by at
most 2^-14 of the sum of its magnitudes where its terms are of like sizes, which
normal values are; blocks are added in fp32 with two roundings for the scales."""
import torch

import tiled_layout_algebra_amd as tla
from oracle import gated as oga
from oracle import grouped as og
from tests.grouped_util import (TORCH, check, half_step, offsets_of, pitched, shifted, values)

FEW = ("few64", "few32", "few16")
VARIANTS = {"general": 0, "two_group": 1, "direct128": 2, "direct64": 3, "few64": 4, "few32": 5,
            "few16": 6}


def act_error(z, kind):
    if kind == tla.ACT_SILU:
        return (z.abs() + 6) * 2.0 ** -24 * oga.act(z, kind).abs() + z.abs() * 2.0 ** -126
    return 3e-7 * z.abs() if kind == tla.ACT_GELU else torch.zeros_like(z)


def slope_error(z, kind):
    if kind == tla.ACT_SILU:
        return 2.0 ** -24 * ((z.abs() + 6) * (1 + z.abs()) * torch.sigmoid(z) + 2)  # (2^-126 is far below)
    return 1e-6 * (1 + z.abs()) if kind == tla.ACT_GELU else torch.zeros_like(z)


def hidden_bound(g, u, eg, eu, kind):
    a = oga.act(g, kind)
    return ((1.13 * eg + act_error(g, kind)) * (u.abs() + eu) + a.abs() * eu
            + (a * u).abs() * 2.0 ** -23)


def up(t, by=0):
    return None if t is None else shifted(t.reshape(-1), by)


def raw(buf, rows, cols, ld):
    """A flat device buffer's logical part and its padding, on the host."""
    m = buf.cpu()[:rows * ld].view(rows, ld)
    return m[:, :cols], m[:, cols:]


def stored(mats, order):
    """[g, K, N] matrices as they are stored: [g, N, K] for TLA_COL_MAJOR."""
    if order == tla.ROW_MAJOR:
        return mats
    v = torch.int8 if mats.element_size() == 1 else torch.int16
    return mats.view(v).transpose(1, 2).contiguous().view(mats.dtype)


def filled(n, kind, shift):
    return shifted(torch.full((n,), 7.0).to(TORCH[kind]), shift)


def block_scales(gen, rows, cols, mid):
    return mid * torch.exp(0.7 * torch.randn(rows, cols, generator=gen))


def place_scales(s, order, pad):
    """[g, r, c] scales in an order with a pitch: (buffer, pitch, distance)."""
    g, r, c = s.shape
    t = s if order == tla.ROW_MAJOR else s.transpose(1, 2)
    ld = t.shape[2] + pad
    buf = torch.full((g, t.shape[1], ld), float("nan"))
    buf[:, :, :t.shape[2]] = t
    return buf.cuda(), ld, t.shape[1] * ld


class Gated:
    """One gated product: inputs on the host, its call, its check."""

    def __init__(self, counts, N, K, kind, h_type=None, order=tla.COL_MAJOR, bias=(False, False),
                 bias_type=None, act=tla.ACT_SILU, keep=False, pad=0, shift=0, lost=0, seed=0,
                 no_offsets=False, one_buffer=False, x_order=tla.COL_MAJOR, w_order=tla.ROW_MAJOR):
        self.N, self.K, self.kind, self.order, self.act = N, K, kind, order, act
        self.keep_z, self.pad, self.shift, self.no_offsets = keep, pad, shift, no_offsets
        self.one_buffer, self.x_order, self.w_order = one_buffer, x_order, w_order
        self.g, self.off = len(counts), offsets_of(counts)
        self.rows = self.off[-1] + lost
        self.h_type = h_type if h_type is not None else (tla.F16 if kind == tla.F16 else tla.BF16)
        gen = torch.Generator().manual_seed(seed)
        std = 1.0 if kind == tla.E4M3 else max(K, 1) ** -0.5
        self.X = values(gen, (self.rows, K), kind)
        self.W = [values(gen, (self.g, K, N), kind, std) for _ in range(2)]
        self.bias_type = self.h_type if bias_type is None else bias_type
        self.b = [torch.randn(self.g, N, generator=gen).to(TORCH[self.bias_type]) if x else None
                  for x in bias]
        self.sx = None
        if kind == tla.E4M3:
            kb, nb = -(-K // 128), -(-N // 128)
            self.sx = block_scales(gen, self.rows, kb, 1.0)
            self.sw = [block_scales(gen, self.g * nb, kb, max(K, 1) ** -0.5).view(self.g, nb, kb)
                       for _ in range(2)]

    def call(self, stream=None, variant=None):
        pad, sh, N, K, rows = self.pad, self.shift, self.N, self.K, self.rows
        X, _ = pitched(self.X[None], K + pad, self.kind)
        if self.one_buffer:
            both = torch.cat([w.view(torch.int16) for w in self.W],
                             dim=2).view(self.W[0].dtype)  # [g, K, 2 N]
            kept = stored(both, self.order)
            ldw = kept.shape[2]
            W = shifted(kept.reshape(-1), sh)
            stride_w = 2 * N * K
            wg, wu = W, W[N:] if self.order == tla.ROW_MAJOR else W[N * K:]
        else:
            bufs = [pitched(stored(w, self.order), (N if self.order == tla.ROW_MAJOR else K) + pad,
                            self.kind, gap=pad) for w in self.W]
            ldw, stride_w = (N if self.order == tla.ROW_MAJOR else K) + pad, bufs[0][1]
            wg, wu = (shifted(b, sh) for b, _ in bufs)
        ldh, ldz = N + pad, 2 * N + pad
        self.H = filled(rows * ldh, self.h_type, sh)
        self.Z = filled(rows * ldz, self.h_type, sh) if self.keep_z else None
        off = None if self.no_offsets else torch.tensor(self.off, dtype=torch.int32).cuda()
        kw = dict(b_gate=up(self.b[0], sh), b_up=up(self.b[1], sh), bias_type=self.bias_type,
                  act=self.act)
        if self.keep_z:
            kw.update(Z_gate=self.Z, Z_up=self.Z[N:], ldz=ldz)
        if self.sx is not None:
            sx, ldsx, _ = place_scales(self.sx[None], self.x_order, pad)
            sg, ldsw, stride = place_scales(self.sw[0], self.w_order, pad)
            su, _, _ = place_scales(self.sw[1], self.w_order, pad)
            kw.update(scale_x=sx, sx_order=self.x_order, ldsx=ldsx, scale_gate=sg, scale_up=su,
                      sw_order=self.w_order, ldsw=ldsw, stride_sw=stride)
        self.args = (self.g, rows, N, K, off, shifted(X, sh), self.kind, K + pad, wg, wu, self.order,
                     ldw, stride_w, self.H, self.h_type, ldh)
        self.kw = kw
        tla.gated_gemm(*self.args, stream=stream, variant=variant, **kw)
        self.exact_sums = variant in (4, 5, 6)
        return self

    def again(self, **kw):
        tla.gated_gemm(*self.args, **self.kw, **kw)

    def sums(self):
        """[(value, error)] of gate and up."""
        out = []
        X = self.X.float().double()
        if self.sx is not None:
            X = X * oga.expand(self.sx, 1, self.rows, self.K)
        for i in range(2):
            W = self.W[i].float().double()
            if self.sx is not None:
                W = W * oga.expand(self.sw[i], 128, self.N, self.K).transpose(1, 2)
            z, S = og.pre_activation(X, W, self.off, bias=self.b[i])
            e = S * ((self.K + 8) * 2.0 ** -24)
            if self.sx is not None and not self.exact_sums:
                e = e + S * 2.0 ** -14
            n = self.off[-1]
            out.append((z[:n], e[:n]))
        return out

    def verify(self):
        torch.cuda.synchronize()
        (g, eg), (u, eu) = self.sums()
        n, N = self.off[-1], self.N
        h = oga.act(g, self.act) * u
        eh = hidden_bound(g, u, eg, eu, self.act)
        got, pad = raw(self.H, self.rows, N, N + self.pad)
        check(got[:n], h, eh + half_step(h.abs() + eh, self.h_type), "H")
        assert (pad == 7.0).all() and (got[n:] == 7.0).all()
        if self.keep_z:
            got, pad = raw(self.Z, self.rows, 2 * N, 2 * N + self.pad)
            for name, z, e, m in (("Z_gate", g, eg, got[:, :N]), ("Z_up", u, eu, got[:, N:])):
                check(m[:n], z, e + half_step(z.abs() + e, self.h_type), name)
            assert (pad == 7.0).all() and (got[n:] == 7.0).all()


class Grad:
    """One gradient of the gated product."""

    def __init__(self, counts, N, K, kind, d_type=None, order=tla.COL_MAJOR, act=tla.ACT_SILU,
                 hidden=True, pad=0, shift=0, lost=0, seed=0, no_offsets=False, z_std=1.5):
        self.N, self.K, self.kind, self.order, self.act = N, K, kind, order, act
        self.hidden, self.pad, self.shift, self.no_offsets = hidden, pad, shift, no_offsets
        self.g, self.off = len(counts), offsets_of(counts)
        self.rows = self.off[-1] + lost
        self.d_type = d_type if d_type is not None else kind
        gen = torch.Generator().manual_seed(seed)
        self.dY = values(gen, (self.rows, K), kind)
        self.W = values(gen, (self.g, K, N), kind, max(K, 1) ** -0.5)
        self.Z = (z_std * torch.randn(self.rows, 2 * N, generator=gen)).to(TORCH[self.d_type])

    def call(self, stream=None, variant=None):
        pad, sh, N, K, rows = self.pad, self.shift, self.N, self.K, self.rows
        dY, _ = pitched(self.dY[None], K + pad, self.kind)
        kept = stored(self.W, self.order)
        ldw = kept.shape[2] + pad
        W, stride_w = pitched(kept, ldw, self.kind, gap=pad)
        ldz, ldd, ldh = 2 * N + pad, 2 * N + pad, N + pad
        Z, _ = pitched(self.Z[None], ldz, self.d_type)
        Z = shifted(Z, sh)
        self.D = filled(rows * ldd, self.d_type, sh)
        self.H = filled(rows * ldh, self.d_type, sh) if self.hidden else None
        off = None if self.no_offsets else torch.tensor(self.off, dtype=torch.int32).cuda()
        self.args = (self.g, rows, N, K, off, shifted(dY, sh), self.kind, K + pad, shifted(W, sh),
                     self.order, ldw, stride_w, Z, Z[N:], ldz, self.D, self.D[N:], self.d_type, ldd)
        self.kw = dict(H=self.H, ldh=ldh, act=self.act)
        tla.gated_gemm_grad(*self.args, stream=stream, variant=variant, **self.kw)
        return self

    def again(self, **kw):
        tla.gated_gemm_grad(*self.args, **self.kw, **kw)

    def expect(self):
        """[(name, value, error)] of dZ_gate, dZ_up, H."""
        n, N = self.off[-1], self.N
        dh, S = og.pre_activation(self.dY.float(), self.W.float(), self.off)
        dh, e = dh[:n], S[:n] * ((self.K + 4) * 2.0 ** -24)
        g, u = self.Z[:n, :N].double(), self.Z[:n, N:].double()
        a, s = oga.act(g, self.act), oga.act_slope(g, self.act)
        ea, es = act_error(g, self.act), slope_error(g, self.act)
        dg, du = dh * u * s, dh * a
        return [("dZ_gate", dg, e * (u * s).abs() + (dh.abs() + e) * u.abs() * es + dg.abs() * 2.0 ** -22),
                ("dZ_up", du, e * a.abs() + (dh.abs() + e) * ea + du.abs() * 2.0 ** -22),
                ("H", a * u, ea * u.abs() + (a * u).abs() * 2.0 ** -23)]

    def verify(self):
        torch.cuda.synchronize()
        n, N = self.off[-1], self.N
        got, pad = raw(self.D, self.rows, 2 * N, 2 * N + self.pad)
        parts = [got[:, :N], got[:, N:]]
        assert (pad == 7.0).all() and (got[n:] == 7.0).all()
        if self.hidden:
            h, pad = raw(self.H, self.rows, N, N + self.pad)
            parts.append(h)
            assert (pad == 7.0).all() and (h[n:] == 7.0).all()
        for (name, want, e), m in zip(self.expect(), parts):
            check(m[:n], want, e + half_step(want.abs() + e, self.d_type), name)


class Blocks:
    """One block-scaled product."""

    def __init__(self, counts, N, K, d_type=tla.BF16, bias=False, bias_type=None, act=tla.ACT_NONE,
                 pad=0, shift=0, lost=0, seed=0, no_offsets=False, a_order=tla.COL_MAJOR,
                 b_order=tla.ROW_MAJOR):
        self.N, self.K, self.d_type, self.act = N, K, d_type, act
        self.pad, self.shift, self.no_offsets = pad, shift, no_offsets
        self.a_order, self.b_order = a_order, b_order
        self.g, self.off = len(counts), offsets_of(counts)
        self.rows = self.off[-1] + lost
        gen = torch.Generator().manual_seed(seed)
        kb, nb = -(-K // 128), -(-N // 128)
        self.A = values(gen, (self.rows, K), tla.E4M3, 2.0)
        self.B = values(gen, (self.g, K, N), tla.E4M3, 2.0)
        self.sa = block_scales(gen, self.rows, kb, 1.0)
        self.sb = block_scales(gen, self.g * nb, kb, max(K, 1) ** -0.5).view(self.g, nb, kb)
        self.bias_type = d_type if bias_type is None else bias_type
        self.bias = torch.randn(self.g, N, generator=gen).to(TORCH[self.bias_type]) if bias else None

    def call(self, stream=None, variant=None):
        pad, sh, N, K, rows = self.pad, self.shift, self.N, self.K, self.rows
        A, _ = pitched(self.A[None], K + pad, tla.E4M3)
        B, stride_b = pitched(stored(self.B, tla.COL_MAJOR), K + pad, tla.E4M3, gap=pad)
        sa, ldsa, _ = place_scales(self.sa[None], self.a_order, pad)
        sb, ldsb, stride_sb = place_scales(self.sb, self.b_order, pad)
        self.D = filled(rows * (N + pad), self.d_type, sh)
        off = None if self.no_offsets else torch.tensor(self.off, dtype=torch.int32).cuda()
        self.args = (self.g, rows, N, K, off, shifted(A, sh), K + pad, sa, self.a_order, ldsa,
                     shifted(B, sh), K + pad, stride_b, sb, self.b_order, ldsb, stride_sb, self.D,
                     self.d_type, N + pad)
        self.kw = dict(bias=up(self.bias, sh), bias_type=self.bias_type, act=self.act)
        tla.gemm_blocks(*self.args, stream=stream, variant=variant, **self.kw)
        self.exact_sums = variant in (4, 5, 6)
        return self

    def again(self, **kw):
        tla.gemm_blocks(*self.args, **self.kw, **kw)

    def verify(self):
        torch.cuda.synchronize()
        n, N = self.off[-1], self.N
        A = self.A.float().double() * oga.expand(self.sa, 1, self.rows, self.K)
        B = self.B.float().double() * oga.expand(self.sb, 128, N, self.K).transpose(1, 2)
        z, S = og.pre_activation(A, B, self.off, bias=self.bias)
        z, S = z[:n], S[:n]
        e = S * ((self.K + 8) * 2.0 ** -24 + (0.0 if self.exact_sums else 2.0 ** -14))
        d = oga.act(z, self.act)
        e = 1.13 * e + act_error(z, self.act) + d.abs() * 2.0 ** -24
        got, pad = raw(self.D, self.rows, N, N + self.pad)
        check(got[:n], d, e + half_step(d.abs() + e, self.d_type), "D")
        assert (pad == 7.0).all() and (got[n:] == 7.0).all()
