"""The gated and block-scaled entry points without a GPU: refusals come back as
status codes before any device work, no-ops need no buffers, packed arguments are
the structures', the binding refuses host tensors and wrong types, and the
64-bit oracle agrees with its definitions."""
import ctypes

import pytest
import torch

import tiled_layout_algebra_amd as tla
from oracle import gated as oga

FAKE = 1 << 20  # aligned, never dereferenced on these paths
I, U = tla.ERR_INVALID_ARG, tla.ERR_UNSUPPORTED
LARGE = (1 << 31) - 4095


def gated(**kw):
    base = dict(groups=4, rows=64, N=64, K=64, offsets=FAKE, X=FAKE, type=tla.BF16, ldx=64, W_gate=FAKE,
                W_up=FAKE, w_order=tla.COL_MAJOR, ldw=64, stride_w=4096, H=2 * FAKE, h_type=tla.BF16,
                ldh=64, b_gate=None, b_up=None, bias_type=tla.BF16, Z_gate=None, Z_up=None, ldz=64,
                scale_x=None, sx_order=tla.COL_MAJOR, ldsx=64, scale_gate=None, scale_up=None,
                sw_order=tla.ROW_MAJOR, ldsw=1, stride_sw=1, act=tla.ACT_SILU)
    base.update(kw)
    return tla.GatedGemmArgs(**base)


SCALED = dict(type=tla.E4M3, scale_x=FAKE, scale_gate=FAKE, scale_up=FAKE)


def grad(**kw):
    base = dict(groups=4, rows=64, N=64, K=64, offsets=FAKE, dY=FAKE, type=tla.BF16, ldy=64, W=FAKE,
                w_order=tla.ROW_MAJOR, ldw=64, stride_w=4096, Z_gate=2 * FAKE, Z_up=3 * FAKE, ldz=64,
                dZ_gate=4 * FAKE, dZ_up=5 * FAKE, d_type=tla.BF16, ldd=64, H=6 * FAKE, ldh=64,
                act=tla.ACT_SILU)
    base.update(kw)
    return tla.GatedGradArgs(**base)


def blocks(**kw):
    base = dict(groups=4, rows=64, N=64, K=64, offsets=FAKE, A=FAKE, lda=64, scale_a=FAKE,
                sa_order=tla.COL_MAJOR, ldsa=64, B=FAKE, ldb=64, stride_b=4096, scale_b=FAKE,
                sb_order=tla.ROW_MAJOR, ldsb=1, stride_sb=1, D=2 * FAKE, d_type=tla.BF16, ldd=64,
                bias=None, bias_type=tla.BF16, act=tla.ACT_NONE)
    base.update(kw)
    return tla.GemmBlocksArgs(**base)


SHARED = [
    (dict(groups=-1), I), (dict(rows=-1), I), (dict(N=-1), I), (dict(K=-1), I), (dict(act=4), I),
    (dict(act=-1), I), (dict(rows=LARGE), U), (dict(N=1 << 30), U), (dict(K=LARGE), U),
    (dict(groups=LARGE), U), (dict(offsets=None), I), (dict(offsets=FAKE + 2), I),
]
GATED = SHARED + [
    (dict(w_order=2), I), (dict(type=tla.F32), U), (dict(type=tla.I8), U), (dict(h_type=tla.F32), U),
    (dict(h_type=tla.F16), U), (dict(SCALED, h_type=tla.F32), U),
    (dict(b_gate=FAKE, bias_type=tla.I8), U), (dict(b_up=FAKE, bias_type=5), U),
    (dict(scale_x=FAKE), U), (dict(scale_gate=FAKE), U), (dict(scale_up=FAKE), U),
    (dict(X=None), I), (dict(W_gate=None), I), (dict(W_up=None), I), (dict(H=None), I),
    (dict(ldx=63), I), (dict(ldw=63), I), (dict(w_order=tla.ROW_MAJOR, ldw=63), I),
    (dict(stride_w=-1), I), (dict(ldh=63), I), (dict(Z_gate=FAKE), I), (dict(Z_up=FAKE), I),
    (dict(Z_gate=FAKE, Z_up=FAKE), I), (dict(Z_gate=2 * FAKE, Z_up=3 * FAKE), I),
    (dict(Z_gate=4 * FAKE, Z_up=3 * FAKE, ldz=63), I), (dict(X=FAKE + 1), I), (dict(W_up=FAKE + 1), I),
    (dict(H=FAKE + 1), I), (dict(b_gate=FAKE + 1), I), (dict(b_up=FAKE + 2, bias_type=tla.F32), I),
    (dict(SCALED, w_order=tla.ROW_MAJOR), U), (dict(SCALED, scale_x=None), I),
    (dict(SCALED, scale_up=None), I), (dict(SCALED, sx_order=2), I), (dict(SCALED, sw_order=-1), I),
    (dict(SCALED, ldsx=63), I), (dict(SCALED, ldsw=0), I), (dict(SCALED, stride_sw=-1), I),
    (dict(SCALED, sw_order=tla.COL_MAJOR, N=129, ldh=129, ldsw=1), I),
    (dict(SCALED, scale_gate=FAKE + 2), I),
]
GRAD = SHARED + [
    (dict(w_order=2), I), (dict(type=tla.F32), U), (dict(type=tla.E4M3), U), (dict(d_type=tla.F32), U),
    (dict(d_type=tla.F16), U), (dict(dY=None), I), (dict(W=None), I), (dict(Z_gate=None), I), (dict(Z_up=None), I),
    (dict(dZ_gate=None), I), (dict(dZ_up=None), I), (dict(ldy=63), I), (dict(ldw=63), I),
    (dict(ldz=63), I), (dict(ldd=63), I), (dict(ldh=63), I), (dict(stride_w=-1), I),
    (dict(dZ_gate=5 * FAKE), I), (dict(H=4 * FAKE), I), (dict(dZ_up=2 * FAKE), I), (dict(H=3 * FAKE), I),
    (dict(dY=FAKE + 1), I), (dict(Z_up=3 * FAKE + 1), I), (dict(H=6 * FAKE + 1), I),
]
BLOCKS = SHARED + [
    (dict(sa_order=2), I), (dict(sb_order=2), I), (dict(d_type=tla.F32), U),
    (dict(bias=FAKE, bias_type=tla.E4M3), U), (dict(A=None), I), (dict(B=None), I), (dict(D=None), I),
    (dict(scale_a=None), I), (dict(scale_b=None), I), (dict(lda=63), I), (dict(ldb=63), I),
    (dict(ldd=63), I), (dict(ldsa=63), I), (dict(ldsb=0), I), (dict(stride_b=-1), I),
    (dict(stride_sb=-1), I), (dict(scale_a=FAKE + 1), I), (dict(D=FAKE + 1), I),
    (dict(bias=FAKE + 1), I), (dict(sa_order=tla.ROW_MAJOR, K=129, lda=129, ldb=129, ldsa=1), I),
]


@pytest.mark.parametrize("name,make,kw,status",
                         [("gated_gemm", gated, *c) for c in GATED]
                         + [("gated_gemm_grad", grad, *c) for c in GRAD]
                         + [("gemm_blocks", blocks, *c) for c in BLOCKS])
def test_refusals(name, make, kw, status):
    a = make(**kw)
    assert getattr(tla.lib(), "tla_" + name)(ctypes.byref(a), None) == status
    assert getattr(tla.lib(), "tla_%s_run_variant" % name)(ctypes.byref(a), 1, None) == status


@pytest.mark.parametrize("name,make", [("gated_gemm", gated), ("gated_gemm_grad", grad),
                                       ("gemm_blocks", blocks)])
def test_no_work_and_variants(name, make):
    f, v = getattr(tla.lib(), "tla_" + name), getattr(tla.lib(), "tla_%s_run_variant" % name)
    for kw in (dict(groups=0), dict(rows=0), dict(N=0)):
        assert f(ctypes.byref(make(**kw)), None) == tla.OK
    assert f(None, None) == I
    for bad in (-1, tla.GROUPED_VARIANTS):
        assert v(ctypes.byref(make()), bad, None) == I
    none = {"gated_gemm": (7, 8, 9), "gated_gemm_grad": (4, 5, 6, 7), "gemm_blocks": (0, 7, 8, 9)}[name]
    for bad in none:
        assert v(ctypes.byref(make()), bad, None) == U
    # rows off a dword: no direct copies
    odd = {"gated_gemm": dict(ldx=65), "gated_gemm_grad": dict(ldy=65), "gemm_blocks": dict(lda=65)}[name]
    for bad in (1, 2, 3):
        assert v(ctypes.byref(make(**odd)), bad, None) == U
    if name == "gated_gemm":
        for bad in (1, 2, 3):
            assert v(ctypes.byref(make(W_up=FAKE + 2)), bad, None) == U
        assert v(ctypes.byref(make(w_order=tla.ROW_MAJOR)), 6, None) == U
        assert v(ctypes.byref(make(**SCALED)), 0, None) == U


QUANT = dict(M=64, K=256, X=FAKE, x_type=tla.BF16, ldx=256, block_rows=1, Q=FAKE, ldq=256, scale=FAKE,
             s_order=tla.COL_MAJOR, lds=64)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), I), (dict(K=-1), I), (dict(block_rows=2), I), (dict(block_rows=0), I), (dict(s_order=2), I),
    (dict(x_type=tla.E4M3), U), (dict(x_type=tla.I8), U), (dict(M=LARGE, lds=LARGE), U), (dict(K=LARGE), U),
    (dict(X=None), I), (dict(Q=None), I), (dict(scale=None), I), (dict(ldx=255), I), (dict(ldq=255), I),
    (dict(lds=63), I), (dict(s_order=tla.ROW_MAJOR, lds=1), I), (dict(X=FAKE + 1), I),
    (dict(x_type=tla.F32, X=FAKE + 2), I), (dict(scale=FAKE + 2), I), (dict(M=0, X=None), tla.OK),
    (dict(K=0, X=None, scale=None), tla.OK),
    (dict(K=2 ** 30 - 127, ldx=2 ** 30, ldq=2 ** 30, block_rows=128), U),
])
def test_quantizer_refusals(kw, status):
    a = tla.QuantizeBlocksArgs(**dict(QUANT, **kw))
    assert tla.lib().tla_quantize_blocks(ctypes.byref(a), None) == status
    assert tla.lib().tla_quantize_blocks(None, None) == I


def test_packed_arguments_are_the_structures():
    for pack, args in ((tla._PACK_GATED, tla.GatedGemmArgs), (tla._PACK_GATED_GRAD, tla.GatedGradArgs),
                       (tla._PACK_BLOCKS, tla.GemmBlocksArgs),
                       (tla._PACK_QUANT_BLOCKS, tla.QuantizeBlocksArgs)):
        values = [i + 1 for i in range(len(args._fields_))]
        a = args.from_buffer_copy(pack.pack(*values).ljust(ctypes.sizeof(args), b"\0"))
        assert [getattr(a, name) for name, _ in args._fields_] == values


def test_binding_refuses_host_tensors_and_types():
    t, f = torch.zeros(64, 64), torch.zeros(64, 64, dtype=torch.float64)
    with pytest.raises(ValueError):
        tla.gated_gemm(1, 64, 64, 64, None, t, tla.BF16, 64, t, t, tla.COL_MAJOR, 64, 0, t, tla.BF16, 64)
    with pytest.raises(ValueError):
        tla.quantize_blocks(64, 64, t, tla.F32, 64, 1, t, 64, t, tla.COL_MAJOR, 64)
    with pytest.raises(ValueError, match="float32"):
        tla.gemm_blocks(1, 64, 64, 64, None, None, 64, f, 0, 64, None, 64, 0, f, 0, 1, 1, None, tla.BF16, 64)
    with pytest.raises(ValueError, match="int32"):
        tla.gated_gemm_grad(1, 64, 64, 64, t, t, tla.BF16, 64, t, 0, 64, 0, t, t, 64, t, t, tla.BF16, 64)


def test_oracle_rounding():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    codes = codes[~codes.isnan()]
    assert torch.equal(oga.round_e4m3(codes), codes)
    s = codes.unique()
    mid = (s[1:] + s[:-1]) / 2
    near = oga.round_e4m3(mid)
    assert ((near - mid).abs() == (s[1:] - s[:-1]) / 2).all()
    assert (near.to(torch.float8_e4m3fn).view(torch.uint8) % 2 == 0).all()  # ties to even
    assert torch.equal(oga.round_e4m3(mid * (1 + 1e-12)), torch.where(mid > 0, s[1:], s[:-1]))


def test_oracle_quantizer():
    gen = torch.Generator().manual_seed(0)
    x = torch.randn(130, 300, generator=gen)
    for rows in (1, 128):
        q, s = oga.quantize_blocks(x, rows)
        assert s.shape == (-(-130 // rows), 3)
        back = q * oga.expand(s, rows, 130, 300)
        step = oga.expand(s, rows, 130, 300) * 2.0 ** -9
        assert ((back - x).abs() <= torch.maximum(x.abs().double() * 2.0 ** -4, step / 2) * (1 + 1e-6)).all()
        assert q.abs().max() == 448


def test_oracle_slopes():
    z = torch.linspace(-9, 9, 401, dtype=torch.float64).requires_grad_()
    for kind in range(4):
        want, = torch.autograd.grad(oga.act(z, kind).sum(), z)
        assert torch.allclose(oga.act_slope(z, kind).detach()[z != 0], want[z != 0], atol=1e-12)
