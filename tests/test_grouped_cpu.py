"""The expert-grouped and int8 entry points without a GPU: refusals come back
as status codes before any device work, no-ops need no buffers, the binding
refuses host tensors and wrong index types, and the 64-bit oracle agrees with
its definitions."""
import ctypes

import pytest
import torch

import tiled_layout_algebra_amd as tla
from oracle import grouped as og

FAKE = 1 << 20  # aligned, never dereferenced on these paths


def _product(**kw):
    base = dict(groups=4, rows=64, N=64, K=64, offsets=FAKE, A=FAKE, type=tla.BF16, lda=64, B=FAKE,
                b_order=tla.COL_MAJOR, ldb=64, stride_b=4096, D=2 * FAKE, d_type=tla.BF16, ldd=64,
                scale_a=None, scale_b=None, bias=None, bias_type=tla.BF16, Z=None, ldz=64,
                z_mode=tla.Z_NONE, act=tla.ACT_NONE)
    base.update(kw)
    return tla.GroupedGemmArgs(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(groups=-1), tla.ERR_INVALID_ARG),
    (dict(rows=-1), tla.ERR_INVALID_ARG),
    (dict(N=-1), tla.ERR_INVALID_ARG),
    (dict(K=-1), tla.ERR_INVALID_ARG),
    (dict(b_order=2), tla.ERR_INVALID_ARG),
    (dict(act=3), tla.ERR_INVALID_ARG),
    (dict(z_mode=3), tla.ERR_INVALID_ARG),
    (dict(z_mode=-1), tla.ERR_INVALID_ARG),
    (dict(type=tla.F32), tla.ERR_UNSUPPORTED),
    (dict(type=5), tla.ERR_UNSUPPORTED),
    (dict(d_type=tla.F32), tla.ERR_UNSUPPORTED),
    (dict(d_type=tla.I8), tla.ERR_UNSUPPORTED),
    (dict(bias=FAKE, bias_type=tla.I8), tla.ERR_UNSUPPORTED),
    (dict(scale_a=FAKE), tla.ERR_UNSUPPORTED),                 # 16-bit operands take no scales
    (dict(scale_b=FAKE), tla.ERR_UNSUPPORTED),
    (dict(type=tla.I8, K=131072, lda=131072, ldb=131072), tla.ERR_UNSUPPORTED),
    (dict(rows=1 << 31), tla.ERR_UNSUPPORTED),
    (dict(N=1 << 31), tla.ERR_UNSUPPORTED),
    (dict(groups=1 << 31), tla.ERR_UNSUPPORTED),
    (dict(offsets=None), tla.ERR_INVALID_ARG),                 # needed with more than one expert
    (dict(A=None), tla.ERR_INVALID_ARG),
    (dict(B=None), tla.ERR_INVALID_ARG),
    (dict(D=None), tla.ERR_INVALID_ARG),
    (dict(lda=63), tla.ERR_INVALID_ARG),
    (dict(ldb=63), tla.ERR_INVALID_ARG),
    (dict(b_order=tla.ROW_MAJOR, ldb=63), tla.ERR_INVALID_ARG),
    (dict(stride_b=-1), tla.ERR_INVALID_ARG),
    (dict(ldd=63), tla.ERR_INVALID_ARG),
    (dict(z_mode=tla.Z_STORE), tla.ERR_INVALID_ARG),           # Z missing
    (dict(z_mode=tla.Z_GRAD, act=tla.ACT_RELU), tla.ERR_INVALID_ARG),
    (dict(z_mode=tla.Z_STORE, Z=2 * FAKE), tla.ERR_INVALID_ARG),   # Z is D
    (dict(z_mode=tla.Z_STORE, Z=FAKE, ldz=63), tla.ERR_INVALID_ARG),
    (dict(A=FAKE + 1), tla.ERR_INVALID_ARG),                   # element alignment
    (dict(D=FAKE + 1), tla.ERR_INVALID_ARG),
    (dict(offsets=FAKE + 2), tla.ERR_INVALID_ARG),
    (dict(type=tla.I8, scale_a=FAKE + 2), tla.ERR_INVALID_ARG),
    (dict(bias=FAKE + 2, bias_type=tla.F32), tla.ERR_INVALID_ARG),
])
def test_product_refusals(kw, status):
    a = _product(**kw)
    assert tla.lib().tla_grouped_gemm(ctypes.byref(a), None) == status
    buf = ctypes.create_string_buffer(64)
    assert tla.lib().tla_grouped_gemm_variant(ctypes.byref(a), buf, 64) == status


def _variant(**kw):
    buf = ctypes.create_string_buffer(64)
    rc = tla.lib().tla_grouped_gemm_variant(ctypes.byref(_product(**kw)), buf, 64)
    assert rc == tla.OK
    return buf.value.decode()


@pytest.mark.parametrize("kw,kernel", [
    (dict(rows=1, groups=1), "grouped_few_rows_16"),
    (dict(rows=4, N=4096, K=4096, lda=4096, ldb=4096, ldd=4096, stride_b=1 << 24), "grouped_few_rows_16"),
    (dict(rows=16384, groups=8, N=4096, K=4096, lda=4096, ldb=4096, ldd=4096, stride_b=1 << 24),
     "grouped_two_group_256x256"),
    (dict(rows=16384, groups=8, N=4096, K=4096, lda=4096, ldb=4096, ldd=4096, stride_b=1 << 24,
          b_order=tla.ROW_MAJOR), "grouped_two_group_256x256"),
    (dict(rows=16384, groups=8, N=4096, K=4095, lda=4095, ldb=4095, ldd=4096, stride_b=4095 * 4096),
     "grouped_two_group_shift_256x256"),
    (dict(rows=16384, groups=8, N=4095, K=4096, lda=4096, ldb=4095, ldd=4095, stride_b=4095 * 4096,
          b_order=tla.ROW_MAJOR), "grouped_general_128x128"),
    (dict(rows=500, N=1024, K=1024, lda=1024, ldb=1024, ldd=1024, stride_b=1 << 20,
          b_order=tla.ROW_MAJOR), "grouped_direct_128x128"),
    (dict(rows=2048, groups=32, N=2048, K=4096, lda=4096, ldb=4096, ldd=2048, stride_b=1 << 23),
     "grouped_direct_64x128"),
    (dict(rows=4096, type=tla.I8, N=1024, K=1024, lda=1024, ldb=1024, ldd=1024, stride_b=1 << 20,
          b_order=tla.ROW_MAJOR), "grouped_general_128x128"),
    (dict(rows=4096, type=tla.E4M3, K=256, lda=256, ldb=256, N=1024, ldd=1024, stride_b=1 << 18),
     "grouped_general_128x128"),
    (dict(K=0, A=None, B=None), "grouped_general_128x128"),
])
def test_kernel_choice(kw, kernel):
    assert _variant(**kw) == kernel


def test_run_variant_refusals():
    f = tla.lib().tla_grouped_gemm_run_variant
    for v in (-1, tla.GROUPED_VARIANTS):
        assert f(ctypes.byref(_product()), v, None) == tla.ERR_INVALID_ARG
    assert f(ctypes.byref(_product(rows=-1)), 0, None) == tla.ERR_INVALID_ARG
    assert f(ctypes.byref(_product(rows=0)), 3, None) == tla.OK
    kn, odd = dict(b_order=tla.ROW_MAJOR), dict(K=63, lda=63, ldb=63)
    wide = dict(lda=1 << 22, ldb=1 << 22)  # rows 8 MiB apart
    e4m3 = dict(type=tla.E4M3)
    for v, bad in ((1, [odd, wide, e4m3, dict(K=0), dict(A=FAKE + 2), dict(stride_b=4097)]),
                   (2, [odd, dict(kn, ldb=65), dict(kn, type=tla.I8)]), (3, [kn, odd, dict(B=FAKE + 2)]),
                   (4, [kn, dict(K=0)]), (5, [kn]), (6, [kn]), (7, [kn, wide, e4m3, dict(K=0)]), (8, [kn, wide]), (9, [kn, e4m3])):
        for kw in bad:
            assert f(ctypes.byref(_product(**kw)), v, None) == tla.ERR_UNSUPPORTED, (v, kw)


def test_noops_and_small_buffers():
    L = tla.lib()
    for kw in (dict(rows=0), dict(N=0), dict(groups=0)):
        a = _product(A=None, B=None, D=None, offsets=None, **kw)
        assert L.tla_grouped_gemm(ctypes.byref(a), None) == tla.OK
        assert _variant(A=None, B=None, D=None, offsets=None, **kw) == "noop"
    assert L.tla_grouped_gemm(None, None) == tla.ERR_INVALID_ARG
    assert L.tla_gemm_i8(None, None) == tla.ERR_INVALID_ARG
    assert L.tla_grouped_gemm_wgrad(None, None) == tla.ERR_INVALID_ARG
    assert L.tla_grouped_gemm_variant(ctypes.byref(_product()), None, 64) == tla.ERR_INVALID_ARG
    buf = ctypes.create_string_buffer(b"xxxxxxxx", 8)
    assert L.tla_grouped_gemm_variant(ctypes.byref(_product()), buf, 4) == tla.OK
    assert len(buf.value) == 3
    # one expert needs no offsets, no K needs no operands, the identity no Z
    assert _variant(groups=1, offsets=None) != "noop"
    assert _variant(K=0, A=None, B=None) != "noop"
    assert _variant(z_mode=tla.Z_GRAD, act=tla.ACT_NONE) != "noop"


def _i8(**kw):
    base = dict(M=8, N=64, K=64, A=FAKE, lda=64, B=FAKE, b_order=tla.COL_MAJOR, ldb=64, D=FAKE,
                d_type=tla.BF16, ldd=64, scale_a=None, scale_b=None, bias=None, bias_type=tla.BF16,
                act=tla.ACT_NONE)
    base.update(kw)
    return tla.GemmI8Args(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), tla.ERR_INVALID_ARG), (dict(K=131072, lda=131072, ldb=131072), tla.ERR_UNSUPPORTED),
    (dict(d_type=tla.F32), tla.ERR_UNSUPPORTED), (dict(lda=1), tla.ERR_INVALID_ARG),
    (dict(A=None), tla.ERR_INVALID_ARG), (dict(act=-1), tla.ERR_INVALID_ARG),
    (dict(M=0, A=None, B=None, D=None), tla.OK), (dict(N=0, A=None, B=None, D=None), tla.OK),
])
def test_int8_refusals(kw, status):
    assert tla.lib().tla_gemm_i8(ctypes.byref(_i8(**kw)), None) == status


def _wgrad(**kw):
    base = dict(groups=4, rows=64, N=64, K=32, offsets=FAKE, A=FAKE, lda=32, Y=FAKE, ldy=64,
                type=tla.BF16, D=FAKE, d_type=tla.F32, d_order=tla.ROW_MAJOR, ldd=64,
                stride_d=2048, dbias=None)
    base.update(kw)
    return tla.GroupedWgradArgs(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(groups=-1), tla.ERR_INVALID_ARG), (dict(rows=-2), tla.ERR_INVALID_ARG),
    (dict(d_order=3), tla.ERR_INVALID_ARG), (dict(type=tla.I8), tla.ERR_UNSUPPORTED),
    (dict(type=tla.E4M3), tla.ERR_UNSUPPORTED), (dict(d_type=tla.E4M3), tla.ERR_UNSUPPORTED),
    (dict(offsets=None), tla.ERR_INVALID_ARG), (dict(A=None), tla.ERR_INVALID_ARG),
    (dict(Y=None), tla.ERR_INVALID_ARG), (dict(D=None), tla.ERR_INVALID_ARG),
    (dict(lda=31), tla.ERR_INVALID_ARG), (dict(ldy=63), tla.ERR_INVALID_ARG),
    (dict(ldd=63), tla.ERR_INVALID_ARG), (dict(stride_d=2047), tla.ERR_INVALID_ARG),
    (dict(d_order=tla.COL_MAJOR, ldd=31), tla.ERR_INVALID_ARG),
    (dict(D=FAKE + 2), tla.ERR_INVALID_ARG), (dict(dbias=FAKE + 2), tla.ERR_INVALID_ARG),
    (dict(N=1 << 31), tla.ERR_UNSUPPORTED),
    (dict(groups=0), tla.OK), (dict(N=0), tla.OK), (dict(K=0), tla.OK),
])
def test_wgrad_refusals(kw, status):
    assert tla.lib().tla_grouped_gemm_wgrad(ctypes.byref(_wgrad(**kw)), None) == status


@pytest.mark.parametrize("args,status", [
    ((-1, 8, FAKE, tla.BF16, 8, FAKE, 8, FAKE), tla.ERR_INVALID_ARG),
    ((4, -8, FAKE, tla.BF16, 8, FAKE, 8, FAKE), tla.ERR_INVALID_ARG),
    ((4, 8, FAKE, tla.E4M3, 8, FAKE, 8, FAKE), tla.ERR_UNSUPPORTED),
    ((4, 8, FAKE, tla.I8, 8, FAKE, 8, FAKE), tla.ERR_UNSUPPORTED),
    ((4, 8, None, tla.BF16, 8, FAKE, 8, FAKE), tla.ERR_INVALID_ARG),
    ((4, 8, FAKE, tla.BF16, 8, None, 8, FAKE), tla.ERR_INVALID_ARG),
    ((4, 8, FAKE, tla.BF16, 8, FAKE, 8, None), tla.ERR_INVALID_ARG),
    ((4, 8, FAKE, tla.BF16, 7, FAKE, 8, FAKE), tla.ERR_INVALID_ARG),
    ((4, 8, FAKE, tla.BF16, 8, FAKE, 7, FAKE), tla.ERR_INVALID_ARG),
    ((4, 8, FAKE + 2, tla.F32, 8, FAKE, 8, FAKE), tla.ERR_INVALID_ARG),
    ((4, 8, FAKE, tla.F32, 8, FAKE, 8, FAKE + 1), tla.ERR_INVALID_ARG),
    ((0, 8, None, tla.F32, 8, None, 8, None), tla.OK),
])
def test_quantizer_refusals(args, status):
    assert tla.lib().tla_quantize_rows(*args, None) == status


def test_packed_arguments_match_the_structures():
    for fmt, cls in ((tla._PACK_GROUPED, tla.GroupedGemmArgs), (tla._PACK_WGRAD, tla.GroupedWgradArgs),
                     (tla._PACK_I8, tla.GemmI8Args)):
        assert fmt.size <= ctypes.sizeof(cls) < fmt.size + 8  # less the padding at the end
        vals = [0x101 * (i + 1) for i in range(len(cls._fields_))]
        raw = fmt.pack(*vals).ljust(ctypes.sizeof(cls), b"\0")
        a = cls.from_buffer_copy(raw)
        assert [getattr(a, name) for name, _ in cls._fields_] == vals


def test_binding_refuses_host_tensors_and_other_index_types():
    t = torch.zeros(64)
    with pytest.raises(ValueError, match="CUDA"):
        tla.quantize_rows(1, 64, t, tla.F32, 64, t, 64, t)
    with pytest.raises(ValueError, match="int32"):
        tla.grouped_gemm(1, 1, 8, 8, torch.zeros(2, dtype=torch.int64), t, tla.BF16, 8, t,
                         tla.COL_MAJOR, 8, 64, t, tla.BF16, 8)
    with pytest.raises(ValueError, match="float32"):
        tla.gemm_i8(1, 8, 8, None, 8, None, tla.COL_MAJOR, 8, None, tla.BF16, 8,
                    scale_a=torch.zeros(1, dtype=torch.float16))


def test_oracle_against_its_definitions():
    gen = torch.Generator().manual_seed(0)
    A, B = torch.randn(7, 5, generator=gen), torch.randn(3, 5, 4, generator=gen)
    off = [0, 3, 3, 7]
    z, S = og.pre_activation(A, B, off, bias=torch.ones(3, 4))
    for r in range(7):
        e = 0 if r < 3 else 2
        for n in range(4):
            want = sum(float(A[r, k]) * float(B[e, k, n]) for k in range(5)) + 1
            assert abs(float(z[r, n]) - want) < 1e-12 and float(S[r, n]) >= abs(want)
    zz = torch.linspace(-6, 6, 101, dtype=torch.float64, requires_grad=True)
    for kind in (og.ACT_NONE, og.ACT_RELU, og.ACT_GELU):
        (slope,) = torch.autograd.grad(og.act(zz, kind).sum(), zz)
        keep = zz != 0
        assert (slope - og.act_slope(zz, kind))[keep].abs().max() < 1e-12
    D, _, db, _ = og.wgrad(A, A[:, :4], off)
    assert torch.allclose(D[2], A[3:].double().t() @ A[3:, :4].double())
    assert (D[1] == 0).all() and torch.allclose(db[0], A[:3, :4].double().sum(0))


def test_quantizer_oracle_rounds_exactly():
    """The float64 quotients against exact rational rounding."""
    from fractions import Fraction
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(4, 60, generator=gen)
    x[0, :5] = torch.tensor([127.0, 0.5, 1.5, -2.5, 63.5])
    q, s = og.quantize_rows(x)
    for r in range(4):
        for c in range(60):
            f = Fraction(float(x[r, c])) / Fraction(float(s[r]))
            assert int(q[r, c]) == max(-127, min(127, round(f)))


def test_slabs_of_k_rows_stay_within_32_bit_offsets():
    """[K, N] weights: a slab holds 64 rows of k however few there are, so the
    direct copies need 64 pitches below 2^31 bytes, and K of them."""
    kn = dict(b_order=tla.ROW_MAJOR, lda=64)
    f = tla.lib().tla_grouped_gemm_run_variant
    for K, ldb in ((8, 1 << 24), (8, 1 << 26), (1, 1 << 30), (64, 1 << 24), (100, 1 << 24), (8, 1 << 62)):
        kw = dict(kn, K=K, ldb=ldb, lda=(K + 7) & ~7, groups=1)
        assert _variant(**kw) == "grouped_general_128x128"
        for v in (1, 2):
            assert f(ctypes.byref(_product(**kw)), v, None) == tla.ERR_UNSUPPORTED
    assert _variant(**dict(kn, K=64, ldb=(1 << 24) - 8, groups=1)) == "grouped_direct_128x128"
    # pitches that no 64-bit count of bytes holds
    assert f(ctypes.byref(_product(groups=1, rows=1, lda=1 << 62)), 1, None) == tla.ERR_UNSUPPORTED
    assert f(ctypes.byref(_product(groups=1, N=1, ldb=1 << 62)), 2, None) == tla.ERR_UNSUPPORTED


@pytest.mark.parametrize("name", ["groups", "rows", "N", "K"])
def test_extents_leave_room_for_the_kernels_counts(name):
    """Counts of tiles and of experts taken 64 at a time run in 32 bits, up to a
    tile past the extent: extents end 4096 short of 2^31."""
    most = (1 << 31) - 4096
    wide = dict(groups=1, rows=1, lda=most, ldb=most, ldd=most, stride_b=0)
    L = tla.lib()
    buf = ctypes.create_string_buffer(64)
    assert L.tla_grouped_gemm_variant(ctypes.byref(_product(**dict(wide, **{name: most}))), buf, 64) == tla.OK
    over = dict(wide, lda=1 << 31, ldb=1 << 31, ldd=1 << 31, **{name: most + 1})
    assert L.tla_grouped_gemm_variant(ctypes.byref(_product(**over)), buf, 64) == tla.ERR_UNSUPPORTED
    assert L.tla_grouped_gemm(ctypes.byref(_product(**over)), None) == tla.ERR_UNSUPPORTED
    w = _wgrad(lda=1 << 31, ldy=1 << 31, ldd=1 << 31, stride_d=1 << 62, **{name: most + 1})
    assert L.tla_grouped_gemm_wgrad(ctypes.byref(w), None) == tla.ERR_UNSUPPORTED


def test_quantizer_rows_it_does_not_count():
    for K, M in ((4096, 1 << 31), (8, 1 << 33), (8, (1 << 63) - 1)):
        assert tla.lib().tla_quantize_rows(M, K, FAKE, tla.BF16, K, FAKE, K, FAKE, None) == tla.ERR_UNSUPPORTED


def test_launches_stay_below_2_to_32_threads():
    """A kernel whose workgroups pass that is not chosen and is refused by name."""
    f = tla.lib().tla_grouped_gemm_run_variant
    wide = dict(groups=1, rows=1, type=tla.I8, K=16, lda=16, ldb=16)
    assert _variant(**dict(wide, N=(1 << 29) - 32, ldd=1 << 29)).startswith("grouped_few_rows")
    over = dict(wide, N=1 << 29, ldd=1 << 29)
    assert not _variant(**over).startswith("grouped_few_rows")
    for v in (4, 5, 6):
        assert f(ctypes.byref(_product(**over)), v, None) == tla.ERR_UNSUPPORTED
    many = dict(groups=1 << 24, rows=1 << 24, N=1, K=1, lda=1, ldb=1, ldd=1, stride_b=0)
    assert tla.lib().tla_grouped_gemm(ctypes.byref(_product(**many)), None) == tla.ERR_UNSUPPORTED
    w = dict(groups=1 << 24, rows=4, N=1, K=1, lda=1, ldy=1, ldd=1, stride_d=1)
    assert tla.lib().tla_grouped_gemm_wgrad(ctypes.byref(_wgrad(**w)), None) == tla.ERR_UNSUPPORTED


def test_binding_refuses_strided_vectors():
    """offsets, scales and bias have no stride argument, so a strided view would
    be misread."""
    t, f = torch.zeros(64), torch.zeros(8, 2)
    call = lambda **kw: tla.grouped_gemm(  # noqa: E731
        1, 1, 8, 8, kw.pop("offsets", None), None, tla.I8, 8, None, tla.COL_MAJOR, 8, 64, None, tla.BF16, 8, **kw)
    for kw in (dict(offsets=torch.zeros(4, dtype=torch.int32)[::2]), dict(scale_a=f[:, 0]), dict(scale_b=f[:, 1]),
               dict(bias=f[:, 0])):
        with pytest.raises(ValueError, match="%s must be contiguous" % list(kw)[0]):
            call(**kw)
    with pytest.raises(ValueError, match="dbias must be contiguous"):
        tla.grouped_gemm_wgrad(1, 1, 8, 8, None, None, 8, None, 8, tla.BF16, None, tla.F32, tla.ROW_MAJOR, 8, 64,
                               dbias=f[:, 0])
    with pytest.raises(ValueError, match="scale must be contiguous"):
        tla.quantize_rows(8, 0, None, tla.F32, 0, None, 0, f[:, 0])
    with pytest.raises(ValueError, match="bias must be contiguous"):
        tla.gemm_i8(1, 8, 8, None, 8, None, tla.COL_MAJOR, 8, None, tla.BF16, 8, bias=t.view(8, 8)[:, 0])


def test_expert_layer_refuses_what_it_would_misread():
    from tiled_layout_algebra_amd.expert_layer import ExpertLayer
    t = lambda *shape, dtype=torch.bfloat16: torch.zeros(*shape, dtype=dtype)  # noqa: E731
    W1, b1, W2 = t(2, 8, 16), t(2, 16), t(2, 16, 8)
    for bad in ((W1, b1, t(2, 8, 16)), (W1, b1.float(), W2), (W1, b1, t(2, 8, 16).transpose(1, 2)),
                (t(2, 16, 8).transpose(1, 2), b1, W2)):
        with pytest.raises(ValueError, match="contiguous bfloat16"):
            ExpertLayer(*bad)
    layer, off = ExpertLayer(W1, b1, W2), torch.tensor([0, 2, 3], dtype=torch.int32)
    for x in (t(3, 9), t(3, 16)[:, :8], t(3, 8, dtype=torch.float16), t(8, 3).t()):
        for call in (layer.forward, layer.decode):
            with pytest.raises(ValueError, match="x must be"):
                call(x, off)
    saved = (t(3, 8), t(3, 16), t(3, 16), off)
    for dy in (t(1, 8).expand(3, 8), t(3, 8, dtype=torch.float32), t(2, 8)):
        with pytest.raises(ValueError, match="dy must be"):
            layer.backward(dy, saved)
