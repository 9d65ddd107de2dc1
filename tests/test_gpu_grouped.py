"""The expert-grouped products on the GPU against 64-bit plain forms: every
operand type and order, ragged and empty experts, odd sizes and pitches with
poisoned padding, activations kept and differentiated, wrong offsets, streams
and graphs.  tests/grouped_util.py derives the bounds."""
import pytest
import torch

import tiled_layout_algebra_amd as tla
from oracle import grouped as og
from tests.grouped_util import (TORCH, Product, check, half_step, offsets_of, pitched, shifted,
                                sum_error, values)

pytestmark = pytest.mark.gpu
TYPES = [tla.BF16, tla.F16, tla.E4M3, tla.I8]
IDS = {tla.BF16: "bf16", tla.F16: "f16", tla.E4M3: "e4m3", tla.I8: "i8"}
COUNTS = {
    "one": [1], "two_tokens": [0, 1, 0, 1], "few": [3, 0, 17, 1, 40], "ragged": [130, 0, 257, 64, 1],
    "many_experts": [i % 3 for i in range(70)], "skewed": [600, 2, 0, 33],
}


@pytest.mark.parametrize("kind", TYPES, ids=IDS.get)
@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_product(kind, counts):
    Product(COUNTS[counts], 160, 256, kind, seed=1).call().verify()


@pytest.mark.parametrize("kind", TYPES, ids=IDS.get)
@pytest.mark.parametrize("N,K", [(1, 1), (7, 3), (129, 15), (40, 16), (33, 257), (264, 136), (9, 1000)])
@pytest.mark.parametrize("order", [tla.COL_MAJOR, tla.ROW_MAJOR], ids=["nk", "kn"])
def test_odd_sizes(kind, N, K, order):
    Product([5, 0, 140], N, K, kind, order=order, bias=True, seed=N + K).call().verify()


@pytest.mark.parametrize("kind", TYPES, ids=IDS.get)
@pytest.mark.parametrize("order", [tla.COL_MAJOR, tla.ROW_MAJOR], ids=["nk", "kn"])
@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (3, 3), (8, 0), (16, 8)])
def test_pitch_and_alignment(kind, order, pad, shift):
    Product([40, 3, 150], 136, 208, kind, order=order, bias=True, act=tla.ACT_RELU, pad=pad,
            shift=shift, seed=pad).call().verify()


@pytest.mark.parametrize("kind", TYPES, ids=IDS.get)
@pytest.mark.parametrize("z", [tla.Z_NONE, tla.Z_STORE, tla.Z_GRAD], ids=["none", "store", "grad"])
@pytest.mark.parametrize("act", [tla.ACT_NONE, tla.ACT_RELU, tla.ACT_GELU], ids=["id", "relu", "gelu"])
@pytest.mark.parametrize("counts", ["few", "skewed"])
def test_epilogue(kind, z, act, counts):
    for bias, d_type, pad in ((True, tla.F16, 0), (False, tla.BF16, 1)):
        Product(COUNTS[counts], 200, 128, kind, d_type=d_type, bias=bias, z=z, act=act, pad=pad,
                seed=3).call().verify()


@pytest.mark.parametrize("bias_type", [tla.F32, tla.F16, tla.BF16])
def test_bias_types(bias_type):
    for N in (64, 67):
        Product([30, 9], N, 64, tla.BF16, bias=True, bias_type=bias_type, seed=4).call().verify()


@pytest.mark.parametrize("kind", TYPES, ids=IDS.get)
@pytest.mark.parametrize("order", [tla.COL_MAJOR, tla.ROW_MAJOR], ids=["nk", "kn"])
def test_large_tiles(kind, order):
    """Enough rows and columns for the widest tiles, ragged on every side."""
    if order == tla.ROW_MAJOR and kind in (tla.E4M3, tla.I8):
        pytest.skip("8-bit operands stored [K, N] take the general kernel, covered above")
    p = Product([1500, 0, 2100, 777], 2312, 320, kind, order=order, bias=True, act=tla.ACT_GELU,
                z=tla.Z_STORE, seed=5)
    p.call().verify()
    p = Product([1500, 0, 2100, 777], 2312, 320, kind, order=order, act=tla.ACT_GELU,
                z=tla.Z_GRAD, seed=6)
    p.call().verify()


def test_rows_of_no_expert_and_no_k():
    Product([20, 0, 5], 64, 64, tla.BF16, lost=9, seed=7).call().verify()
    Product([20, 0, 5], 70, 0, tla.BF16, bias=True, act=tla.ACT_GELU, seed=8).call().verify()
    Product([33], 64, 64, tla.I8, no_offsets=True, seed=9).call().verify()


@pytest.mark.parametrize("off", [[0, 900, -5, 60], [50, 20, 40, 60], [-7, 10, 10, 1 << 30],
                                 [0, 60, 60, 60]])
def test_wrong_offsets_stay_inside(off):
    """Offsets are clamped into [0, rows]: whatever they hold, nothing outside
    D's rows and columns is written."""
    p = Product([20, 20, 20], 96, 64, tla.BF16, pad=5, seed=10)
    p.off = off
    p.call()
    torch.cuda.synchronize()
    assert (p.logical(p.D)[1] == 7.0).all()
    Y = values(torch.Generator().manual_seed(1), (60, 96), tla.BF16).cuda()
    D = torch.full((3, 64, 96), 7.0, device="cuda")
    tla.grouped_gemm_wgrad(3, 60, 96, 64, torch.tensor(off, dtype=torch.int32).cuda(),
                           p.A.cuda(), 64, Y, 96, tla.BF16, D, tla.F32, tla.ROW_MAJOR, 96, 64 * 96)
    assert torch.isfinite(D).all()


def test_nan_and_infinity_pass_through():
    for act in (tla.ACT_NONE, tla.ACT_RELU, tla.ACT_GELU):
        for counts in ([3, 2], [300, 2]):
            p = Product(counts, 32, 64, tla.BF16, act=act, seed=11)
            p.A[1, 5] = float("nan")
            p.A[2, 7] = float("inf")
            p.B[0, 7] = 1.0
            p.call()
            got = p.logical(p.D)[0]
            assert got[1].isnan().all() and (got[2] == float("inf")).all()
            rest = [r for r in range(sum(counts)) if r not in (1, 2)]
            (_, ref, bound), = p.expect()
            check(got[rest], ref[rest], bound[rest], "rows beside")


def test_int8_sums_are_exact():
    """The largest sum that 32 bits hold, and mixed signs that cancel to a few
    units of 2^31 terms."""
    K = 131071
    for rows in (2, 150):
        A = torch.full((rows, K), -128, dtype=torch.int8)
        A[1] = torch.tensor([127, -128], dtype=torch.int8).repeat(K)[:K]
        B = torch.full((3, K), -128, dtype=torch.int8)
        B[1] = torch.arange(K).remainder(2).mul(2).sub(1).to(torch.int8)
        want = (A.double() @ B.double().t())
        D = torch.empty(rows, 3, dtype=torch.bfloat16, device="cuda")
        tla.gemm_i8(rows, 3, K, A.cuda(), K, B.cuda(), tla.COL_MAJOR, K, D, tla.BF16, 3)
        assert torch.equal(D.cpu(), want.float().bfloat16())


@pytest.mark.parametrize("M,N,K", [(1, 64, 512), (1, 37, 129), (17, 512, 256), (300, 200, 1024),
                                   (2500, 2304, 384)])
@pytest.mark.parametrize("out", [tla.BF16, tla.F16])
def test_gemm_i8(M, N, K, out):
    p = Product([M], N, K, tla.I8, d_type=out, bias=True, act=tla.ACT_GELU, seed=M)
    D = torch.empty(M, N, dtype=TORCH[out], device="cuda")
    tla.gemm_i8(M, N, K, p.A.cuda(), K, p.B[0].t().contiguous().cuda(), tla.COL_MAJOR, K, D, out, N,
                scale_a=p.sa.cuda(), scale_b=p.sb.cuda(), bias=p.bias.cuda(), act=tla.ACT_GELU)
    (_, ref, bound), = p.expect()
    check(D.cpu(), ref, bound, "D")


@pytest.mark.parametrize("kind", [tla.BF16, tla.F16], ids=IDS.get)
@pytest.mark.parametrize("d_type", [tla.F32, tla.BF16, tla.F16])
@pytest.mark.parametrize("order", [tla.ROW_MAJOR, tla.COL_MAJOR], ids=["kn", "nk"])
@pytest.mark.parametrize("counts,N,K", [
    ([1], 8, 8), ([0, 5, 1], 7, 3), ([3, 0, 70, 64], 130, 129), ([200, 0, 1000], 264, 136),
    ([65, 63, 0, 128], 256, 256), ([0, 0], 16, 24)], ids=str)
def test_wgrad(kind, d_type, order, counts, N, K):
    _wgrad(kind, d_type, order, counts, N, K, pad=0)


@pytest.mark.parametrize("pad,shift", [(1, 0), (8, 0), (8, 8), (3, 5)])
@pytest.mark.parametrize("order", [tla.ROW_MAJOR, tla.COL_MAJOR], ids=["kn", "nk"])
def test_wgrad_pitch_and_alignment(pad, shift, order):
    _wgrad(tla.BF16, tla.F32, order, [90, 0, 140], 136, 72, pad, shift)
    _wgrad(tla.F16, tla.F16, order, [90, 0, 140], 136, 72, pad, shift)


@pytest.mark.parametrize("order", [tla.ROW_MAJOR, tla.COL_MAJOR], ids=["kn", "nk"])
def test_wgrad_large_tiles(order):
    _wgrad(tla.BF16, tla.BF16, order, [333, 0, 1000, 1], 1544, 2312, 0)


def _wgrad(kind, d_type, order, counts, N, K, pad, shift=0):
    g, off = len(counts), offsets_of(counts)
    rows = off[-1]
    gen = torch.Generator().manual_seed(rows + N)
    A, Y = values(gen, (rows, K), kind), values(gen, (rows, N), kind, 0.1)
    a, _ = pitched(A[None], K + pad, kind)
    y, _ = pitched(Y[None], N + pad, kind)
    r, c = (K, N) if order == tla.ROW_MAJOR else (N, K)
    ldd = c + pad
    stride = r * ldd + pad
    D = shifted(torch.full((g * stride,), 7.0).to(TORCH[d_type]), shift)
    db = torch.full((g, N), 7.0, device="cuda")
    tla.grouped_gemm_wgrad(g, rows, N, K, torch.tensor(off, dtype=torch.int32).cuda(),
                           shifted(a, shift), K + pad, shifted(y, shift), N + pad, kind, D, d_type,
                           order, ldd, stride, dbias=db)
    want, S, want_b, Sb = og.wgrad(A, Y, off)
    if order == tla.COL_MAJOR:
        want, S = want.transpose(1, 2), S.transpose(1, 2)
    got = D.cpu()
    eps = 2.0 ** -24
    for e, n in enumerate(counts):
        m = got[e * stride:e * stride + r * ldd].view(r, ldd)
        err = S[e] * ((n + 4) * eps)
        check(m[:, :c], want[e], err + half_step(want[e].abs() + err, d_type), "D of %d" % e)
        assert (m[:, c:] == 7.0).all()
        assert (got[e * stride + r * ldd:(e + 1) * stride] == 7.0).all()
        check(db[e].cpu(), want_b[e], Sb[e] * ((n + 4) * eps) + 1e-45, "dbias of %d" % e)


def test_layer_gradients_against_autograd_and_differences():
    """One expert layer x -> gelu(x W1 + b1) W2: the kernels' dW, db and dh
    against float64 autograd of the same stored values, and against central
    differences of the loss."""
    g, N, K, counts = 3, 48, 40, [50, 0, 33]
    off, rows = offsets_of(counts), 83
    gen = torch.Generator().manual_seed(3)
    x, W = values(gen, (rows, K), tla.F16), values(gen, (g, K, N), tla.F16, K ** -0.5)
    b, W2 = values(gen, (g, N), tla.F16), values(gen, (g, N, K), tla.F16, N ** -0.5)
    dy = values(gen, (rows, K), tla.F16, 0.1)
    offs = torch.tensor(off, dtype=torch.int32).cuda()
    xd, Wd, bd, W2d, dyd = (t.cuda() for t in (x, W, b, W2, dy))
    h, z, dz = (torch.empty(rows, N, dtype=torch.float16, device="cuda") for _ in range(3))
    tla.grouped_gemm(g, rows, N, K, offs, xd, tla.F16, K, Wd, tla.ROW_MAJOR, N, K * N, h, tla.F16,
                     N, bias=bd, Z=z, ldz=N, z_mode=tla.Z_STORE, act=tla.ACT_GELU)
    # dz = (dy W2^T) gelu'(z): W2 stored [N, K] is the K-contiguous operand of it
    tla.grouped_gemm(g, rows, N, K, offs, dyd, tla.F16, K, W2d, tla.COL_MAJOR, K, K * N, dz,
                     tla.F16, N, Z=z, ldz=N, z_mode=tla.Z_GRAD, act=tla.ACT_GELU)
    dW = torch.empty(g, K, N, device="cuda")
    db = torch.empty(g, N, device="cuda")
    tla.grouped_gemm_wgrad(g, rows, N, K, offs, xd, K, dz, N, tla.F16, dW, tla.F32, tla.ROW_MAJOR,
                           N, K * N, dbias=db)

    def loss(Wp, bp):
        out = 0.0
        for e, (lo, hi) in enumerate(og.spans(off)):
            hh = og.act(x[lo:hi].double() @ Wp[e] + bp[e], tla.ACT_GELU)
            out = out + ((hh @ W2[e].double()) * dy[lo:hi].double()).sum()
        return out

    Wp, bp = W.double().requires_grad_(), b.double().requires_grad_()
    gW, gb = torch.autograd.grad(loss(Wp, bp), (Wp, bp))
    # dz carries the roundings of z (half a step, slope of gelu' at most 0.8)
    # and of itself; dW sums them over the expert's rows
    step = 2.0 ** -11
    n = max(counts)
    tol_z = (0.8 * z.abs().max().item() * 1.2 + 1.2) * step * dy.abs().sum(1).max().item() * \
        W2.abs().max().item()
    assert (dW.cpu() - gW).abs().max() <= n * x.abs().max().item() * tol_z
    assert (db.cpu() - gb).abs().max() <= n * tol_z
    # differences: error of the central form below 1e-6 at this step
    for e, i, j in ((0, 1, 2), (2, 39, 47), (2, 0, 11)):
        d = torch.zeros_like(gW)
        d[e, i, j] = 1e-4
        with torch.no_grad():
            num = (loss(Wp + d, bp) - loss(Wp - d, bp)) / 2e-4
        assert abs(num - gW[e, i, j]) <= 1e-6 * (1 + abs(gW[e, i, j]))
        assert abs(dW[e, i, j].item() - num) <= n * x.abs().max().item() * tol_z + 1e-6


def test_other_stream_and_graph():
    """A call on a side stream, and a captured product and gradient replayed
    with new inputs and eager work between the replays."""
    p = Product([40, 0, 200], 256, 128, tla.BF16, bias=True, act=tla.ACT_GELU, seed=12)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p.call()
    torch.cuda.synchronize()
    eager = p.D.clone()
    args, kw = p.keep
    with torch.cuda.stream(side):
        p.D.fill_(7.0)
        tla.grouped_gemm(*args, **kw)
    side.synchronize()
    assert torch.equal(p.D, eager)
    g, rows, N, K, off, A = args[:6]
    dW, db = torch.empty(g, K, N, device="cuda"), torch.empty(g, N, device="cuda")
    Q = torch.empty(rows, N, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, device="cuda")

    def work():
        tla.grouped_gemm(*args, **kw)
        tla.grouped_gemm_wgrad(g, rows, N, K, off, A, K, p.D, N, tla.BF16, dW, tla.F32,
                               tla.ROW_MAJOR, N, K * N, dbias=db)
        tla.quantize_rows(rows, N, p.D, tla.BF16, N, Q, N, s)

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for i in range(4):
        A.copy_(values(torch.Generator().manual_seed(i), A.shape, tla.BF16))
        work()
        torch.cuda.synchronize()
        want = [t.clone() for t in (p.D, dW, db, Q, s)]
        for t in (p.D, dW, db, Q, s):
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for w, t in zip(want, (p.D, dW, db, Q, s)):
            assert torch.equal(w, t)


def test_gradient_order_is_fixed():
    """Two calls give the same bits."""
    outs = []
    gen = torch.Generator().manual_seed(5)
    A, Y = values(gen, (900, 256), tla.BF16).cuda(), values(gen, (900, 128), tla.BF16).cuda()
    off = torch.tensor([0, 300, 900], dtype=torch.int32).cuda()
    for _ in range(3):
        D, db = torch.empty(2, 256, 128, device="cuda"), torch.empty(2, 128, device="cuda")
        tla.grouped_gemm_wgrad(2, 900, 128, 256, off, A, 256, Y, 128, tla.BF16, D, tla.F32,
                               tla.ROW_MAJOR, 128, 256 * 128, dbias=db)
        outs.append((D, db))
    assert all(torch.equal(a, b) for o in outs[1:] for a, b in zip(outs[0], o))


def _takes(variant, kind, order, N, K, pad, shift):
    """The conditions include/tla.h names."""
    eb = 1 if kind in (tla.E4M3, tla.I8) else 2
    nk = order == tla.COL_MAJOR
    if variant == 0:
        return True
    if variant in (4, 5, 6):
        return nk
    if kind == tla.E4M3 and K < 512:
        return False
    if variant >= 7:
        return nk
    ldb = (K if nk else N) + pad
    stride_b = (N if nk else K) * ldb + pad
    aligned = all(x * eb % 4 == 0 for x in (K + pad, ldb, shift, stride_b))
    if variant == 3 and not nk:
        return False
    return aligned and (nk or eb == 2)


@pytest.mark.parametrize("variant", range(tla.GROUPED_VARIANTS))
@pytest.mark.parametrize("kind", TYPES, ids=IDS.get)
@pytest.mark.parametrize("order", [tla.COL_MAJOR, tla.ROW_MAJOR], ids=["nk", "kn"])
@pytest.mark.parametrize("N,K,pad,shift", [
    (40, 16, 0, 0), (300, 96, 0, 0), (264, 576, 0, 0), (136, 1040, 16, 16), (7, 47, 0, 0),
    (300, 97, 1, 1), (129, 511, 2, 3), (280, 1055, 3, 0), (257, 600, 5, 2), (300, 98, 0, 0),
    (130, 525, 3, 4), (18, 1043, 1, 0)], ids=str)
def test_every_kernel(variant, kind, order, N, K, pad, shift):
    """Each kernel on tiles it fills and tiles it does not, K from less than a
    step to several k-tiles, and at any byte address where it takes that: the
    padding and the next row's bytes are poison."""
    p = Product([300, 0, 5, 129, 1], N, K, kind, order=order, bias=True, act=tla.ACT_RELU, pad=pad,
                shift=shift, seed=K)
    if _takes(variant, kind, order, N, K, pad, shift):
        p.call(variant=variant).verify()
    else:
        with pytest.raises(tla.TlaError) as err:
            p.call(variant=variant)
        assert err.value.status == tla.ERR_UNSUPPORTED
        torch.cuda.synchronize()
        assert (p.D == 7.0).all()


@pytest.mark.parametrize("variant", range(tla.GROUPED_VARIANTS))
def test_every_kernel_keeps_and_differentiates(variant):
    for kind in (tla.F16, tla.I8):
        for z in (tla.Z_STORE, tla.Z_GRAD):
            Product([150, 3, 0, 70], 200, 512, kind, z=z, act=tla.ACT_GELU,
                    seed=z).call(variant=variant).verify()


@pytest.mark.parametrize("variant", range(tla.GROUPED_VARIANTS))
def test_offsets_past_32_bits(variant):
    """Rows of A and D and the experts' matrices further apart than 2^32
    bytes: 1100 rows 4 MiB apart, the second expert's weights 4.3 GB on."""
    rows, N, K, lda, ldd, stride = 1100, 40, 512, 1 << 21, 1 << 21, (1 << 31) + 64
    p = Product([600, 500], N, K, tla.BF16, bias=True, seed=13)
    A = torch.empty(rows, lda, dtype=torch.bfloat16, device="cuda")
    A[:, :K] = p.A.cuda()
    D = torch.empty(rows, ldd, dtype=torch.bfloat16, device="cuda")
    B = torch.empty(stride + N * K, dtype=torch.bfloat16, device="cuda")
    nk = p.B.transpose(1, 2).contiguous().cuda()
    for e in range(2):
        B[e * stride:e * stride + N * K] = nk[e].reshape(-1)
    off = torch.tensor(p.off, dtype=torch.int32).cuda()
    tla.grouped_gemm(2, rows, N, K, off, A, tla.BF16, lda, B, tla.COL_MAJOR, K, stride, D, tla.BF16,
                     ldd, bias=p.bias.cuda(), variant=variant)
    (_, ref, bound), = p.expect()
    check(D[:, :N].cpu(), ref, bound, "D")


def test_gradient_and_codes_past_32_bits():
    """A gradient over rows 8 MiB apart (9.2 GB of A), into matrices 4.3 GB
    apart, and codes of rows 8 MiB apart."""
    rows, N, K, lda, stride = 1100, 24, 40, 1 << 22, (1 << 30) + 8
    gen = torch.Generator().manual_seed(6)
    A, Y = values(gen, (rows, K), tla.BF16), values(gen, (rows, N), tla.BF16)
    Ad = torch.empty(rows, lda, dtype=torch.bfloat16, device="cuda")
    Ad[:, :K] = A.cuda()
    D = torch.empty(stride + K * N, device="cuda")
    off = [0, 700, rows]
    tla.grouped_gemm_wgrad(2, rows, N, K, torch.tensor(off, dtype=torch.int32).cuda(), Ad, lda,
                           Y.cuda(), N, tla.BF16, D, tla.F32, tla.ROW_MAJOR, N, stride)
    want, S, _, _ = og.wgrad(A, Y, off)
    for e in range(2):
        got = D[e * stride:e * stride + K * N].view(K, N).cpu()
        check(got, want[e], S[e] * (704 * 2.0 ** -24) + half_step(want[e].abs(), tla.F32), "D")
    Q = torch.empty(rows, lda, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, device="cuda")
    tla.quantize_rows(rows, K, Ad, tla.BF16, lda, Q, lda, s)
    q, scale = og.quantize_rows(A)
    assert torch.equal(Q[:, :K].cpu(), q) and torch.equal(s.cpu(), scale)


@pytest.mark.parametrize("variant", range(tla.GROUPED_VARIANTS))
def test_e4m3_nan_stays_in_its_row(variant):
    p = Product([40, 150], 72, 512, tla.E4M3, seed=14)
    raw = p.A.view(torch.int8)
    raw[3, 5] = 0x7F
    raw[100, 511] = -1  # the negative NaN, 0xFF
    p.call(variant=variant)
    got = p.logical(p.D)[0]
    assert got[3].isnan().all() and got[100].isnan().all()
    rest = [r for r in range(190) if r not in (3, 100)]
    (_, ref, bound), = p.expect()
    check(got[rest], ref[rest], bound[rest], "rows beside")
