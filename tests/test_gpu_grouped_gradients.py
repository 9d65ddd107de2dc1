"""The weight and bias gradients of a grouped product through each of their
kernels: extents that end inside a 16-byte chunk with poisoned padding behind
them, and values that are not finite in one column, which must stay in it.
The sizes choose the kernel: rows off a dword take the register-staged one;
256 tiles of 256 x 256 or more, over all experts, the two-group kernel; the
direct kernel otherwise, with three stages up to 256 tiles of 128 x 128 and two
beyond.  Bounds as in tests/grouped_util.py: (rows + 4) 2^-24 of the terms'
magnitudes and half a step of the stored type."""
import pytest
import torch

import tiled_layout_algebra_amd as tla
from oracle import grouped as og
from tests.grouped_util import TORCH, check, half_step, offsets_of, pitched, shifted, values

pytestmark = pytest.mark.gpu
ORDERS = pytest.mark.parametrize("order", [tla.ROW_MAJOR, tla.COL_MAJOR], ids=["kn", "nk"])
# kernel: (experts, least extents of D_e, elements by which the buffers start off a dword)
KERNELS = {"direct_three_stages": (3, 0, 0), "direct_two_stages": (130, 128, 0),
           "two_group": (260, 0, 0), "general": (3, 0, 1)}


def counts_of(experts):
    """Ragged experts: none, a few and, for the first ones, several k-tiles of rows."""
    return ([150, 0, 33] + [(7 * e) % 11 for e in range(experts)])[:experts]


class Gradient:
    def __init__(self, counts, N, K, kind=tla.BF16, seed=0):
        self.counts, self.N, self.K, self.kind = counts, N, K, kind
        self.off = offsets_of(counts)
        gen = torch.Generator().manual_seed(seed + N)
        self.A = values(gen, (self.off[-1], K), kind)
        self.Y = values(gen, (self.off[-1], N), kind, 0.1)

    def run(self, d_type, order, pad_a, pad_y, shift=0, pad_d=0):
        """D [experts, K, N] and dbias on the host; whatever lies beside D is untouched."""
        g, rows, N, K = len(self.counts), self.off[-1], self.N, self.K
        a, _ = pitched(self.A[None], K + pad_a, self.kind)
        y, _ = pitched(self.Y[None], N + pad_y, self.kind)
        r, c = (K, N) if order == tla.ROW_MAJOR else (N, K)
        ldd = c + pad_d
        D = torch.full((g * r * ldd,), 7.0).to(TORCH[d_type]).cuda()
        db = torch.full((g, N), 7.0, device="cuda")
        off = torch.tensor(self.off, dtype=torch.int32).cuda()
        tla.grouped_gemm_wgrad(g, rows, N, K, off, shifted(a, shift), K + pad_a, shifted(y, shift),
                               N + pad_y, self.kind, D, d_type, order, ldd, r * ldd, dbias=db)
        m = D.cpu().view(g, r, ldd)
        assert (m[:, :, c:] == 7.0).all()
        m = m[:, :, :c]
        return (m if order == tla.ROW_MAJOR else m.transpose(1, 2)), db.cpu()

    def verify(self, d_type, order, pad_a, pad_y, shift=0, pad_d=0):
        D, db = self.run(d_type, order, pad_a, pad_y, shift, pad_d)
        want, S, want_b, Sb = og.wgrad(self.A, self.Y, self.off)
        eps = (torch.tensor(self.counts, dtype=torch.float64) + 4) * 2.0 ** -24
        err, err_b = S * eps[:, None, None], Sb * eps[:, None]
        fin, fin_b = want.isfinite(), want_b.isfinite()
        for name, got, ref, ok in (("D", D, want, fin), ("dbias", db, want_b, fin_b)):
            assert torch.equal(got.isnan()[~ok], ref.isnan()[~ok]), name
            inf = ref.isinf()
            assert torch.equal(got[inf].double(), ref[inf]), name
        zero = torch.zeros((), dtype=torch.float64)
        bound = err + half_step(want.abs() + err, d_type)
        check(torch.where(fin, D.double(), zero), torch.where(fin, want, zero),
              torch.where(fin, bound, zero), "D")
        check(torch.where(fin_b, db.double(), zero), torch.where(fin_b, want_b, zero),
              torch.where(fin_b, err_b + 1e-45, zero), "dbias")


@pytest.mark.parametrize("kernel", KERNELS)
@ORDERS
@pytest.mark.parametrize("N,K,pad_y,pad_a", [(20, 20, 4, 4), (22, 18, 2, 6), (30, 28, 8, 4), (21, 27, 3, 5)],
                         ids=str)
def test_padding_behind_a_chunk(kernel, order, N, K, pad_y, pad_a):
    """Extents of 17 to 31 modulo 32 that are 2, 4, 6 and odd modulo 8, rows on
    dwords: the chunk that crosses the extent holds NaN from the padding."""
    experts, least, shift = KERNELS[kernel]
    Gradient(counts_of(experts), least + N, least + K).verify(tla.F32, order, pad_a, pad_y, shift)


@pytest.mark.parametrize("kernel", KERNELS)
@ORDERS
@pytest.mark.parametrize("kind", [tla.BF16, tla.F16])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")], ids=str)
def test_not_finite_stays_in_its_column(kernel, order, kind, bad):
    """One such value in dY reaches its column of dW and of the bias gradient,
    one in A its row of dW, of its expert alone."""
    experts, least, shift = KERNELS[kernel]
    p = Gradient(counts_of(experts), least + 64, least + 40, kind)
    p.Y[140, 20] = bad      # of expert 0, in its last k-tile
    p.Y[151, 3] = -bad      # of expert 2
    p.A[3, 33] = bad
    p.verify(tla.F32, order, 0, 0, shift)


def test_wide_pitches_with_few_rows():
    """8 rows 128 MiB apart: a slab of the direct copies has 64 rows, whose byte
    offsets would pass 2^32 and come back to rows and padding in use."""
    rows, N, K, ld = 8, 24, 40, (1 << 26) + 64
    gen = torch.Generator().manual_seed(2)
    A, Y = values(gen, (rows, K), tla.BF16), values(gen, (rows, N), tla.BF16)
    bufs = []
    for m in (A, Y):
        buf = torch.full((rows, ld), float("nan"), dtype=torch.bfloat16, device="cuda")
        buf[:, :m.shape[1]] = m.cuda()
        bufs.append(buf)
    D, db = torch.empty(1, K, N, device="cuda"), torch.empty(1, N, device="cuda")
    tla.grouped_gemm_wgrad(1, rows, N, K, None, bufs[0], ld, bufs[1], ld, tla.BF16, D, tla.F32,
                           tla.ROW_MAJOR, N, K * N, dbias=db)
    want, S, want_b, Sb = og.wgrad(A, Y, [0, rows])
    eps = (rows + 4) * 2.0 ** -24
    check(D.cpu(), want, S * eps + half_step(want.abs(), tla.F32), "D")
    check(db.cpu(), want_b, Sb * eps + 1e-45, "dbias")
    # the [K, N] product over the same rows: D [rows of X, N] = X A with X [5, 8]
    X = values(gen, (5, rows), tla.BF16)
    for buf, m in zip(bufs, (A, Y)):
        n = m.shape[1]
        P = torch.empty(5, n, dtype=torch.bfloat16, device="cuda")
        tla.grouped_gemm(1, 5, n, rows, None, X.cuda(), tla.BF16, rows, buf, tla.ROW_MAJOR, ld, 0, P,
                         tla.BF16, n)
        ref, s = X.double() @ m.double(), X.double().abs() @ m.double().abs()
        check(P.cpu(), ref, s * eps + half_step(ref.abs() + s * eps, tla.BF16), "product")


@pytest.mark.parametrize("kernel", KERNELS)
@ORDERS
@pytest.mark.parametrize("kind", [tla.BF16, tla.F16])
@pytest.mark.parametrize("d_type", [tla.F32, tla.BF16, tla.F16])
def test_results_of_each_kernel(kernel, order, kind, d_type):
    """Every result type from every kernel, extents off the tile and off a
    chunk, D's rows pitched at any element."""
    experts, least, shift = KERNELS[kernel]
    Gradient(counts_of(experts), least + 74, least + 53, kind, seed=1).verify(d_type, order, 3, 6, shift, pad_d=5)
    Gradient(counts_of(experts), least + 64, least + 72, kind, seed=2).verify(d_type, order, 0, 0, shift)


@ORDERS
@pytest.mark.parametrize("kind,d_type", [(tla.BF16, tla.F32), (tla.F16, tla.F32), (tla.F16, tla.F16)])
def test_two_group_tiles_filled(order, kind, d_type):
    """280 tiles of 256 x 256 over whole and ragged ones, rows pitched on dwords."""
    Gradient([333, 0, 1000, 1], 1550, 2314, kind, seed=3).verify(d_type, order, 6, 2, pad_d=2)
