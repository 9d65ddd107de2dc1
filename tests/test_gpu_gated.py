"""The gated product and its gradient on the GPU: every kernel by name over odd
sizes, pitches and alignments with poisoned padding, activations, biases, kept
pre-activations, experts without rows, wrong offsets, NaN and infinity, autograd
and differences, streams and graphs.  Bounds: tests/gated_util.py."""
import pytest
import torch

import tiled_layout_algebra_amd as tla
from oracle import gated as oga
from tests.gated_util import VARIANTS, Gated, Grad, check, raw

pytestmark = pytest.mark.gpu
NK, KN = tla.COL_MAJOR, tla.ROW_MAJOR

# rows of experts, N, K, padding of every pitch
SHAPES = [
    ([1], 16, 64, 0),
    ([37], 130, 72, 2),
    ([300], 264, 520, 8),
    ([5, 0, 131, 1], 200, 200, 4),
    ([256, 130, 0], 129, 66, 2),
    ([0, 0, 70], 96, 8, 0),
]


def variants(order, role):
    out = ["general", "two_group", "direct128"]
    if order == NK:
        out += ["direct64"] + (["few64", "few32", "few16"] if role == "gated" else [])
    return out


def shape_of(i, order):
    """Direct copies want rows on dwords: an even pitch of [K, N] weights."""
    counts, N, K, pad = SHAPES[i]
    return counts, N + (order == KN and (N + pad) % 2), K, pad


CASES = [(v, o, s) for o in (NK, KN) for v in variants(o, "gated") for s in range(len(SHAPES))]


@pytest.mark.parametrize("variant,order,shape", CASES)
def test_gated_every_kernel(variant, order, shape):
    counts, N, K, pad = shape_of(shape, order)
    kind = tla.BF16 if shape % 2 else tla.F16
    Gated(counts, N, K, kind, order=order, pad=pad, keep=shape % 3 != 1, lost=shape % 2 * 3,
          bias=(shape in (1, 3), shape in (1, 4)), act=(3, 2, 1, 3, 0, 3)[shape],
          seed=shape).call(variant=VARIANTS[variant]).verify()


@pytest.mark.parametrize("variant,order,shape",
                         [c for c in CASES if c[0] in variants(c[1], "grad")])
def test_grad_every_kernel(variant, order, shape):
    counts, N, K, pad = shape_of(shape, order)
    kind = tla.BF16 if shape % 2 else tla.F16
    Grad(counts, N, K, kind, order=order, pad=pad, hidden=shape != 1, lost=shape % 2 * 3,
         act=(3, 2, 1, 3, 0, 3)[shape], seed=shape).call(variant=VARIANTS[variant]).verify()


@pytest.mark.parametrize("order", [NK, KN])
@pytest.mark.parametrize("variant", ["general", "two_group", "direct128"])
def test_many_tiles(variant, order):
    """Several tiles each way, experts that end inside one, the last k-tile short."""
    v = VARIANTS[variant]
    Gated([700, 0, 389, 130], 712, 328, tla.BF16, order=order, keep=True).call(variant=v).verify()
    Grad([700, 0, 389, 130], 712, 328, tla.F16, order=order, act=tla.ACT_GELU).call(variant=v).verify()


@pytest.mark.parametrize("order", [NK, KN])
def test_many_experts_and_short_lines(order):
    """More experts than lanes, most of them empty, on every kernel."""
    counts = [3 if e % 7 == 2 else 0 for e in range(150)]
    for v in ((0, 1, 2, 3, 6) if order == NK else (0, 1, 2)):
        Gated(counts, 32, 64, tla.BF16, order=order).call(variant=v).verify()
    Gated(counts, 5, 6, tla.BF16, order=order, bias=(True, True), lost=2).call().verify()
    Grad(counts, 5, 6, tla.BF16, order=order, lost=2).call().verify()


@pytest.mark.parametrize("variant", ["general", "two_group", "direct64"])
def test_offsets_past_32_bits(variant):
    """Rows 8 MiB apart: the last ones' offsets pass 2^32 bytes in every buffer."""
    rows, N, K, ld = 520, 64, 64, (1 << 22) + 8
    v = VARIANTS[variant]
    gen = torch.Generator().manual_seed(4)
    W = (torch.randn(2, N, K, generator=gen) / 8).bfloat16()
    X = torch.randn(rows, K, generator=gen).bfloat16()
    pitch = ld if variant == "general" else (1 << 22) - 8
    Xd, H, Z, Z2 = (torch.empty(rows * pitch, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    Xd.view(rows, pitch)[:, :K] = X.cuda()
    Wd = W.cuda()
    tla.gated_gemm(1, rows, N, K, None, Xd, tla.BF16, pitch, Wd[0], Wd[1], NK, K, 0, H, tla.BF16, pitch,
                   Z_gate=Z, Z_up=Z2, ldz=pitch, variant=v)
    dY = Xd  # [rows, K]
    D, D2 = (torch.empty(rows * pitch, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tla.gated_gemm_grad(1, rows, N, K, None, dY, tla.BF16, pitch, Wd[0], NK, K, 0, Z, Z2, pitch, D, D2,
                        tla.BF16, pitch, variant=v)
    torch.cuda.synchronize()
    part = lambda t: t.view(rows, pitch)[:, :N].cpu().double()  # noqa: E731
    g, u = X.double() @ W[0].double().t(), X.double() @ W[1].double().t()
    e = 2.0 ** -24 * (K + 4) * (X.double().abs() @ W.double().abs().amax(0).t())
    check(part(Z), g, e + g.abs() * 2.0 ** -8, "Z_gate")
    check(part(Z2), u, e + u.abs() * 2.0 ** -8, "Z_up")
    h = oga.act(g, 3) * u
    check(part(H), h, 1.13 * e * (u.abs() + e) + e * g.abs() + h.abs() * 2.0 ** -8 + 1e-6, "H")
    zg, zu = part(Z), part(Z2)
    dg = g * zu * oga.act_slope(zg, 3)
    check(part(D), dg, e * (zu.abs() + 1) + dg.abs() * 2.0 ** -8 + 1e-6, "dZ_gate")
    check(part(D2), g * oga.act(zg, 3), e * (zg.abs() + 1) + (g * oga.act(zg, 3)).abs() * 2.0 ** -8 + 1e-6,
          "dZ_up")


@pytest.mark.parametrize("order", [NK, KN])
@pytest.mark.parametrize("N,K,pad,shift", [(99, 77, 0, 0), (99, 77, 1, 1), (64, 80, 3, 1),
                                           (7, 5, 0, 0), (3, 40, 1, 1), (40, 3, 2, 1), (1, 1, 0, 0)])
def test_rows_at_any_element(order, N, K, pad, shift):
    """Rows off a dword, lines shorter than a 16-byte chunk: the library's choice."""
    kw = dict(order=order, pad=pad, shift=shift)
    Gated([3, 0, 90], N, K, tla.BF16, keep=True, bias=(True, True), **kw).call().verify()
    Grad([3, 0, 90], N, K, tla.F16, **kw).call().verify()


@pytest.mark.parametrize("variant", ["few64", "few32", "few16"])
@pytest.mark.parametrize("K,shift", [(77, 1), (519, 0), (40, 1), (1000, 0)])
def test_few_rows_off_dwords(variant, K, shift):
    Gated([3, 0, 20], 50, K, tla.BF16, pad=1, shift=shift, bias=(True, False)).call(
        variant=VARIANTS[variant]).verify()


@pytest.mark.parametrize("variant,order", [("two_group", NK), ("two_group", KN), ("direct128", NK),
                                           ("direct128", KN), ("direct64", NK), ("general", NK),
                                           ("general", KN), ("few16", NK)])
def test_halves_of_one_buffer(variant, order):
    """[2 N, K] and [K, 2 N] weights whose K ends inside a k-tile: the rows past
    the gate's last one are the up projection's, and the other way round."""
    Gated([70, 9], 136, 200, tla.BF16, order=order, one_buffer=True, keep=True).call(
        variant=VARIANTS[variant]).verify()


@pytest.mark.parametrize("kind", [tla.F16, tla.BF16])
@pytest.mark.parametrize("bias_type", [tla.F16, tla.BF16, tla.F32])
def test_types(kind, bias_type):
    for variant in (0, 1, 2, 3, 6):
        Gated([200], 136, 96, kind, bias=(True, True), bias_type=bias_type, keep=True).call(
            variant=variant).verify()
        if variant < 4:
            Grad([200], 136, 96, kind).call(variant=variant).verify()


@pytest.mark.parametrize("act", [tla.ACT_NONE, tla.ACT_RELU, tla.ACT_GELU, tla.ACT_SILU])
@pytest.mark.parametrize("rows", [1, 17, 700])
def test_activations(act, rows):
    Gated([rows], 264, 256, tla.BF16, act=act, keep=True, no_offsets=True).call().verify()
    Grad([rows], 264, 256, tla.BF16, act=act, no_offsets=True, z_std=4.0).call().verify()


def test_no_k():
    """K = 0: the sums are the biases; the gradient's are zero."""
    Gated([40], 24, 0, tla.BF16, bias=(True, True), keep=True).call().verify()
    Gated([40], 24, 0, tla.F16).call().verify()
    Grad([40], 24, 0, tla.BF16).call().verify()


def test_wrong_offsets_stay_inside():
    """Offsets past the rows or out of order lose rows and touch nothing else."""
    c = Gated([20, 20, 20], 64, 64, tla.BF16, keep=True).call()
    for bad in ([0, 90, 20, 60], [-5, 20, 1000, 2000], [60, 40, 20, 0], [0, 0, 0, 0]):
        args = list(c.args)
        args[4] = torch.tensor(bad, dtype=torch.int32).cuda()
        for v in (0, 1, 2, 3, 4, 5, 6):
            tla.gated_gemm(*args, variant=v, **c.kw)
    torch.cuda.synchronize()
    c.again()
    c.verify()


@pytest.mark.parametrize("variant", ["general", "two_group", "direct128", "direct64", "few16"])
def test_nan_and_infinity_stay_in_their_rows(variant):
    c = Gated([100], 72, 104, tla.BF16)
    c.X[3, 5], c.X[60, 103] = float("nan"), float("inf")
    c.call(variant=VARIANTS[variant])
    torch.cuda.synchronize()
    got, _ = raw(c.H, c.rows, c.N, c.N)
    assert got[3].isnan().all() and not got[60].isfinite().all()
    fine = [i for i in range(100) if i not in (3, 60)]
    assert got[fine].isfinite().all()
    c.X[3], c.X[60] = 0, 0
    want = Gated.sums(c)
    h = oga.act(want[0][0], c.act) * want[1][0]
    assert torch.allclose(got[fine].double(), h[fine], atol=2e-2, rtol=1e-2)


def test_large_arguments():
    """Gates far out: SiLU ends in 0 and z, its derivative in 0 and 1, nothing overflows."""
    c = Grad([64], 64, 64, tla.BF16, z_std=300.0)
    c.call().verify()
    assert c.D.float().isfinite().all() and c.H.float().isfinite().all()


@pytest.mark.parametrize("act", [tla.ACT_SILU, tla.ACT_GELU])
def test_gradient_against_autograd_and_differences(act):
    """The pair of calls against float64 autograd of the formula, and a directional
    difference of the forward call itself (bf16 outputs: 2^-9 of a value, over the
    step's size)."""
    rows, N, K = 48, 40, 56
    f = Gated([rows], N, K, tla.BF16, act=act, keep=True, no_offsets=True).call()
    torch.cuda.synchronize()
    g = Grad([rows], N, 72, tla.BF16, act=act, no_offsets=True, seed=3)
    g.Z = f.Z.cpu()[:rows * 2 * N].view(rows, 2 * N).clone()
    g.call().verify()
    z = g.Z.double().requires_grad_()
    dh = g.dY.double() @ g.W[0].double()
    gate = torch.nn.functional.silu(z[:, :N]) if act == tla.ACT_SILU else torch.nn.functional.gelu(z[:, :N])
    want, = torch.autograd.grad((gate * z[:, N:] * dh).sum(), z)
    got, _ = raw(g.D, rows, 2 * N, 2 * N)
    bound = torch.cat([e + x.abs() * 2.0 ** -8 + 1e-9 for _, x, e in g.expect()[:2]], dim=1)
    check(got, want.detach(), bound, "autograd")
    # differences of the formula along a direction
    step = torch.randn(rows, 2 * N, generator=torch.Generator().manual_seed(9), dtype=torch.float64)
    loss = lambda t: (oga.act(t[:, :N], act) * t[:, N:] * dh).sum().item()  # noqa: E731
    zd = g.Z.double()
    diff = (loss(zd + 1e-5 * step) - loss(zd - 1e-5 * step)) / 2e-5
    assert abs(diff - (got.double() * step).sum().item()) <= (bound * step.abs()).sum().item() + 1e-6 * abs(diff)


@pytest.mark.parametrize("make", [lambda: Gated([70, 0, 300], 136, 200, tla.BF16, keep=True),
                                  lambda: Gated([3], 136, 200, tla.BF16),
                                  lambda: Grad([70, 0, 300], 136, 200, tla.BF16)])
def test_streams_and_graphs(make):
    """A side stream; a captured call replayed over changed inputs, each replay
    against the eager call."""
    c = make()
    s = torch.cuda.Stream()
    c.call(stream=s.cuda_stream)
    s.synchronize()
    c.verify()
    out = [t for t in ((c.H, c.Z) if isinstance(c, Gated) else (c.D, c.H)) if t is not None]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.again()
    x = c.args[5]
    for k in range(4):
        x.copy_(x.roll(1) if k else x)
        for t in out:
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        first = [t.clone() for t in out]
        for t in out:
            t.fill_(7.0)
        c.again()
        torch.cuda.synchronize()
        for a, b in zip(first, out):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_two_calls_at_once():
    """Two streams, the same weights, outputs of their own."""
    a, b = (Gated([200], 264, 512, tla.BF16, keep=True).call() for _ in range(2))
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for c, t in zip((a, b), s):
            c.again(stream=t.cuda_stream)
    torch.cuda.synchronize()
    a.verify()
    b.verify()
