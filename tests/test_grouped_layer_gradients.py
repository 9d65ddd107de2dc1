"""The gradients of one expert layer x -> gelu(x W1 + b1) W2, element by element.

Each element's bound follows the roundings that reach it: the stored z is off
by its sum's error and half a step; gelu' passes that on with a slope of at most
2 phi(0) < 0.8 and adds 1e-6 (1 + |z|) of its own; dz = g gelu'(z) takes g's sum
error and half a step; dW and db sum dz's errors over the expert's rows, with
|x| as weights for dW, and add (rows + 4) 2^-24 of the terms' magnitudes.  The
tests on the CPU show that the layer with its rounding emulated stays within the bounds
and that a wrong derivative or a lost row does not."""
import math

import pytest
import torch

import tiled_layout_algebra_amd as tla
from oracle import grouped as og
from tests.grouped_util import half_step, offsets_of, values

EPS = 2.0 ** -24


class Layer:
    """Values in f16 and float64 references with the bounds of z, dz, dW and db."""

    def __init__(self, counts, N, K, seed):
        self.counts, self.N, self.K, self.off = counts, N, K, offsets_of(counts)
        self.g, self.rows = len(counts), sum(counts)
        gen = torch.Generator().manual_seed(seed)
        self.x, self.dy = values(gen, (self.rows, K), tla.F16), values(gen, (self.rows, K), tla.F16, 0.1)
        self.W1 = values(gen, (self.g, K, N), tla.F16, K ** -0.5)
        self.W2 = values(gen, (self.g, N, K), tla.F16, N ** -0.5)
        self.b1 = values(gen, (self.g, N), tla.F16)
        z, Sz = og.pre_activation(self.x, self.W1, self.off, bias=self.b1)
        gr, Sg = og.pre_activation(self.dy, self.W2.transpose(1, 2), self.off)
        slope = og.act_slope(z, og.ACT_GELU)
        ez = Sz * (K + 4) * EPS
        ez = ez + half_step(z.abs() + ez, tla.F16)
        es = 0.8 * ez + 1e-6 * (1 + z.abs())
        dz = gr * slope
        edz = gr.abs() * es + Sg * (K + 4) * EPS * (slope.abs() + es) + dz.abs() * 2.0 ** -23
        edz = edz + half_step(dz.abs() + edz, tla.F16)
        self.z, self.gr, self.dz = z, gr, dz
        self.want, self.bound = self.sums(dz), self.errors(edz)

    def sums(self, dz, keep=None):
        """dW, db of a given dz, rows in `keep` only."""
        keep = torch.ones(self.rows, 1, dtype=torch.float64) if keep is None else keep
        dz = dz.double() * keep
        return {"dW": torch.stack([self.x[lo:hi].double().t() @ dz[lo:hi] for lo, hi in og.spans(self.off)]),
                "db": torch.stack([dz[lo:hi].sum(0) for lo, hi in og.spans(self.off)])}

    def errors(self, edz):
        out = {"dW": [], "db": []}
        for lo, hi in og.spans(self.off):
            x, e, n = self.x[lo:hi].double().abs(), edz[lo:hi], (hi - lo + 4) * EPS
            m = self.dz[lo:hi].abs() + e
            out["dW"].append(x.t() @ e + x.t() @ m * n + 1e-30)
            out["db"].append(e.sum(0) + m.sum(0) * n + 1e-30)
        return {k: torch.stack(v) for k, v in out.items()}

    def worst(self, got):
        """The largest share of its bound that an element of each output is off by."""
        return {k: ((got[k].double() - self.want[k]).abs() / self.bound[k]).max().item() for k in self.want}


CASES = [([50, 0, 33], 48, 40, 3), ([260, 1, 0, 700], 136, 96, 4)]


@pytest.mark.parametrize("counts,N,K,seed", CASES, ids=str)
def test_bounds_hold_for_the_roundings_and_for_nothing_else(counts, N, K, seed):
    p = Layer(counts, N, K, seed)
    stored = p.z.half().double()
    dz = (p.gr * og.act_slope(stored, og.ACT_GELU)).half()
    assert all(w <= 1 for w in p.worst(p.sums(dz)).values())
    phi = 0.5 * torch.special.erfc(-p.z / math.sqrt(2.0))
    lost = torch.ones(p.rows, 1, dtype=torch.float64)
    lost[counts[0] // 2] = 0
    for wrong in (p.sums(p.gr * phi), p.sums(p.gr * (p.z > 0)), p.sums(p.gr), p.sums(p.dz, lost)):
        assert all(w > 2 for w in p.worst(wrong).values())


@pytest.mark.gpu
@pytest.mark.parametrize("counts,N,K,seed", CASES, ids=str)
def test_kernels_stay_within_the_bounds(counts, N, K, seed):
    p = Layer(counts, N, K, seed)
    g, rows = p.g, p.rows
    off = torch.tensor(p.off, dtype=torch.int32).cuda()
    x, dy, W1, b1, W2 = (t.cuda() for t in (p.x, p.dy, p.W1, p.b1, p.W2))
    h, z, dz = (torch.empty(rows, N, dtype=torch.float16, device="cuda") for _ in range(3))
    tla.grouped_gemm(g, rows, N, K, off, x, tla.F16, K, W1, tla.ROW_MAJOR, N, K * N, h, tla.F16, N, bias=b1,
                     Z=z, ldz=N, z_mode=tla.Z_STORE, act=tla.ACT_GELU)
    tla.grouped_gemm(g, rows, N, K, off, dy, tla.F16, K, W2, tla.COL_MAJOR, K, K * N, dz, tla.F16, N, Z=z,
                     ldz=N, z_mode=tla.Z_GRAD, act=tla.ACT_GELU)
    dW, db = torch.empty(g, K, N, device="cuda"), torch.empty(g, N, device="cuda")
    tla.grouped_gemm_wgrad(g, rows, N, K, off, x, K, dz, N, tla.F16, dW, tla.F32, tla.ROW_MAJOR, N, K * N,
                           dbias=db)
    worst = p.worst({"dW": dW.cpu(), "db": db.cpu()})
    assert all(w <= 1 for w in worst.values()), worst
