"""GEMM operands stored as rows of k (column-major A, row-major B) with 8 rows
128 MiB apart: a slab of the direct copies has 64 rows, whose byte offsets would
pass 2^32 and come back to rows and padding in use.  Eight products summed in
fp32 are off by at most (8 + 4) 2^-24 of the terms' magnitudes, the store by
half a bf16 step, 2^-8."""
import pytest
import torch

import tiled_layout_algebra_amd as tla


def _args(ld, order_a, **kw):
    fake = 1 << 20
    return dict(M=64, N=64, K=8, A=fake, a_type=tla.BF16, a_order=order_a,
                lda=ld if order_a == tla.COL_MAJOR else 8, B=fake, b_type=tla.BF16, b_order=tla.ROW_MAJOR,
                ldb=ld, D=2 * fake, d_type=tla.BF16, d_order=tla.ROW_MAJOR, ldd=64, c_type=tla.BF16,
                bias_type=tla.BF16, alpha=1.0, scale_a=1.0, scale_b=1.0)


@pytest.mark.parametrize("order_a", [tla.ROW_MAJOR, tla.COL_MAJOR])
def test_choice(order_a):
    import ctypes
    for ld, kernel in (((1 << 24) - 8, "gemm_fast_128x128"), (1 << 24, "gemm_general_128x128"),
                       (1 << 26, "gemm_general_128x128")):
        a, buf = tla.GemmArgs(), ctypes.create_string_buffer(64)
        for k, v in _args(ld, order_a).items():
            setattr(a, k, v)
        assert tla.lib().tla_gemm_variant(ctypes.byref(a), buf, 64) == tla.OK
        assert buf.value.decode() == kernel


@pytest.mark.gpu
def test_values():
    K, n, ld = 8, 64, (1 << 26) + 64
    gen = torch.Generator().manual_seed(3)
    mats, bufs = [], []
    for _ in range(2):
        m = torch.randn(K, n, generator=gen).bfloat16()
        buf = torch.full((K, ld), float("nan"), dtype=torch.bfloat16, device="cuda")
        buf[:, :n] = m.cuda()
        mats.append(m.double())
        bufs.append(buf)
    row = mats[0].t().contiguous().bfloat16().cuda()
    for A, order, lda in ((bufs[0], tla.COL_MAJOR, ld), (row, tla.ROW_MAJOR, K)):
        D = torch.empty(n, n, dtype=torch.bfloat16, device="cuda")
        tla.gemm_epilogue(n, n, K, A, tla.BF16, order, lda, bufs[1], tla.BF16, tla.ROW_MAJOR, ld, D,
                          tla.BF16, tla.ROW_MAJOR, n)
        ref, S = mats[0].t() @ mats[1], mats[0].t().abs() @ mats[1].abs()
        err = (D.cpu().double() - ref).abs()
        assert (err <= S * (K + 4) * 2.0 ** -24 + ref.abs() * 2.0 ** -8 + 1e-30).all()
