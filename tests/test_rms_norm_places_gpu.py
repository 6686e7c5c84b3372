"""GPU tests that where the buffers of the RMS norm lie changes its results by no more than
another order of the sums does."""
from __future__ import annotations

import pytest
import torch

import feed_forward_reference as ref
from test_rms_norm_gpu import ADDS, D_R, DEV, DTYPES, EPS, U, draw, g, half_step, moved  # noqa: F401  (g: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("xt", list(DTYPES))
@pytest.mark.parametrize("dim", [64, 2048, 2050, 4097, 20001])
def test_codes_off_the_grid(g, dim, xt, pow2):  # noqa: F811
    x, r, _, _, w = draw(10, dim, DTYPES[xt], DTYPES[xt], 3)
    want = g.rms_norm_fp8(x, w, residual=r, eps=EPS, pow2=pow2)
    for by in (1, 2, 5):
        Q = torch.empty(10 * dim + 8, dtype=torch.uint8, device=DEV)[by:by + 10 * dim].view(torch.float8_e4m3fn).reshape(10, dim)
        got = g.rms_norm_fp8(x, w, residual=r, eps=EPS, pow2=pow2, Q=Q)
        off = g.rms_norm_fp8(moved(x), moved(w), residual=moved(r), eps=EPS, pow2=pow2)
        for q, s, h in (got, off):
            assert torch.equal(h, want[2])
            sa, sb = (torch.exp2(v.double() - 127) if pow2 else v.double() for v in (s, want[1]))
            if pow2:
                # beside a power of two the maximum's rounding may take the next one
                same = sa == sb
                assert same.double().mean() > 0.95 and ((sa / sb).log2().abs() <= 1).all()
                same = ref.spread(same, 1, 10, dim)
            else:
                # rstd's difference and the products' roundings, in both
                assert ((sa - sb).abs() <= 2 * (D_R + 4 * U) * sb).all()
                same = torch.ones_like(q, dtype=torch.bool)
            a, b = (v.float().double() for v in (q, want[0]))
            # y / s: y's and s's differences, and the quotient's rounding; a code to either side of them
            err = (4 * D_R + 12 * U) * b.abs()
            assert ((a - b).abs() <= 2 * ref.e4m3_half_step(b.abs() + err) + err)[same].all()
            assert (a == b)[same].double().mean() > 0.99
    assert g.check() == g.GEMM_OK


@pytest.mark.parametrize("xt,wt,rows,dim", [("fp16", "fp16", 1300, 4097), ("bf16", "fp32", 1300, 4999), ("fp32", "fp32", 900, 3001),
                                            ("bf16", "bf16", 200, 16371), ("fp16", "fp16", 2001, 514), ("fp32", "fp32", 400, 2048)])
def test_gradients_off_the_grid(g, xt, wt, rows, dim):  # noqa: F811
    x, _, dy, dh, w = draw(rows, dim, DTYPES[xt], DTYPES[wt], rows + dim)
    _, H, rstd = g.rms_norm_fwd(x, w, eps=EPS)
    dX, dg = g.rms_norm_bwd(dy, H, rstd, w, dH=dh)
    z = H.double() * rstd.double()[:, None]
    gr = dy.double() * w.double()
    d_c = (ADDS + 5) * U * (gr * z).abs().mean(-1, keepdim=True)
    c = (gr * z).mean(-1, keepdim=True)
    rel, tiny = half_step(x.dtype)
    # twice what either may be off
    step = rstd.double()[:, None] * (z.abs() * d_c + 6 * U * (gr.abs() + (z * c).abs())) + 2 * U * dX.double().abs()
    step = 2.02 * (step + rel * dX.double().abs() + tiny)
    wrel, wtiny = half_step(w.dtype)
    wstep = 2.02 * ((rows / 152 + 24) * U * (dy.double() * z).abs().sum(0) + wrel * dg.double().abs() + wtiny)
    places = [(moved(H), moved(dy), moved(w), moved(dh)), (moved(H), dy, w, dh), (H, moved(dy), w, moved(dh)), (H, dy, moved(w), dh)]
    for h, y, v, s in places:
        out = g.rms_norm_bwd(y, h, rstd, v, dH=s)
        assert ((out[0].double() - dX.double()).abs() <= step).all()
        assert ((out[1].double() - dg.double()).abs() <= wstep).all()
    assert g.check() == g.GEMM_OK
